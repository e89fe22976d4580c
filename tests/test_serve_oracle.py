"""CPU checks of the operators around the key/value cache: the fp64 oracle
against hand-worked values and closed forms, the frequencies, the workspace
sizes, and the refusals of the C entry points (which need no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import moe_gqa_query_gqe_b200 as gqe
from moe_gqa_query_gqe_b200 import lib
from gqe_inputs import Dims
from oracle import gqe_ref, serve_ref as ref


# ---- oracle ---------------------------------------------------------------------------
def test_rope_oracle_quarter_turns_and_partial_heads():
    x = np.zeros((1, 1, 64))
    x[0, 0, 0], x[0, 0, 2], x[0, 0, 1], x[0, 0, 63] = 3.0, 5.0, 7.0, 11.0
    f = np.array([math.pi / 2, 0.0])
    half, _ = ref.qk_rope(x, None, f, [1], "half", 4, 0.0, 1.0)      # pairs (0, 2) and (1, 3)
    np.testing.assert_allclose(half[0, 0, :4], [-5.0, 7.0, 3.0, 0.0], atol=1e-12)
    assert half[0, 0, 63] == 11.0
    inter, _ = ref.qk_rope(x, None, f, [1], "interleaved", 4, 0.0, 2.0)  # pairs (0, 1) and (2, 3), scaled
    np.testing.assert_allclose(inter[0, 0, :4], [-14.0, 6.0, 10.0, 0.0], atol=1e-12)
    assert inter[0, 0, 63] == 11.0


def test_rope_oracle_scores_depend_on_distance_only():
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(2, 1, 1, 64))
    f = 10000.0 ** (-np.arange(32) / 32)
    for layout in ("half", "interleaved"):
        s = [(ref.qk_rope(q, None, f, [p + 7], layout, 64, 0.0, 1.0)[0] * ref.qk_rope(k, None, f, [p], layout, 64, 0.0, 1.0)[0]).sum()
             for p in (0, 3, 1000)]
        np.testing.assert_allclose(s, s[0], rtol=1e-10)


def test_rope_oracle_norm_gives_unit_rms():
    x = np.full((1, 1, 64), 3.0)
    y, _ = ref.qk_rope(x, np.full((1, 1, 64), 0.5), np.zeros(1), [9], "half", 2, 0.0, 1.0)
    np.testing.assert_allclose(y, 0.5, rtol=1e-14)


def test_ancestors_of_a_small_tree():
    #  0 -> 1 -> 3, 0 -> 2, and 4 on its own
    sees = ref.ancestors([-1, 0, 0, 1, -1], 5)
    want = [[0], [0, 1], [0, 2], [0, 1, 3], [4]]
    assert [list(np.flatnonzero(r)) for r in sees] == want
    assert ref.ancestors(None, 3).tolist() == np.tril(np.ones((3, 3), bool)).tolist()


def test_tree_oracle_chain_equals_causal_attention():
    rng = np.random.default_rng(1)
    B, T, G, k, L = 2, 5, 2, 2, 6
    Q, Kn, Vn = rng.normal(size=(B * T, 5, 64)), rng.normal(size=(B * T, G, 64)), rng.normal(size=(B * T, G, 64))
    Kc, Vc = rng.normal(size=(2, B, L, G, 64))
    got = ref.tree_attn(Q, Kn, Vn, Kc, Vc, [L, L], None, None, B, T, G, k)
    for b in range(B):
        for g in range(G):
            K = np.concatenate([Kc[b, :, g], Kn[b * T:(b + 1) * T, g]])
            V = np.concatenate([Vc[b, :, g], Vn[b * T:(b + 1) * T, g]])
            for h in ref.group_slots(g, G, k):
                want = gqe_ref.causal_attention(Q[b * T:(b + 1) * T, h], np.arange(L, L + T), K, V, 1 / 8.0)
                # both sides add at most 11 weighted values of size up to 4: about 20 roundings of 4 * 2^-53 each
                np.testing.assert_allclose(got["O"][b * T:(b + 1) * T, h], want, rtol=1e-12, atol=1e-14)


def test_commit_oracle_mass_adds_up_to_one_a_row():
    rng = np.random.default_rng(2)
    B, T, G, k, cap = 1, 4, 2, 1, 12
    Q, Kn, Vn = rng.normal(size=(T, 3, 64)), rng.normal(size=(T, G, 64)), rng.normal(size=(T, G, 64))
    Kc, Vc = rng.normal(size=(2, B, cap, G, 64))
    parent = [-1, 0, 0, 2]
    att = ref.tree_attn(Q, Kn, Vn, Kc, Vc, [5], None, parent, B, T, G, k)
    got = ref.tree_commit([[0, 2, 3, 0]], [3], None, Q, att["lse"], Kn, Vn, [5], Kc, Vc, np.zeros((1, G, cap), int),
                          np.zeros((1, G, cap)), B, T, G, k)
    np.testing.assert_allclose(got["mass"].sum(2), [[6.0, 3.0]], rtol=1e-12)  # 3 tokens, in group 0 the shared row too
    assert got["len"].tolist() == [8] and got["pos"][0, 0, 5:8].tolist() == [5, 6, 7]
    np.testing.assert_array_equal(got["K"][0, 5:8], Kn[[0, 2, 3]])


def test_evict_oracle_by_hand():
    mass = [[[5.0, 1.0, 4.0, 1.0, 9.0, 1.0, 0.0, 3.0]]]
    pos = [[[0, 1, 2, 3, 4, 5, 6, 7]]]
    # keep 4 of 8: row 0 is the sink, row 7 recent, then 4 (9.0) and 2 (4.0)
    assert ref.cache_evict(4, 1, 1, [8], [8], mass, pos, 1, 1) == [[[0, 4, 2, 7]]]
    # ties go to the lower row: 1, 3 and 5 are equal, one of them stays
    assert ref.cache_evict(5, 0, 0, [8], [8], mass, pos, 1, 1) == [[[0, 1, 2, 7, 4]]]
    assert ref.cache_evict(8, 1, 1, [8], [8], mass, pos, 1, 1) == [[list(range(8))]]
    # NaN is last, an order of positions of its own
    mass[0][0][0] = float("nan")
    assert ref.cache_evict(2, 0, 1, [8], [4], mass, [[[9, 8, 7, 3, 2, 1, 0, -5]]], 1, 1) == [[[0, 1]]]


# ---- frequencies ------------------------------------------------------------------------
def test_rope_frequencies():
    f, s = gqe.rope_frequencies(64, device="cpu")
    assert s == 1.0 and f.dtype == torch.float32
    want = 10000.0 ** (-np.arange(32) / 32)
    # rounded once: half a step of fp32
    assert (np.abs(f.double().numpy() - want) <= 2.0 ** -24 * want * 1.0001).all()
    lin, s = gqe.rope_frequencies(64, scaling="linear", factor=8.0, device="cpu")
    assert s == 1.0 and torch.equal(lin, f / 8.0)  # a power of two: exact
    ntk, _ = gqe.rope_frequencies(64, scaling="ntk", factor=8.0, device="cpu")
    assert ntk[0] == f[0] and abs(float(ntk[-1] / f[-1]) * 8.0 - 1.0) < 1e-6
    yarn, s = gqe.rope_frequencies(64, scaling="yarn", factor=8.0, trained_len=4096, device="cpu")
    assert abs(s - (0.1 * math.log(8.0) + 1.0)) < 1e-15
    r = (yarn / f).double().numpy()
    turns = 4096 * want / (2 * math.pi)
    assert (r[turns > 40] == 1.0).all() and (np.abs(r[turns < 0.9] * 8.0 - 1.0) < 1e-6).all()
    assert ((np.diff(r) <= 1e-7) & (r[1:] <= 1.0) & (r[1:] >= 0.1249)).all()


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=66), dict(rot=7), dict(rot=64, scaling="other"),
                                dict(rot=64, scaling="linear", factor=0.5), dict(rot=2, scaling="ntk", factor=2.0),
                                dict(rot=64, scaling="yarn", factor=2.0), dict(rot=64, base=1.0)])
def test_rope_frequencies_refusals(kw):
    with pytest.raises(ValueError):
        gqe.rope_frequencies(device="cpu", **kw)


# ---- C entry points: sizes and refusals --------------------------------------------------
D = Dims(B=2, T=16, D=256, G=4, M=2, k=1)
P = 1 << 20  # aligned, never dereferenced


def _raw(name, d, *args):
    return getattr(lib.load(), name)(ctypes.byref(lib.dims_struct(d)), *args)


def _rope(d=D, layout=0, rot=64, eps=1e-6, scale=1.0, Q=P, K=P, wq=P, wk=P, sel=P, inv=P, pos=None, Qo=P, Ko=P):
    return _raw("gqe_qk_rope", d, layout, rot, eps, scale, Q, K, wq, wk, sel, inv, pos, Qo, Ko, None)


NODEV = 0 if torch.cuda.is_available() else -6


@pytest.mark.parametrize("kw", [dict(layout=2), dict(layout=-1), dict(rot=66), dict(rot=-2), dict(rot=31), dict(eps=-1.0),
                                dict(eps=float("nan")), dict(Q=None), dict(Qo=None), dict(K=None), dict(Ko=None),
                                dict(Q=None, Qo=None, K=None, Ko=None), dict(sel=None), dict(inv=None), dict(Q=P + 8),
                                dict(wk=P + 2), dict(pos=P + 4), dict(Ko=P + 8), dict(d=D.with_(T=0))])
def test_rope_refusals(kw):
    assert _rope(**kw) == -1


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
@pytest.mark.parametrize("kw", [dict(), dict(Q=None, Qo=None, sel=None), dict(K=None, Ko=None), dict(wq=None, wk=None, sel=None),
                                dict(rot=0, inv=None), dict(rot=2, layout=1)])
def test_rope_valid_calls_reach_the_device_check(kw):
    assert _rope(**kw) == -6


def test_tree_workspace():
    ws = gqe.workspace_bytes(D, gqe.OP_TREE_ATTN)
    assert 0 < ws < 64 << 20
    assert gqe.workspace_bytes(D.with_(T=129), gqe.OP_TREE_ATTN) == 0
    assert gqe.workspace_bytes(D.with_(k=3), gqe.OP_TREE_ATTN) == 0


def _tree(d=D, cap=100, Q=P, Kn=P, Vn=P, Kc=P, Vc=P, L=P, n=None, par=None, O=2 * P, lse=None, ws=P, nbytes=1 << 40):
    return _raw("gqe_tree_attn", d, cap, Q, Kn, Vn, Kc, Vc, L, n, par, O, lse, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), -1), (dict(Kn=None), -1), (dict(Vn=None), -1), (dict(Kc=None), -1), (dict(Vc=None), -1), (dict(L=None), -1),
    (dict(O=None), -1), (dict(O=P), -1), (dict(O=P + 8), -1), (dict(lse=P + 4), -1), (dict(par=P + 4), -1), (dict(n=P + 4), -1), (dict(cap=0), -1),
    (dict(cap=-5), -1), (dict(d=D.with_(T=129)), -2), (dict(cap=1 << 30), -2), (dict(ws=None), -3), (dict(ws=P + 16), -3),
    (dict(nbytes=16), -3), (dict(d=D.with_(dh=32)), -2)])
def test_tree_refusals(kw, code):
    assert _tree(**kw) == code


def _commit(d=D, cap=100, path=None, n=None, positions=None, Q=P, lse=P, Kn=P, Vn=P, L=P, Kc=P, Vc=P, pos=None, mi=P, mo=P,
            new=2 * P):
    return _raw("gqe_tree_commit", d, cap, path, n, positions, Q, lse, Kn, Vn, L, Kc, Vc, pos, mi, mo, new, None)


@pytest.mark.parametrize("kw,code", [
    (dict(Kn=None), -1), (dict(Vn=None), -1), (dict(L=None), -1), (dict(Kc=None), -1), (dict(Vc=None), -1), (dict(new=None), -1),
    (dict(new=P), -1), (dict(n=2 * P), -1), (dict(mi=None), -1), (dict(mo=None), -1), (dict(Q=None), -1), (dict(lse=None), -1), (dict(path=P + 4), -1),
    (dict(pos=P + 4), -1), (dict(positions=P + 4), -1), (dict(n=P + 4), -1), (dict(cap=0), -1), (dict(d=D.with_(T=200)), -2)])
def test_commit_refusals(kw, code):
    assert _commit(**kw) == code


def _evict(d=D, keep=8, sink=1, recent=2, L=P, nxt=P, Kc=P, Vc=P, mi=P, mo=P, pi=P, po=P, new=2 * P, ws=P, nbytes=1 << 40):
    return _raw("gqe_cache_evict", d, keep, sink, recent, L, nxt, Kc, Vc, mi, mo, pi, po, new, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(keep=0), -1), (dict(keep=-1), -1), (dict(sink=-1), -1), (dict(recent=-1), -1), (dict(sink=4, recent=5), -1),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), -1), (dict(L=None), -1), (dict(nxt=None), -1), (dict(Kc=None), -1),
    (dict(mo=None), -1), (dict(po=P + 4), -1), (dict(new=P), -1), (dict(nxt=2 * P), -1), (dict(ws=None), -3), (dict(nbytes=8), -3), (dict(ws=P + 64), -3)])
def test_evict_refusals(kw, code):
    assert _evict(**kw) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device answer")
def test_valid_cache_calls_reach_the_device_check():
    assert _tree() == -6 and _commit() == -6 and _commit(mi=None, mo=None, Q=None, lse=None) == -6 and _evict() == -6
    with pytest.raises(lib.GqeError):
        gqe.gqe_tree_attn(D, 100, *[None] * 11)
