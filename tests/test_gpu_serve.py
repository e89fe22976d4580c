"""GPU tests of the operators around the key/value cache against the fp64
oracle: norms with rotation, attention of a tree of drafted tokens, commit,
eviction, each alone and in a run of them together.

Tolerances, from the arithmetic of each operator (HALF = half a step of bf16
relative to the value, 2^-8):
  rope    fp32 throughout, rounded once: HALF |y| + 2^-18 times the size of the
          terms added (norm: 64 squares, a reciprocal root of 2 ulp, two
          products; angle and sine and cosine within 2^-21)
  tree    scores in fp32, 64 products: off by s = 2^-17 sum |q_d k_d| / 8 at
          most, e^score by s relative; P rounded to bf16 (HALF of each term),
          the result rounded (HALF): HALF (|O| + sum p|v|) + (2 s + 2^-14) sum p|v|
  lse     s + 2^-20 (1 + |lse|)
  mass    each term by s + 2^-20 (1 + |lse| + |score|) relative, added in fp32:
          R 2^-23 relative more over R rows
"""
import numpy as np
import pytest
import torch

from gqe_inputs import Dims, make_inputs
from oracle import gqe_ref, serve_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_gqa_query_gqe_b200 as gqe
    from _gpu import assert_close_bf16, f64

HALF = torch.finfo(torch.bfloat16).eps / 2
NAN = float("nan")


def bf(rng, *shape, std=1.0):
    return torch.from_numpy(rng.normal(size=shape) * std).to(torch.bfloat16)


def i32(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32)


def within(got, want, tol, what):
    got, want, tol = f64(got), np.asarray(want), np.broadcast_to(tol, np.shape(want))
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {np.nanmax(np.abs(got - want) / np.maximum(tol, 1e-300)):.2f} x the tolerance"


def ok():
    assert gqe.gqe_check_error() == 0


# ---- rope -----------------------------------------------------------------------------
ROPE = [
    (Dims(B=1, T=1, D=64, G=8, M=2, k=1), "half", 64, 0, True),
    (Dims(B=1, T=1, D=64, G=1, M=8, k=8), "interleaved", 64, 1_000_000, True),
    (Dims(B=3, T=37, D=64, G=4, M=2, k=1), "half", 64, 2_000_000_000, True),
    (Dims(B=2, T=19, D=64, G=8, M=4, k=2), "half", 32, 131071, True),
    (Dims(B=2, T=19, D=64, G=8, M=4, k=2), "half", 48, 7, False),
    (Dims(B=5, T=8, D=64, G=2, M=8, k=4), "half", 20, 99999, True),
    (Dims(B=5, T=8, D=64, G=2, M=8, k=4), "half", 2, 99999, True),
    (Dims(B=1, T=300, D=64, G=64, M=1, k=1), "half", 62, 1000, True),
    (Dims(B=1, T=2500, D=64, G=8, M=2, k=1), "interleaved", 20, 1000, True),
    (Dims(B=7, T=333, D=64, G=8, M=8, k=8), "interleaved", 64, 5000, True),
    (Dims(B=2, T=33, D=64, G=16, M=4, k=1), "half", 0, 0, True),
]


def rope_inputs(d, seed, norm, far):
    rng = np.random.default_rng(seed)
    N, Ha = d.B * d.T, d.G * d.k + 1
    x = {"Q": bf(rng, N, Ha, 64), "K": bf(rng, N, d.G, 64, std=3.0),
         "wq": 1 + bf(rng, d.G * d.M + 1, 64, std=0.2) if norm else None, "wk": 1 + bf(rng, d.G, 64, std=0.2) if norm else None}
    x["sel"] = i32(np.sort(np.argsort(rng.random((N, d.G, d.M)), axis=2)[:, :, :d.k], axis=2))
    x["positions"] = i32(far + np.arange(N) % d.T)
    return x


def cu(x):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in x.items()}


def check_rope(d, x, q, k, inv, layout, rot, scale, positions):
    wq = None if x["wq"] is None else ref.query_weights(x["wq"], x["sel"], d.G, d.M)
    wk = None if x["wk"] is None else np.broadcast_to(f64(x["wk"]), (d.B * d.T, d.G, 64))
    for got, src, w, what in ((q, x["Q"], wq, "Q"), (k, x["K"], wk, "K")):
        want, size = ref.qk_rope(src, w, inv.cpu(), positions, layout, rot, 1e-6, scale)
        within(got, want, HALF * np.abs(want) + 2.0 ** -18 * size, what)


@pytest.mark.parametrize("d,layout,rot,far,norm", ROPE, ids=[f"{c[1]}{c[2]}_g{c[0].G}m{c[0].M}k{c[0].k}_n{c[0].B * c[0].T}" for c in ROPE])
def test_rope_matches_oracle(d, layout, rot, far, norm):
    x = rope_inputs(d, 3, norm, far)
    v = cu(x)
    inv, scale = gqe.rope_frequencies(rot, scaling="yarn", factor=4.0, trained_len=2048) if rot else (None, 1.0)
    q, k = torch.full_like(v["Q"], NAN), torch.full_like(v["K"], NAN)
    lay = gqe.ROPE_HALF if layout == "half" else gqe.ROPE_INTERLEAVED
    gqe.gqe_qk_rope(d, v["Q"], v["K"], v["wq"], v["wk"], v["sel"], inv, v["positions"], q, k, layout=lay, rot=rot, scale=scale)
    ok()
    check_rope(d, x, q, k, torch.zeros(0) if inv is None else inv, layout, rot, scale, x["positions"].numpy())
    # in place, and each side alone: the same bits
    q2, k2 = v["Q"].clone(), v["K"].clone()
    gqe.gqe_qk_rope(d, q2, k2, v["wq"], v["wk"], v["sel"], inv, v["positions"], q2, k2, layout=lay, rot=rot, scale=scale)
    q3, k3 = torch.empty_like(q), torch.empty_like(k)
    gqe.gqe_qk_rope(d, v["Q"], None, v["wq"], None, v["sel"], inv, v["positions"], q3, None, layout=lay, rot=rot, scale=scale)
    gqe.gqe_qk_rope(d, None, v["K"], None, v["wk"], None, inv, v["positions"], None, k3, layout=lay, rot=rot, scale=scale)
    ok()
    assert torch.equal(q2, q) and torch.equal(k2, k) and torch.equal(q3, q) and torch.equal(k3, k)


def test_rope_positions_default_and_zero_rows():
    d = Dims(B=3, T=21, D=64, G=4, M=2, k=1)
    x = rope_inputs(d, 4, True, 0)
    x["Q"][5] = 0  # a row of zeros stays zero: eps keeps its norm finite
    v = cu(x)
    inv, _ = gqe.rope_frequencies(64)
    q, k = torch.empty_like(v["Q"]), torch.empty_like(v["K"])
    gqe.gqe_qk_rope(d, v["Q"], v["K"], v["wq"], v["wk"], v["sel"], inv, None, q, k)
    ok()
    check_rope(d, x, q, k, inv, "half", 64, 1.0, np.arange(d.B * d.T) % d.T)
    assert (q[5] == 0).all()


def test_rope_negative_positions_and_expert_out_of_range():
    d = Dims(B=1, T=9, D=64, G=4, M=2, k=1)
    x = rope_inputs(d, 5, True, -100000)
    v = cu(x)
    inv, _ = gqe.rope_frequencies(64)
    q, k = torch.empty_like(v["Q"]), torch.empty_like(v["K"])
    gqe.gqe_qk_rope(d, v["Q"], v["K"], v["wq"], v["wk"], v["sel"], inv, v["positions"], q, k)
    ok()
    check_rope(d, x, q, k, inv, "half", 64, 1.0, x["positions"].numpy())
    bad = v["sel"].clone()
    bad[4, 2, 0] = 2
    q2 = torch.empty_like(q)
    gqe.gqe_qk_rope(d, v["Q"], v["K"], v["wq"], v["wk"], bad, inv, v["positions"], q2, k)
    assert gqe.gqe_check_error() == -7 and gqe.gqe_check_error() == 0
    keep = torch.ones(9, 5, dtype=torch.bool)
    keep[4, 2] = False
    assert torch.equal(q2.cpu()[keep], q.cpu()[keep])


# ---- tree attention ----------------------------------------------------------------------
def random_parents(rng, B, T, shape):
    if shape == "chain":
        return None
    if shape == "roots":
        return np.full((B, T), -1)
    par = np.full((B, T), -1)
    for b in range(B):
        for i in range(1, T):
            par[b, i] = -1 if rng.random() < 0.1 else rng.integers(max(0, i - 6), i)
    return par


def tree_inputs(d, cap, lens, drafts, shape, seed, rotten=True):
    """Everything that a masked place can hold is there: rows past the lengths
    are NaN or infinite."""
    rng = np.random.default_rng(seed)
    N, Ha = d.B * d.T, d.G * d.k + 1
    x = {"Q": bf(rng, N, Ha, 64, std=1.5), "Kn": bf(rng, N, d.G, 64), "Vn": bf(rng, N, d.G, 64),
         "Kc": bf(rng, d.B, cap, d.G, 64), "Vc": bf(rng, d.B, cap, d.G, 64)}
    if rotten:
        for b in range(d.B):
            for key, v in (("Kc", NAN), ("Vc", float("inf"))):
                x[key][b, lens[b]:] = v
            n = d.T if drafts is None else drafts[b]
            for key in ("Q", "Kn", "Vn"):
                x[key][b * d.T + n:(b + 1) * d.T] = NAN
    par = random_parents(rng, d.B, d.T, shape)
    x["parent"] = None if par is None else i32(par.reshape(-1))
    x["lens"], x["drafts"] = i32(lens), None if drafts is None else i32(drafts)
    return x


def run_tree(d, cap, v, O=None, lse=None, ws=None, with_lse=True):
    Ha = d.G * d.k + 1
    O = torch.full((d.B * d.T, Ha, 64), 7.0, dtype=torch.bfloat16, device="cuda") if O is None else O
    lse = torch.full((d.B * d.T, Ha), 7.0, device="cuda") if lse is None and with_lse else lse
    ws = gqe.workspace(d, gqe.OP_TREE_ATTN) if ws is None else ws
    gqe.gqe_tree_attn(d, cap, v["Q"], v["Kn"], v["Vn"], v["Kc"], v["Vc"], v["lens"], v["drafts"], v["parent"], O, lse, ws)
    return O, lse


def check_tree(d, x, O, lse, only=slice(None)):
    want = ref.tree_attn(x["Q"], x["Kn"], x["Vn"], x["Kc"], x["Vc"], x["lens"].numpy(),
                         None if x["drafts"] is None else x["drafts"].numpy(),
                         None if x["parent"] is None else x["parent"].numpy(), d.B, d.T, d.G, d.k)
    live = np.zeros(want["lse"].shape, bool)
    live[only] = ~np.isnan(want["lse"][only])
    s = 2.0 ** -17 * want["score"]
    tol = HALF * (np.abs(want["O"]) + want["terms"]) + (2 * s + 2.0 ** -14)[..., None] * want["terms"]
    within(f64(O)[live], want["O"][live], tol[live], "O")
    within(f64(lse)[live], want["lse"][live], (s + 2.0 ** -20 * (1 + np.abs(want["lse"])))[live], "lse")
    dead = np.isnan(want["lse"])
    assert (f64(O)[dead] == 7.0).all() and (f64(lse)[dead] == 7.0).all(), "rows past draft_len changed"


TREE = [
    # one token: empty cache, one row, around the key blocks
    (Dims(B=6, T=1, D=64, G=4, M=2, k=1), 200, [0, 1, 63, 64, 65, 200], None, "chain"),
    (Dims(B=4, T=1, D=64, G=1, M=8, k=8), 300, [127, 128, 129, 300], [1, 0, 1, 1], "chain"),
    # a row tile of 16, one row more, and of 32 and 64
    (Dims(B=3, T=16, D=64, G=4, M=2, k=1), 700, [650, 0, 64], None, "tree"),
    (Dims(B=3, T=17, D=64, G=4, M=2, k=1), 400, [400, 3, 65], [17, 16, 0], "tree"),
    (Dims(B=2, T=13, D=64, G=8, M=4, k=2), 1501, [1501, 77], [13, 9], "tree"),
    (Dims(B=2, T=33, D=64, G=2, M=8, k=2), 130, [128, 1], [33, 1], "tree"),
    (Dims(B=2, T=63, D=64, G=2, M=4, k=1), 100, [100, 31], None, "tree"),
    (Dims(B=1, T=64, D=64, G=1, M=8, k=4), 333, [333], None, "tree"),
    (Dims(B=2, T=65, D=64, G=4, M=4, k=2), 129, [129, 0], [65, 64], "tree"),
    (Dims(B=1, T=100, D=64, G=8, M=8, k=8), 50, [50], [99], "tree"),
    (Dims(B=1, T=128, D=64, G=4, M=2, k=1), 500, [499], None, "chain"),
    (Dims(B=2, T=128, D=64, G=8, M=1, k=1), 64, [0, 64], [128, 127], "roots"),
    (Dims(B=1, T=128, D=64, G=1, M=8, k=4), 300, [257], None, "tree"),
    # more units than the GPU has room for: no key split
    (Dims(B=40, T=3, D=64, G=16, M=4, k=1), 70, [(i * 7) % 71 for i in range(40)], [i % 4 for i in range(40)], "tree"),
]


@pytest.mark.parametrize("d,cap,lens,drafts,shape", TREE,
                         ids=[f"b{c[0].B}t{c[0].T}g{c[0].G}k{c[0].k}_{c[4]}_{max(c[2])}" for c in TREE])
def test_tree_matches_oracle(d, cap, lens, drafts, shape):
    x = tree_inputs(d, cap, lens, drafts, shape, 11)
    v = cu(x)
    O, lse = run_tree(d, cap, v)
    ok()
    check_tree(d, x, O, lse)
    # the same call again, and without lse: the same bits
    O2, lse2 = run_tree(d, cap, v)
    O3, _ = run_tree(d, cap, v, with_lse=False)
    ok()
    assert torch.equal(O2, O) and torch.equal(lse2, lse) and torch.equal(O3, O)


def roomier(x, cap):
    """The same sequences in caches of `cap` rows, all the others NaN."""
    x = dict(x)
    for key in ("Kc", "Vc"):
        c = torch.full((x[key].shape[0], cap, *x[key].shape[2:]), NAN, dtype=torch.bfloat16, device="cuda")
        c[:, :x[key].shape[1]] = x[key].cuda()
        x[key] = c
    return x


def large_capacity(d):
    """A capacity that has the call take the kernel for long caches (20 million scores)."""
    return 20_000_000 // (d.B * d.G * d.T * d.k) + 130


@pytest.mark.parametrize("d,cap,lens,drafts,shape", [c for c in TREE if c[0].T * c[0].k > 32],
                         ids=[f"b{c[0].B}t{c[0].T}g{c[0].G}k{c[0].k}_{c[4]}_{max(c[2])}" for c in TREE if c[0].T * c[0].k > 32])
def test_tree_in_a_large_cache_matches_oracle(d, cap, lens, drafts, shape):
    x = tree_inputs(d, cap, lens, drafts, shape, 12)
    big = large_capacity(d)
    v = cu(roomier(x, big))
    O, lse = run_tree(d, big, v)
    ok()
    check_tree(d, x, O, lse)
    O2, lse2 = run_tree(d, big, v)
    O3, _ = run_tree(d, big, v, with_lse=False)
    ok()
    assert torch.equal(O2, O) and torch.equal(lse2, lse) and torch.equal(O3, O)


@pytest.mark.parametrize("B,T,k,lens", [(3, 128, 2, [20000, 0, 7001]), (2, 70, 1, [30000, 12345]), (2, 34, 1, [40001, 128])])
def test_tree_long_caches_match_the_formula(B, T, k, lens):
    """Lengths at which a sequence's keys are cut into many ranges, against
    torch in 64 bits (the oracle's loops would take minutes)."""
    d = Dims(B=B, T=T, D=64, G=4, M=2, k=k)
    x = tree_inputs(d, max(lens) + 3, lens, None, "chain", 13)
    big = max(large_capacity(d), max(lens) + 3)
    O, lse = run_tree(d, big, cu(roomier(x, big)))
    ok()
    Ha = d.G * k + 1
    for b, L in enumerate(lens):
        rows = slice(b * T, (b + 1) * T)
        late = torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1)
        for g in range(d.G):
            K = torch.cat([x["Kc"][b, :L, g], x["Kn"][rows, g]]).cuda().double()
            V = torch.cat([x["Vc"][b, :L, g], x["Vn"][rows, g]]).cuda().double()
            for h in ref.group_slots(g, d.G, k):
                q = x["Q"][rows, h].cuda().double()
                s = q @ K.T / 8.0
                s[:, L:][late] = -float("inf")
                p = torch.softmax(s, 1)
                size = (q.abs() @ K.abs().T).amax(1, keepdim=True) / 8.0 * 2.0 ** -17
                terms = p @ V.abs()
                want = p @ V
                # besides the terms above: l adds up to 40 thousand terms in fp32, 2^-24 a step along chains of at most 64
                # a thread and 2^10 blocks
                tol = HALF * (want.abs() + terms) + (2 * size + 2.0 ** -13) * terms
                within(O[rows, h], f64(want), f64(tol), f"O {b} {h}")
                ls = torch.logsumexp(s, 1)
                within(lse[rows, h], f64(ls), f64(size[:, 0]) + 2.0 ** -14 + 2.0 ** -20 * (1 + np.abs(f64(ls))), f"lse {b} {h}")


@pytest.mark.parametrize("B,T,G,k,lens", [(1, 64, 4, 1, [14001]), (2, 33, 4, 1, [15000, 1023]), (3, 60, 2, 2, [9000, 0, 2111]), (1, 128, 1, 8, [9999]),
                                          (1, 40, 64, 1, [5001])])
def test_tree_many_rows_over_cut_caches_match_the_formula(B, T, G, k, lens):
    """More than 32 rows a group over caches below the other kernel's 20 million
    scores, in blocks of 64 rows whose keys are cut into ranges."""
    d = Dims(B=B, T=T, D=64, G=G, M=max(k, 8 // G), k=k)
    cap = max(lens) + 3
    assert T * k > 32 and T * k * G * B * cap < 20_000_000
    x = tree_inputs(d, cap, lens, None, "tree", 14)
    v = cu(x)
    O, lse = run_tree(d, cap, v)
    O2, lse2 = run_tree(d, cap, v)
    ok()
    assert torch.equal(O2, O) and torch.equal(lse2, lse)
    for b, L in enumerate(lens):
        rows = slice(b * T, (b + 1) * T)
        hidden = ~torch.from_numpy(ref.ancestors(x["parent"].numpy().reshape(B, T)[b], T)).cuda()
        for g in range(0, G, max(1, G // 4)):
            K = torch.cat([v["Kc"][b, :L, g], v["Kn"][rows, g]]).double()
            V = torch.cat([v["Vc"][b, :L, g], v["Vn"][rows, g]]).double()
            for h in ref.group_slots(g, G, k):
                q = v["Q"][rows, h].double()
                s = q @ K.T / 8.0
                s[:, L:][hidden] = -float("inf")
                p = torch.softmax(s, 1)
                size = (q.abs() @ K.abs().T).amax(1, keepdim=True) / 8.0 * 2.0 ** -17
                terms, want = p @ V.abs(), p @ V
                # l adds up to 15 thousand terms in fp32, 2^-24 a step along chains of at most 16 a thread and 2^8 blocks
                tol = HALF * (want.abs() + terms) + (2 * size + 2.0 ** -13) * terms
                within(O[rows, h], f64(want), f64(tol), f"O {b} {h}")
                ls = torch.logsumexp(s, 1)
                within(lse[rows, h], f64(ls), f64(size[:, 0]) + 2.0 ** -14 + 2.0 ** -20 * (1 + np.abs(f64(ls))), f"lse {b} {h}")


@pytest.mark.parametrize("k,T,large", [(1, 12, False), (4, 40, False), (4, 40, True), (1, 50, True)])
def test_tree_values_that_are_not_finite_reach_descendants_only(k, T, large):
    d = Dims(B=1, T=T, D=64, G=2, M=4, k=k)
    x = tree_inputs(d, 90, [70], None, "tree", 5)
    cap = large_capacity(d) if large else 90
    par = x["parent"].numpy()
    sees = ref.ancestors(par, T)
    clean = {key: t.clone() if torch.is_tensor(t) else t for key, t in x.items()}
    x["Vn"][3, 1, 7], x["Vn"][6, 1, 8], x["Kn"][8, 0, 2] = float("inf"), NAN, NAN
    O, lse = (f64(t) for t in run_tree(d, cap, cu(roomier(x, cap))))
    Oc, lsec = (f64(t) for t in run_tree(d, cap, cu(roomier(clean, cap))))
    ok()
    hit = np.zeros(O.shape, bool)
    g1, g0 = slice(k, 2 * k), list(range(k)) + [2 * k]
    hit[sees[:, 3], g1, 7] = True
    assert np.isposinf(O[hit]).all() and hit.any()
    nan = np.zeros(O.shape, bool)
    nan[sees[:, 6], g1, 8] = True
    for h in g0:
        nan[sees[:, 8], h] = True
    assert np.isnan(O[nan]).all() and nan.any()
    rest = ~(hit | nan)
    np.testing.assert_array_equal(O[rest], Oc[rest])
    assert np.isnan(lse[sees[:, 8]][:, g0]).all() and np.array_equal(lse[:, g1], lsec[:, g1])


@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("T,k,lens", [(12, 1, [70]), (17, 2, [128, 3]), (34, 1, [5000, 129]), (64, 1, [300]), (100, 1, [257]), (128, 2, [90])])
def test_tree_cached_values_that_are_not_finite(T, k, lens, large):
    """Every token attends the cached rows: an infinite value is infinite in its
    column of the group's rows, one of either sign or a NaN is NaN, and the other columns
    are what they would be (in both kernels, whatever rows share a tile)."""
    d = Dims(B=len(lens), T=T, D=64, G=2, M=4, k=k)
    x = tree_inputs(d, max(lens) + 2, lens, None, "tree", 9)
    for b, L in enumerate(lens):
        V = x["Vc"][b]
        V[0, 1, 3], V[L - 1, 1, 4], V[L // 2, 1, 63] = float("inf"), -float("inf"), NAN
        V[0, 1, 17], V[L - 1, 1, 17] = float("inf"), -float("inf")
        V[L // 3, 0, 0] = float("inf")
        V[:L, 0, 40] = -float("inf")
    x["Vn"][2, 1, 3], x["Vn"][3, 1, 4] = float("inf"), float("inf")  # drafted values of the same columns
    cap = max(large_capacity(d), max(lens) + 2) if large else max(lens) + 2
    O, lse = run_tree(d, cap, cu(roomier(x, cap)))
    ok()
    with np.errstate(invalid="ignore"):
        want = ref.tree_attn(x["Q"], x["Kn"], x["Vn"], x["Kc"], x["Vc"], lens, None, x["parent"].numpy(), d.B, d.T, d.G, d.k)
    got = f64(O)
    for kind in (np.isnan, np.isposinf, np.isneginf):
        assert kind(want["O"]).any()
        np.testing.assert_array_equal(kind(got), kind(want["O"]))
    fine = np.isfinite(want["O"])
    s = 2.0 ** -17 * want["score"]
    tol = HALF * (np.abs(want["O"]) + want["terms"]) + (2 * s + 2.0 ** -14)[..., None] * want["terms"]
    within(got[fine], want["O"][fine], tol[fine], "O")
    within(lse, want["lse"], s + 2.0 ** -20 * (1 + np.abs(want["lse"])), "lse")


@pytest.mark.parametrize("T", [4, 40])
def test_tree_extreme_scores(T):
    """Scores of several thousand either way: the softmax is a choice of one key."""
    d = Dims(B=1, T=T, D=64, G=4, M=2, k=1)
    x = tree_inputs(d, 300, [280], None, "tree", 6)
    x["Q"] *= 64
    x["Kc"][:, 17] *= 32
    cap = 300 if T == 4 else large_capacity(d)
    O, lse = run_tree(d, cap, cu(roomier(x, cap)))
    ok()
    check_tree(d, x, O, lse)


def test_tree_out_of_range_lengths_and_parents_are_reported():
    d = Dims(B=4, T=6, D=64, G=4, M=2, k=1)
    x = tree_inputs(d, 50, [10, 20, 30, 40], None, "tree", 7, rotten=False)
    v = cu(x)
    O, lse = run_tree(d, 50, v)
    ok()
    for key, b, val in (("lens", 1, 51), ("lens", 1, -1), ("drafts", 1, 7), ("drafts", 1, -2)):
        w = dict(v)
        w[key] = i32([10, 20, 30, 40]).cuda() if key == "lens" else i32([6] * 4).cuda()
        w[key][b] = val
        O2, lse2 = run_tree(d, 50, w)
        assert gqe.gqe_check_error() == -7
        assert (O2[6:12] == 7.0).all() and (lse2[6:12] == 7.0).all()
        # (the others' keys may be cut into other ranges: the same up to rounding)
        for rows in (slice(0, 6), slice(12, 24)):
            check_tree(d, x, O2, lse2, only=rows)
    for bad in (3, 5, -2, 2 ** 31 - 1):
        w = dict(v, parent=v["parent"].clone())
        w["parent"][6 + 3] = bad  # token 3 of sequence 1: its own index, a later one, below -1
        O2, lse2 = run_tree(d, 50, w)
        assert gqe.gqe_check_error() == -7
        par = x["parent"].clone()
        par[6 + 3] = -1
        check_tree(d, dict(x, parent=par), O2, lse2)
    assert gqe.gqe_check_error() == 0


def test_tree_single_token_equals_the_decode_step():
    """The attention inside gqe_decode, given the same queries, keys and values."""
    from gqe_inputs import make_decode_inputs
    from test_gpu_decode import run_decode
    d = Dims(B=3, T=300, D=256, G=4, M=2, k=1)
    lens = [0, 131, 299]
    inp = make_decode_inputs(d, lens, seed=1)
    dev = cu(inp)
    step = run_decode(d, dev)
    one = d.with_(T=1)
    seg_off, seg_tok = torch.empty(d.G * d.M * d.B + 1, dtype=torch.int32, device="cuda"), torch.empty(d.B * d.G * d.k, dtype=torch.int32, device="cuda")
    sel, w = torch.empty(3, 4, 1, dtype=torch.int32, device="cuda"), torch.empty(3, 4, 1, device="cuda")
    gqe.gqe_route(one, dev["x_new"], dev["Wr"], dev["br"], sel, w, None, seg_off, seg_tok, None, gqe.workspace(one, gqe.OP_ROUTE))
    Q, K, V = (torch.empty(3, h, 64, dtype=torch.bfloat16, device="cuda") for h in (5, 4, 4))
    gqe.gqe_qproj(one, dev["x_new"], dev["Wq"], dev["Wk"], dev["Wv"], sel, seg_off, seg_tok, Q, K, V)
    O, lse = run_tree(one, d.T, {"Q": Q, "Kn": K, "Vn": V, "Kc": dev["K_cache"], "Vc": dev["V_cache"], "lens": dev["cache_len"],
                                 "drafts": None, "parent": None})
    y = torch.empty(3, 256, dtype=torch.bfloat16, device="cuda")
    gqe.gqe_combine(one, O, w, dev["Wo"], y, gqe.workspace(one, gqe.OP_COMBINE))
    Kc, Vc, new_len = dev["K_cache"].clone(), dev["V_cache"].clone(), torch.empty(3, dtype=torch.int32, device="cuda")
    gqe.gqe_tree_commit(one, d.T, None, None, None, None, None, K, V, dev["cache_len"], Kc, Vc, None, None, None, new_len)
    ok()
    assert torch.equal(sel.cpu(), step["sel"]) and new_len.tolist() == [n + 1 for n in lens]
    assert torch.equal(Kc.cpu(), step["K"]) and torch.equal(Vc.cpu(), step["V"])
    assert_close_bf16(y.cpu(), f64(step["y"]), "y of the two paths")


def test_tree_offsets_past_32_bits():
    """K and V of 2^31 elements and more each: the last rows of the last
    sequence are far beyond 32-bit element offsets."""
    d = Dims(B=2, T=2, D=64, G=64, M=1, k=1)
    cap = 270_000
    Kc = torch.zeros(d.B, cap, d.G, 64, dtype=torch.bfloat16, device="cuda")
    Vc = torch.zeros_like(Kc)
    assert Kc.numel() > 2 ** 31
    x = tree_inputs(d, 300, [300, 300], None, "tree", 8)
    # all but the last 300 rows of each cache are zero keys with zero values: each adds e^0 to l and nothing to O
    Kc[:, cap - 300:], Vc[:, cap - 300:] = x["Kc"].cuda(), x["Vc"].cuda()
    v = dict(cu(x), Kc=Kc, Vc=Vc, lens=i32([cap, cap]).cuda())
    O, lse = run_tree(d, cap, v)
    ok()
    want = ref.tree_attn(x["Q"], x["Kn"], x["Vn"], x["Kc"], x["Vc"], [300, 300], None, x["parent"].numpy(), 2, 2, 64, 1)
    total = np.logaddexp(want["lse"], np.log(cap - 300))
    share = np.exp(want["lse"] - total)[..., None]
    s = 2.0 ** -17 * want["score"]
    # l adds 270 thousand terms in fp32 over splits of at most 64 blocks and more: 2^-23 a step of the longest chain
    chain = cap * 2.0 ** -23 / 64
    within(lse, total, s + chain + 2.0 ** -20 * (1 + total), "lse")
    tol = HALF * (np.abs(want["O"] * share) + want["terms"] * share) + (2 * s + chain + 2.0 ** -14)[..., None] * want["terms"] * share
    within(O, want["O"] * share, tol, "O")


# ---- commit --------------------------------------------------------------------------------
COMMIT = [
    (Dims(B=3, T=1, D=64, G=4, M=2, k=1), 200, [0, 1, 199], None, "none"),
    (Dims(B=4, T=16, D=64, G=4, M=2, k=1), 300, [284, 0, 64, 100], [16, 5, 0, 1], "path"),
    (Dims(B=2, T=13, D=64, G=8, M=4, k=2), 700, [650, 63], [7, 13], "path"),
    (Dims(B=1, T=128, D=64, G=2, M=8, k=4), 400, [272], [128], "none"),
    (Dims(B=1, T=100, D=64, G=1, M=8, k=8), 150, [31], [77], "path"),
    (Dims(B=2, T=40, D=64, G=8, M=1, k=1), 129, [64, 1], [40, 33], "path"),
]


def commit_inputs(d, cap, lens, acc, kind, seed):
    rng = np.random.default_rng(seed)
    x = tree_inputs(d, cap, lens, None, "chain", seed, rotten=False)
    for b in range(d.B):
        x["Kc"][b, lens[b]:], x["Vc"][b, lens[b]:] = 9.0, 9.0
    N, Ha = d.B * d.T, d.G * d.k + 1
    x["acc"] = None if acc is None else i32(acc)
    x["path"] = None
    if kind == "path":
        x["path"] = i32(np.stack([np.concatenate([np.sort(rng.permutation(d.T)[:n]), np.full(d.T - n, -9)]) for n in acc]))
    x["positions"] = i32(rng.integers(0, 10 ** 6, N))
    x["lse"] = torch.from_numpy(rng.normal(size=(N, Ha)) + np.log(np.asarray(lens).repeat(d.T) + 2.0)[:, None] + 1.0).float()
    x["mass"] = torch.from_numpy(rng.random((d.B, d.G, cap))).float()
    x["pos"] = i32(rng.integers(0, 10 ** 6, (d.B, d.G, cap)))
    for b in range(d.B):
        x["mass"][b, :, lens[b]:] = NAN  # a row that was never used
    return x


def run_commit(d, cap, v, mass_out=None):
    Kc, Vc, pos = v["Kc"].clone(), v["Vc"].clone(), v["pos"].clone()
    mass_out = torch.full_like(v["mass"], 5.0) if mass_out is None else mass_out
    new_len = torch.full((d.B,), -1, dtype=torch.int32, device="cuda")
    gqe.gqe_tree_commit(d, cap, v["path"], v["acc"], v["positions"], v["Q"], v["lse"], v["Kn"], v["Vn"], v["lens"], Kc, Vc, pos,
                        v["mass"], mass_out, new_len)
    return Kc, Vc, pos, mass_out, new_len


@pytest.mark.parametrize("d,cap,lens,acc,kind", COMMIT, ids=[f"b{c[0].B}t{c[0].T}g{c[0].G}k{c[0].k}_{c[4]}" for c in COMMIT])
def test_commit_matches_oracle(d, cap, lens, acc, kind):
    x = commit_inputs(d, cap, lens, acc, kind, 21)
    v = cu(x)
    Kc, Vc, pos, mass, new_len = run_commit(d, cap, v)
    ok()
    n = [d.T] * d.B if acc is None else acc
    want = ref.tree_commit(None if x["path"] is None else x["path"].numpy(), n, x["positions"].numpy(), x["Q"], x["lse"], x["Kn"],
                           x["Vn"], lens, x["Kc"], x["Vc"], x["pos"].numpy(), x["mass"], d.B, d.T, d.G, d.k)
    np.testing.assert_array_equal(f64(Kc), want["K"])
    np.testing.assert_array_equal(f64(Vc), want["V"])
    np.testing.assert_array_equal(pos.cpu().numpy(), want["pos"])
    np.testing.assert_array_equal(new_len.cpu().numpy(), want["len"])
    rel = 2.0 ** -17 * want["score"] + 2.0 ** -20 * (1 + float(x["lse"].abs().max()) + want["score"]) + d.T * (d.k + 1) * 2.0 ** -23
    for b in range(d.B):
        m = want["mass"][b, :, :lens[b] + n[b]]
        within(f64(mass)[b, :, :lens[b] + n[b]], m, rel * m + 1e-12, "mass")
        assert (mass[b, :, lens[b] + n[b]:] == 5.0).all(), "sums past the new length changed"
    # in place: the same bits
    w = dict(v, mass=v["mass"].clone())
    again = run_commit(d, cap, w, mass_out=w["mass"])
    ok()
    for b in range(d.B):
        assert torch.equal(again[3][b, :, :lens[b] + n[b]], mass[b, :, :lens[b] + n[b]])


def test_commit_rows_out_of_range_are_reported():
    d = Dims(B=3, T=5, D=64, G=4, M=2, k=1)
    x = commit_inputs(d, 40, [10, 20, 30], [3, 4, 5], "path", 3)
    v = cu(x)
    good = run_commit(d, 40, v)
    ok()
    for key, val in (("lens", 41), ("lens", -3), ("acc", 6), ("acc", -1), ("lens", 38)):  # 38 + 4 drafts are past the capacity
        w = dict(v)
        w[key] = v[key].clone()
        w[key][1] = val
        got = run_commit(d, 40, w)
        assert gqe.gqe_check_error() == -7
        assert torch.equal(got[0][1], v["Kc"][1]) and torch.equal(got[1][1], v["Vc"][1]) and torch.equal(got[2][1], v["pos"][1])
        assert (got[3][1] == 5.0).all() and int(got[4][1]) == int(w["lens"][1])
        for b in (0, 2):
            assert all(torch.equal(a[b], c[b]) or torch.equal(a[b].nan_to_num(), c[b].nan_to_num()) for a, c in zip(got, good))
    w = dict(v, path=v["path"].clone())
    w["path"][1, 2] = 5
    got = run_commit(d, 40, w)
    assert gqe.gqe_check_error() == -7
    assert torch.equal(got[0][1, 22], v["Kc"][1, 22]) and torch.equal(got[0][1, 23], good[0][1, 23])
    assert gqe.gqe_check_error() == 0


@pytest.mark.parametrize("d,cap,lens,acc", [(Dims(B=3, T=5, D=64, G=4, M=2, k=1), 40, [10, 20, 30], [3, 4, 5]),
                                            (Dims(B=2, T=60, D=64, G=2, M=8, k=4), 300, [200, 130], [60, 41])], ids=["few", "many"])
def test_commit_path_index_out_of_range_adds_nothing(d, cap, lens, acc):
    """Its place keeps its K, V and position with a sum of 0; its query rows add
    nothing to the others' sums; new_len counts the place."""
    x = commit_inputs(d, cap, lens, acc, "path", 4)
    j, L, n = acc[1] - 2, lens[1], acc[1]
    token = int(x["path"][1, j])
    for bad in (-1, d.T, 2 ** 31 - 1):
        v = cu(x)
        v["path"][1, j] = bad
        Kc, Vc, pos, mass, new_len = run_commit(d, cap, v)
        assert gqe.gqe_check_error() == -7
        assert new_len.tolist() == [a + b for a, b in zip(lens, acc)]
        assert torch.equal(Kc[1, L + j], v["Kc"][1, L + j]) and torch.equal(Vc[1, L + j], v["Vc"][1, L + j])
        assert torch.equal(pos[1, :, L + j], v["pos"][1, :, L + j]) and (mass[1, :, L + j] == 0).all()
        # the formula without that token's rows: a log-sum of +infinity is a weight of zero
        silent = x["lse"].clone()
        silent[d.T + token] = float("inf")
        want = ref.tree_commit(x["path"].numpy(), acc, x["positions"].numpy(), x["Q"], silent, x["Kn"], x["Vn"], lens, x["Kc"], x["Vc"],
                               x["pos"].numpy(), x["mass"], d.B, d.T, d.G, d.k)
        keep = np.arange(L + n) != L + j
        np.testing.assert_array_equal(f64(Kc)[1, :L + n][keep], want["K"][1, :L + n][keep])
        rel = 2.0 ** -17 * want["score"] + 2.0 ** -20 * (1 + float(x["lse"].abs().max()) + want["score"]) + d.T * (d.k + 1) * 2.0 ** -23
        m = want["mass"][1, :, :L + n][:, keep]
        within(f64(mass)[1, :, :L + n][:, keep], m, rel * m + 1e-12, "mass")
    assert gqe.gqe_check_error() == 0


@pytest.mark.parametrize("d,cap,lens", [(Dims(B=2, T=9, D=64, G=4, M=2, k=1), 300, [280, 130]), (Dims(B=1, T=25, D=64, G=2, M=8, k=4), 700, [640]),
                                        (Dims(B=1, T=128, D=64, G=1, M=8, k=8), 300, [129])], ids=["few", "many", "most"])
def test_commit_weights_of_zero_add_nothing(d, cap, lens):
    """e^-300 is no fp32 number, and a token does not see the places behind its
    own: sums of such weights alone are exactly zero, whatever columns of the
    products they fall in."""
    x = commit_inputs(d, cap, lens, None, "none", 22)
    far = dict(x, lse=torch.full_like(x["lse"], 300.0), mass=torch.zeros_like(x["mass"]))
    mass = run_commit(d, cap, cu(far))[3]
    last = dict(x, lse=x["lse"].clone(), mass=torch.zeros_like(x["mass"]))
    last["lse"].view(d.B, d.T, -1)[:, -1] = 300.0
    mass_last = run_commit(d, cap, cu(last))[3]
    ok()
    for b, L in enumerate(lens):
        assert (mass[b, :, :L + d.T] == 0).all()
        assert (mass_last[b, :, L + d.T - 1] == 0).all() and (mass_last[b, :, :L + d.T - 1] > 0).all()


@pytest.mark.parametrize("value", [NAN, -float("inf")])
@pytest.mark.parametrize("d,cap,L,n", [(Dims(B=1, T=12, D=64, G=4, M=2, k=1), 300, 200, 10), (Dims(B=1, T=60, D=64, G=2, M=8, k=4), 500, 300, 60)],
                         ids=["few", "many"])
def test_commit_weights_that_are_not_numbers_reach_what_their_token_sees(d, cap, L, n, value):
    """A log-sum of NaN, or of -infinity (all of its scores are -infinity), makes
    NaN of the group's cached sums and of those up to the token's own place; the
    places behind, which the token does not see, keep theirs."""
    x = commit_inputs(d, cap, [L], [n], "path", 23)
    for j in (0, 1, n // 2, n - 2, n - 1):
        for slot in (0, d.k, d.G * d.k):  # of group 0, group 1, and the shared head of group 0
            y = dict(x, lse=x["lse"].clone(), Q=x["Q"].clone(), Kc=x["Kc"].abs(), Kn=x["Kn"].abs())
            base = run_commit(d, cap, cu(y))[3]
            tok = int(x["path"][0, j])
            y["lse"][tok, slot] = value
            if value == -float("inf"):
                y["Q"][tok, slot] = 0
                y["Q"][tok, slot, 5] = -float("inf")  # (keys are not negative here)
            mass = run_commit(d, cap, cu(y))[3]
            want = torch.zeros_like(mass, dtype=torch.bool)
            want[0, 1 if slot == d.k else 0, :L + j + 1] = True
            assert torch.equal(mass.isnan() & ~base.isnan(), want & ~base.isnan()), (j, slot)
            rest = ~(want | base.isnan())
            assert torch.equal(mass[rest], base[rest]), (j, slot)
    ok()


# ---- eviction ------------------------------------------------------------------------------
EVICT = [
    (Dims(B=1, T=8, D=64, G=8, M=1, k=1), [8], 7, 1, 1),
    (Dims(B=3, T=50, D=64, G=4, M=2, k=1), [50, 20, 0], 20, 2, 5),
    (Dims(B=2, T=1500, D=64, G=2, M=4, k=1), [1500, 1025], 1024, 4, 256),
    (Dims(B=2, T=5000, D=64, G=1, M=8, k=2), [5000, 4097], 512, 4, 100),
    (Dims(B=1, T=20011, D=64, G=8, M=2, k=1), [20011], 1, 0, 1),
    (Dims(B=1, T=40000, D=64, G=1, M=8, k=1), [39999], 39998, 0, 0),
    (Dims(B=2, T=3000, D=64, G=8, M=2, k=1), [3000, 2999], 1500, 700, 800),
    (Dims(B=1, T=70001, D=64, G=2, M=4, k=1), [70001], 9000, 8, 1000),
    # more rows than a cluster holds keys of
    (Dims(B=1, T=400_000, D=64, G=1, M=8, k=1), [399_999], 100_000, 4, 1000),
]


def evict_inputs(d, lens, seed, kind="mixed"):
    rng = np.random.default_rng(seed)
    m = np.exp(2 * rng.normal(size=(d.B, d.G, d.T)))
    if kind == "mixed":
        u = rng.random(m.shape)
        m = np.where(u < 0.2, np.round(m * 4) / 4, np.where(u < 0.25, 0.0, m))
        m.reshape(-1)[rng.integers(0, m.size, max(1, m.size // 50))] = np.nan
        m.reshape(-1)[rng.integers(0, m.size, max(1, m.size // 100))] = -0.0
        m.reshape(-1)[rng.integers(0, m.size, max(1, m.size // 100))] = np.inf
    elif kind == "equal":
        m = np.ones_like(m)
    pos = np.argsort(rng.random((d.B, d.G, 2 * d.T)), axis=2)[:, :, :d.T]
    return {"lens": i32(lens), "nxt": i32([2 * d.T] * d.B), "mass": torch.from_numpy(m).float(), "pos": i32(pos),
            "Kc": bf(rng, d.B, d.T, d.G, 64), "Vc": bf(rng, d.B, d.T, d.G, 64)}


def run_evict(d, keep, sink, recent, v, in_place=False, ws=None):
    Kc, Vc = v["Kc"].clone(), v["Vc"].clone()
    mo, po = (v["mass"].clone(), v["pos"].clone()) if in_place else (torch.full_like(v["mass"], 5.0), torch.full_like(v["pos"], -5))
    mi, pi = (mo, po) if in_place else (v["mass"], v["pos"])
    new_len = torch.full((d.B,), -1, dtype=torch.int32, device="cuda")
    gqe.gqe_cache_evict(d, keep, sink, recent, v["lens"], v["nxt"], Kc, Vc, mi, mo, pi, po, new_len,
                        gqe.workspace(d, gqe.OP_CACHE_EVICT) if ws is None else ws)
    return Kc, Vc, mo, po, new_len


def check_evict(d, keep, sink, recent, x, got, in_place=False):
    src = ref.cache_evict(keep, sink, recent, x["lens"].numpy(), x["nxt"].numpy(), x["mass"].numpy(), x["pos"].numpy(), d.B, d.G)
    Kc, Vc, mo, po, new_len = (t.cpu() for t in got)
    for b in range(d.B):
        n = min(int(x["lens"][b]), keep)
        assert int(new_len[b]) == n
        for g in range(d.G):
            rows = torch.as_tensor(src[b][g], dtype=torch.long)
            for new, old in ((Kc, x["Kc"]), (Vc, x["Vc"])):
                assert torch.equal(new[b, :n, g], old[b, rows, g]) and torch.equal(new[b, n:, g], old[b, n:, g])
            assert torch.equal(po[b, g, :n], x["pos"][b, g, rows])
            np.testing.assert_array_equal(mo[b, g, :n].numpy(), x["mass"][b, g, rows].numpy())
            if not in_place:
                assert (po[b, g, n:] == -5).all() and (mo[b, g, n:] == 5.0).all()


@pytest.mark.parametrize("d,lens,keep,sink,recent", EVICT, ids=[f"b{c[0].B}g{c[0].G}_{max(c[1])}to{c[2]}" for c in EVICT])
def test_evict_matches_oracle(d, lens, keep, sink, recent):
    x = evict_inputs(d, lens, 31)
    v = cu(x)
    check_evict(d, keep, sink, recent, x, run_evict(d, keep, sink, recent, v))
    check_evict(d, keep, sink, recent, x, run_evict(d, keep, sink, recent, v, in_place=True), in_place=True)
    ok()


def test_evict_equal_masses_keep_the_lower_rows():
    d = Dims(B=2, T=2500, D=64, G=4, M=2, k=1)
    x = evict_inputs(d, [2500, 1300], 32, "equal")
    check_evict(d, 1200, 3, 40, x, run_evict(d, 1200, 3, 40, cu(x)))
    ok()


def test_evict_length_out_of_range_is_reported():
    d = Dims(B=3, T=100, D=64, G=4, M=2, k=1)
    x = evict_inputs(d, [100, 90, 80], 33)
    v = cu(x)
    for bad in (101, -1):
        w = dict(v, lens=i32([100, bad, 80]).cuda())
        got = run_evict(d, 30, 1, 5, w)
        assert gqe.gqe_check_error() == -7
        assert torch.equal(got[0][1], v["Kc"][1]) and (got[2][1] == 5.0).all() and int(got[4][1]) == bad
        sub = {k: t[[0, 2]] for k, t in x.items()}
        check_evict(d.with_(B=2), 30, 1, 5, sub, [t[[0, 2]] for t in got])
    assert gqe.gqe_check_error() == 0


def test_most_sequences():
    """1024 sequences, as many as the dimensions allow, some without drafts or
    cache, through tree attention, commit and eviction."""
    d, cap = Dims(B=1024, T=2, D=64, G=8, M=1, k=1), 12
    lens, drafts = [(7 * b) % 10 for b in range(1024)], [b % 3 for b in range(1024)]
    x = tree_inputs(d, cap, lens, drafts, "chain", 17)
    O, lse = run_tree(d, cap, cu(x))
    ok()
    check_tree(d, x, O, lse)
    c = commit_inputs(d, cap, lens, drafts, "none", 18)
    Kc, Vc, pos, mass, new_len = run_commit(d, cap, cu(c))
    ok()
    want = ref.tree_commit(None, drafts, c["positions"].numpy(), c["Q"], c["lse"], c["Kn"], c["Vn"], lens, c["Kc"], c["Vc"],
                           c["pos"].numpy(), c["mass"], d.B, d.T, d.G, d.k)
    np.testing.assert_array_equal(f64(Kc), want["K"])
    np.testing.assert_array_equal(pos.cpu().numpy(), want["pos"])
    np.testing.assert_array_equal(new_len.cpu().numpy(), want["len"])
    used = np.broadcast_to(np.arange(cap)[None, None] < want["len"][:, None, None], want["mass"].shape)
    rel = 2.0 ** -17 * want["score"] + 2.0 ** -20 * (1 + float(c["lse"].abs().max()) + want["score"]) + 2.0 ** -19
    within(f64(mass)[used], want["mass"][used], rel * want["mass"][used] + 1e-12, "mass")
    e = evict_inputs(d.with_(T=cap), lens, 19)
    check_evict(d.with_(T=cap), 5, 1, 2, e, run_evict(d.with_(T=cap), 5, 1, 2, cu(e)))
    ok()


# ---- together ------------------------------------------------------------------------------
def layer_inputs(d, seed):
    inp = make_inputs(d, seed=seed)
    rng = np.random.default_rng(seed)
    inp["wq"], inp["wk"] = 1 + bf(rng, d.G * d.M + 1, 64, std=0.2), 1 + bf(rng, d.G, 64, std=0.2)
    return cu(inp)


def project(d, x, dev, positions, inv):
    """Router, projections, norms and rotation of B x T tokens."""
    N, Ha = d.B * d.T, d.G * d.k + 1
    e = dict(device="cuda", dtype=torch.int32)
    sel, w = torch.empty(N, d.G, d.k, **e), torch.empty(N, d.G, d.k, device="cuda")
    seg_off, seg_tok = torch.empty(d.B * d.G * d.M + 1, **e), torch.empty(N * d.G * d.k, **e)
    gqe.gqe_route(d, x, dev["Wr"], dev["br"], sel, w, None, seg_off, seg_tok, None, gqe.workspace(d, gqe.OP_ROUTE))
    Q, K, V = (torch.empty(N, h, 64, dtype=torch.bfloat16, device="cuda") for h in (Ha, d.G, d.G))
    gqe.gqe_qproj(d, x, dev["Wq"], dev["Wk"], dev["Wv"], sel, seg_off, seg_tok, Q, K, V)
    gqe.gqe_qk_rope(d, Q, K, dev["wq"], dev["wk"], sel, inv, positions, Q, K, rot=2 * inv.numel())
    return sel, w, Q, K, V


def combine(d, O, w, dev):
    y = torch.empty(d.B * d.T, d.D, dtype=torch.bfloat16, device="cuda")
    gqe.gqe_combine(d, O, w, dev["Wo"], y, gqe.workspace(d, gqe.OP_COMBINE))
    return y


@pytest.mark.parametrize("k", [1, 2])
def test_chunks_over_the_cache_equal_the_prompt_pass(k):
    """A prompt in chunks of several sizes through rope, tree attention and
    commit gives what the whole-prompt stages (gqe_attn) give."""
    full = Dims(B=2, T=230, D=256, G=4, M=4, k=k)
    dev = layer_inputs(full, 41)
    inv, _ = gqe.rope_frequencies(64)
    sel, w, Q, K, V = project(full, dev["x"], dev, None, inv)
    O = torch.empty_like(Q)
    gqe.gqe_attn(full, Q, K, V, O)
    y = combine(full, O, w, dev)
    cap = 256
    Kc, Vc = (torch.full((2, cap, 4, 64), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mass, pos = torch.full((2, 4, cap), NAN, device="cuda"), torch.full((2, 4, cap), -1, dtype=torch.int32, device="cuda")
    lens, t0 = [torch.zeros(2, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")], 0
    x = dev["x"].view(2, 230, 256)
    for T in (100, 1, 128, 1):
        d = full.with_(T=T)
        at = (torch.arange(T, device="cuda").repeat(2) + t0).int()
        sel, w, q, kn, vn = project(d, x[:, t0:t0 + T].reshape(-1, 256).contiguous(), dev, at, inv)
        o, lse = torch.empty_like(q), torch.empty(2 * T, 4 * k + 1, device="cuda")
        gqe.gqe_tree_attn(d, cap, q, kn, vn, Kc, Vc, lens[0], None, None, o, lse, gqe.workspace(d, gqe.OP_TREE_ATTN))
        got = combine(d, o, w, dev).view(2, T, 256)
        gqe.gqe_tree_commit(d, cap, None, None, at, q, lse, kn, vn, lens[0], Kc, Vc, pos, mass, mass, lens[1])
        lens.reverse()
        assert_close_bf16(got, f64(y.view(2, 230, 256)[:, t0:t0 + T]), f"chunk of {T} at {t0}")
        t0 += T
    ok()
    assert lens[0].tolist() == [230, 230] and torch.equal(Kc[:, :230].reshape(-1, 4, 64), K) and torch.equal(Vc[:, :230].reshape(-1, 4, 64), V)
    assert torch.equal(pos[:, :, :230], torch.arange(230, device="cuda", dtype=torch.int32).expand(2, 4, 230))
    rows = torch.full((2, 4), 230.0 * k)
    rows[:, 0] += 230
    np.testing.assert_allclose(f64(mass[:, :, :230]).sum(2), f64(rows), rtol=1e-4)  # each row's weights add up to one
    # rows past the end are left as they were
    assert Kc[:, 230:].isnan().all() and mass[:, :, 230:].isnan().all() and (pos[:, :, 230:] == -1).all()


def test_a_round_of_drafts_commit_and_eviction_matches_the_oracle():
    """Two steps of a server with a bounded cache: drafts in a tree, the
    accepted path committed, the cache cut to its budget, and the next drafts
    over what is left; every step against the oracle on the step's own inputs."""
    d, cap, keep = Dims(B=2, T=9, D=256, G=4, M=2, k=1), 64, 24
    dev = layer_inputs(d, 42)
    inv, _ = gqe.rope_frequencies(32)
    rng = np.random.default_rng(42)
    st = tree_inputs(d, cap, [30, 20], None, "tree", 42)
    for key in ("Kc", "Vc"):
        st[key] *= 0.6
    v = cu(st)
    mass, pos = torch.from_numpy(rng.random((2, 4, cap))).float().cuda(), torch.arange(cap, device="cuda", dtype=torch.int32).expand(2, 4, cap).contiguous()
    lens, new_len, nxt = v["lens"], torch.empty_like(v["lens"]), [30, 20]
    parent = i32([-1, 0, 0, 1, 1, 3, 2, 6, -1] * 2)
    for step in range(2):
        at = i32(np.concatenate([[nxt[b] + s for s in (0, 1, 1, 2, 2, 3, 2, 3, 0)] for b in range(2)])).cuda()
        xs = bf(rng, 18, 256).cuda()
        sel, w, q, kn, vn = project(d, xs, dev, at, inv)
        x = {"Q": q.cpu(), "Kn": kn.cpu(), "Vn": vn.cpu(), "Kc": v["Kc"].cpu(), "Vc": v["Vc"].cpu(), "lens": lens.cpu(), "drafts": None, "parent": parent}
        O, lse = run_tree(d, cap, cu(x))
        check_tree(d, x, O, lse)
        path, acc = i32([[0, 1, 3, 5] + [0] * 5, [0, 2] + [0] * 7]), i32([4, 2 - step])
        m0, p0 = mass.cpu(), pos.cpu()
        gqe.gqe_tree_commit(d, cap, path.cuda(), acc.cuda(), at, q, lse, kn, vn, lens, v["Kc"], v["Vc"], pos, mass, mass, new_len)
        want = ref.tree_commit(path.numpy(), acc.tolist(), at.cpu().numpy(), x["Q"], lse.cpu(), x["Kn"], x["Vn"], x["lens"].tolist(),
                               x["Kc"], x["Vc"], p0.numpy(), m0, 2, 9, 4, 1)
        n = want["len"]
        assert new_len.tolist() == n.tolist()
        for b in range(2):
            np.testing.assert_array_equal(f64(v["Kc"])[b, :n[b]], want["K"][b, :n[b]])
            np.testing.assert_array_equal(pos.cpu().numpy()[b, :, :n[b]], want["pos"][b, :, :n[b]])
            rel = 2.0 ** -16 * want["score"] + 2.0 ** -18 * (1 + float(lse.abs().max()))
            m = want["mass"][b, :, :n[b]]
            within(f64(mass)[b, :, :n[b]], m, rel * m, "mass")
        nxt = [nxt[b] + int(acc[b]) for b in range(2)]
        e = {"lens": new_len.cpu(), "nxt": i32(nxt), "mass": mass.cpu(), "pos": pos.cpu(), "Kc": v["Kc"].cpu(), "Vc": v["Vc"].cpu()}
        lens = torch.empty_like(new_len)
        dc = d.with_(T=cap)
        gqe.gqe_cache_evict(dc, keep, 2, 6, new_len, i32(nxt).cuda(), v["Kc"], v["Vc"], mass, mass, pos, pos, lens, gqe.workspace(dc, gqe.OP_CACHE_EVICT))
        nan_rows = {k: t for k, t in e.items()}
        src = ref.cache_evict(keep, 2, 6, e["lens"].numpy(), nxt, e["mass"].numpy(), e["pos"].numpy(), 2, 4)
        for b in range(2):
            for g in range(4):
                rows = torch.as_tensor(src[b][g])
                assert torch.equal(v["Kc"].cpu()[b, :len(rows), g], nan_rows["Kc"][b, rows, g])
                assert torch.equal(pos.cpu()[b, g, :len(rows)], e["pos"][b, g, rows])
        assert lens.tolist() == [min(keep, int(i)) for i in n]
    ok()


def test_captured_steps_replay_with_new_contents():
    """rope, tree attention, commit and eviction in one CUDA graph: a replay
    works on what the buffers hold then."""
    d, cap = Dims(B=2, T=5, D=64, G=4, M=2, k=1), 300
    dc = d.with_(T=cap)
    inv, _ = gqe.rope_frequencies(64)

    def inputs(seed):
        x = tree_inputs(d, cap, [200, 120], [5, 3], "tree", seed, rotten=False)
        r = rope_inputs(d, seed, True, 500)
        x.update({k: r[k] for k in ("wq", "wk", "sel", "positions")})
        g = torch.Generator().manual_seed(seed)
        x["mass"], x["pos"] = torch.rand(2, 4, cap, generator=g), torch.arange(cap, dtype=torch.int32).expand(2, 4, cap).contiguous()
        x["acc"] = i32([4, 2])
        return cu(x)

    def outputs():
        z = dict(device="cuda")
        return {"q": torch.zeros(10, 5, 64, dtype=torch.bfloat16, **z), "k": torch.zeros(10, 4, 64, dtype=torch.bfloat16, **z),
                "O": torch.zeros(10, 5, 64, dtype=torch.bfloat16, **z), "lse": torch.zeros(10, 5, **z), "n1": torch.zeros(2, dtype=torch.int32, **z),
                "n2": torch.zeros(2, dtype=torch.int32, **z), "mass": torch.zeros(2, 4, cap, **z), "pos": torch.zeros(2, 4, cap, dtype=torch.int32, **z),
                "nxt": i32([204, 122]).cuda(), "ws1": gqe.workspace(d, gqe.OP_TREE_ATTN), "ws2": gqe.workspace(dc, gqe.OP_CACHE_EVICT)}

    def step(v, o):
        gqe.gqe_qk_rope(d, v["Q"], v["Kn"], v["wq"], v["wk"], v["sel"], inv, v["positions"], o["q"], o["k"])
        gqe.gqe_tree_attn(d, cap, o["q"], o["k"], v["Vn"], v["Kc"], v["Vc"], v["lens"], v["drafts"], v["parent"], o["O"], o["lse"], o["ws1"])
        gqe.gqe_tree_commit(d, cap, None, v["acc"], v["positions"], o["q"], o["lse"], o["k"], v["Vn"], v["lens"], v["Kc"], v["Vc"], v["pos"],
                            v["mass"], o["mass"], o["n1"])
        gqe.gqe_cache_evict(dc, 90, 4, 20, o["n1"], o["nxt"], v["Kc"], v["Vc"], o["mass"], o["mass"], v["pos"], o["pos"], o["n2"], o["ws2"])

    want = []
    for seed in (1, 2):
        v, o = inputs(seed), outputs()
        step(v, o)
        want.append((v, o))
    ok()
    v, o = inputs(1), outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(v, o)
    for seed, (wv, wo) in ((1, want[0]), (2, want[1])):
        for key, t in inputs(seed).items():
            if torch.is_tensor(t):
                v[key].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for key in ("q", "k", "O", "lse", "n1", "n2"):
            assert torch.equal(o[key], wo[key]), key
        for key in ("Kc", "Vc"):
            assert torch.equal(v[key], wv[key]), key
        for key in ("mass", "pos"):
            assert torch.equal(o[key][:, :, :90], wo[key][:, :, :90]), key
    ok()


def test_two_streams_with_workspaces_of_their_own():
    d, cap = Dims(B=2, T=16, D=64, G=8, M=2, k=1), 3000
    xs = [cu(tree_inputs(d, cap, [2900, 1000], None, "tree", s)) for s in (1, 2)]
    want = [run_tree(d, cap, x) for x in xs]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    buf = [(torch.empty_like(O), torch.empty_like(l), gqe.workspace(d, gqe.OP_TREE_ATTN)) for O, l in want]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, x, (O, l, ws) in zip(streams, xs, buf):
            gqe.gqe_tree_attn(d, cap, x["Q"], x["Kn"], x["Vn"], x["Kc"], x["Vc"], x["lens"], None, x["parent"], O, l, ws, stream=s)
    torch.cuda.synchronize()
    for (O, l, _), (Ow, lw) in zip(buf, want):
        assert torch.equal(O, Ow) and torch.equal(l, lw)
    ok()


def test_two_streams_of_commits_and_evictions():
    """Calls at once on buffers of their own, in place and call after call, give
    what they give one by one."""
    d, cap, keep = Dims(B=3, T=8, D=64, G=8, M=2, k=1), 6000, 3000
    dc = d.with_(T=cap)

    def state(seed):
        x = cu(commit_inputs(d, cap, [5000, 3100, 800], [8, 0, 3], "path", seed))
        x["pos"] = torch.arange(cap, dtype=torch.int32, device="cuda").expand(d.B, d.G, cap).contiguous()
        x.update(n1=torch.empty_like(x["lens"]), n2=torch.empty_like(x["lens"]), nxt=i32([6000] * 3).cuda(), ws=gqe.workspace(dc, gqe.OP_CACHE_EVICT))
        return x

    def steps(x, stream):
        at, to = x["lens"], x["n1"]
        for _ in range(4):
            gqe.gqe_tree_commit(d, cap, x["path"], x["acc"], x["positions"], x["Q"], x["lse"], x["Kn"], x["Vn"], at, x["Kc"], x["Vc"], x["pos"],
                                x["mass"], x["mass"], to, stream=stream)
            gqe.gqe_cache_evict(dc, keep, 4, 100, to, x["nxt"], x["Kc"], x["Vc"], x["mass"], x["mass"], x["pos"], x["pos"], x["n2"], x["ws"], stream=stream)
            at, to = x["n2"], x["n1"]

    want = [state(s) for s in (61, 62)]
    for x in want:
        steps(x, None)
        torch.cuda.synchronize()
    got, streams = [state(s) for s in (61, 62)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for x, s in zip(got, streams):
        steps(x, s)
    torch.cuda.synchronize()
    ok()
    for x, w in zip(got, want):
        assert w["n2"].tolist() == [3000, 3000, 812] and torch.equal(x["n2"], w["n2"])
        for b, n in enumerate(w["n2"].tolist()):
            assert torch.equal(x["mass"][b, :, :n], w["mass"][b, :, :n]) and torch.equal(x["pos"][b, :, :n], w["pos"][b, :, :n])
            assert torch.equal(x["Kc"][b, :n], w["Kc"][b, :n]) and torch.equal(x["Vc"][b, :n], w["Vc"][b, :n])


def test_tensors_of_another_kind_are_refused():
    d, cap = Dims(B=2, T=4, D=64, G=4, M=2, k=1), 50
    v = cu(tree_inputs(d, cap, [10, 20], None, "tree", 1))
    O, lse, ws = torch.empty(8, 5, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(8, 5, device="cuda"), gqe.workspace(d, gqe.OP_TREE_ATTN)

    def call(**kw):
        a = dict(Q=v["Q"], Kn=v["Kn"], Vn=v["Vn"], Kc=v["Kc"], Vc=v["Vc"], lens=v["lens"], drafts=None, parent=v["parent"], O=O, lse=lse, ws=ws)
        a.update(kw)
        gqe.gqe_tree_attn(d, cap, *a.values())

    call()
    for kw in (dict(Q=v["Q"].float()), dict(Q=v["Q"].cpu()), dict(Q=v["Q"][:4]), dict(lens=v["lens"].long()), dict(Q=None),
               dict(Kc=v["Kc"].transpose(1, 2)), dict(parent=v["parent"].view(2, 4).t()), dict(O=torch.empty(8, 10, 64, dtype=torch.bfloat16, device="cuda")[:, ::2]),
               dict(lse=lse.half())):
        with pytest.raises(gqe.GqeError) as e:
            call(**kw)
        assert e.value.code == -1
    for short in (ws[:-256], None):
        with pytest.raises(gqe.GqeError) as e:
            call(ws=short)
        assert e.value.code == -3
    with pytest.raises(gqe.GqeError) as e:
        gqe.gqe_tree_attn(d, 0, *[v["Q"]] * 11)
    assert e.value.code == -1
    ok()
