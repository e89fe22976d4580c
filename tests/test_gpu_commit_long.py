"""GPU tests of gqe_tree_commit's sums where a block of threads works through
many blocks of keys and many units: long caches, runs of sequences that accept
nothing, caches past 32-bit offsets. Against the formula in 64 bits (torch).

Tolerance of a sum of R terms e^(score - lse), relative: 64 products added in
fp32 put the exponent off by 2^-17 times the size of its terms; exponent and
log-sum are rounded in fp32, 2^-20 (1 + |lse| + |score|); the exponential by
2^-18 at most (the polynomial's 2.7e-6); R additions by 2^-23 R.
"""
import pytest
import torch

from gqe_inputs import Dims
from oracle import serve_ref as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_gqa_query_gqe_b200 as gqe


def inputs(d, cap, lens, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    e = dict(device="cuda", generator=gen)
    N, Ha = d.B * d.T, d.G * d.k + 1

    def bf(*shape, std=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen)

    x = {"Q": bf(N, Ha, 64, std=1.3), "Kn": bf(N, d.G, 64), "Vn": bf(N, d.G, 64), "Kc": bf(d.B, cap, d.G, 64), "Vc": bf(d.B, cap, d.G, 64),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "mass": torch.rand(d.B, d.G, cap, **e)}
    x["lse"] = torch.randn(N, Ha, **e) + torch.log(x["lens"].float() + 2.0).repeat_interleave(d.T)[:, None] + 1.0
    for b, n in enumerate(lens):
        x["mass"][b, :, n:] = float("nan")  # a row that was never used
        x["Kc"][b, n:] = float("nan")
    return x


def run(d, cap, x, path, acc, mass_out):
    Kc, Vc = x["Kc"].clone(), x["Vc"].clone()
    new_len = torch.full((d.B,), -1, dtype=torch.int32, device="cuda")
    gqe.gqe_tree_commit(d, cap, path, acc, None, x["Q"], x["lse"], x["Kn"], x["Vn"], x["lens"], Kc, Vc, None,
                        x["mass"] if mass_out is not None else None, mass_out, new_len)
    return Kc, Vc, new_len


def check(d, x, lens, acc, order, mass, groups=None):
    for b, (L, n) in enumerate(zip(lens, acc)):
        if n == 0:
            assert torch.equal(mass[b, :, :L], x["mass"][b, :, :L]), f"sums of sequence {b}, which accepts nothing"
            assert (mass[b, :, L:] == 5.0).all()
            continue
        rows = torch.tensor([b * d.T + t for t in order[b][:n]], device="cuda")
        for g in range(d.G) if groups is None else groups:
            K = torch.cat([x["Kc"][b, :L, g], x["Kn"][rows, g]]).double()
            total, size = torch.zeros(L + n, dtype=torch.float64, device="cuda"), torch.zeros(L + n, dtype=torch.float64, device="cuda")
            worst = 0.0
            for h in ref.group_slots(g, d.G, d.k):
                q, lse = x["Q"][rows, h].double(), x["lse"][rows, h].double()
                w = torch.exp(K @ q.T / 8.0 - lse)
                w[L:].masked_fill_(torch.ones(n, n, dtype=torch.bool, device="cuda").tril(-1), 0.0)  # place j is seen from j on
                total += w.sum(1)
                size = torch.maximum(size, (K.abs() @ q.abs().T).amax(1) / 8.0)
                worst = max(worst, float(lse.abs().max()))
            total[:L] += x["mass"][b, g, :L].double()
            rel = 2.0 ** -17 * size + 2.0 ** -20 * (1 + worst + size) + 2.0 ** -18 + n * (d.k + 1) * 2.0 ** -23
            off = (mass[b, g, :L + n].double() - total).abs()
            assert bool((off <= rel * total).all()), f"sequence {b}, group {g}: worst {float((off / (rel * total)).max()):.2f} x the tolerance"
        assert (mass[b, :, L + n:] == 5.0).all(), "sums past the new length changed"


def commit_and_check(d, cap, lens, acc, seed, groups=None):
    x = inputs(d, cap, lens, seed)
    gen = torch.Generator().manual_seed(seed)
    order = [sorted(torch.randperm(d.T, generator=gen)[:n].tolist()) + [0] * (d.T - n) for n in acc]
    path, n_acc = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (order, acc))
    mass = torch.full_like(x["mass"], 5.0)
    Kc, Vc, new_len = run(d, cap, x, path, n_acc, mass)
    assert gqe.gqe_check_error() == 0
    assert new_len.tolist() == [a + n for a, n in zip(lens, acc)]
    check(d, x, lens, acc, order, mass, groups)
    for b, (L, n) in enumerate(zip(lens, acc)):
        rows = torch.tensor([b * d.T + t for t in order[b][:n]], dtype=torch.long, device="cuda")
        assert torch.equal(Kc[b, L:L + n], x["Kn"][rows]) and torch.equal(Vc[b, L:L + n], x["Vn"][rows])
        assert torch.equal(Kc[b, :L], x["Kc"][b, :L]) and torch.equal(Vc[b, :L], x["Vc"][b, :L])
    # in place: the same bits
    again = dict(x, mass=x["mass"].clone())
    run(d, cap, again, path, n_acc, again["mass"])
    assert gqe.gqe_check_error() == 0
    for b, (L, n) in enumerate(zip(lens, acc)):
        assert torch.equal(again["mass"][b, :, :L + n], mass[b, :, :L + n])


# Sequences that accept nothing, several in a row, between ones that do: the
# groups side by side (few rows) and one after the other; with two stages of K.
NOTHING = [
    (Dims(B=200, T=4, D=64, G=8, M=2, k=1), 300, [100 + b for b in range(200)], [3 if b % 23 == 22 else 0 for b in range(200)]),
    (Dims(B=12, T=16, D=64, G=4, M=2, k=1), 4000, [4000 - 16 - 300 * b for b in range(12)], [0] * 5 + [16] + [0] * 4 + [1, 0]),
    (Dims(B=6, T=128, D=64, G=8, M=4, k=2), 3000, [2800, 2500, 2000, 2872, 0, 1000], [0, 0, 128, 0, 0, 5]),
    (Dims(B=6, T=128, D=64, G=8, M=8, k=8), 3000, [2800, 2500, 2000, 2872, 2600, 1000], [0, 0, 128, 0, 0, 5]),
    (Dims(B=5, T=3, D=64, G=2, M=8, k=1), 9000, [8990, 8000, 0, 1, 5000], [0] * 5),
    (Dims(B=70, T=128, D=64, G=1, M=8, k=1), 900, [700 + b for b in range(70)], [0] * 69 + [128]),
]


@pytest.mark.parametrize("d,cap,lens,acc", NOTHING, ids=[f"b{c[0].B}t{c[0].T}g{c[0].G}k{c[0].k}" for c in NOTHING])
def test_sequences_that_accept_nothing(d, cap, lens, acc):
    commit_and_check(d, cap, lens, acc, 51)


LONG = [
    (Dims(B=4, T=6, D=64, G=8, M=2, k=1), 30010, [30000, 20011, 0, 25088], [6, 1, 6, 3]),
    (Dims(B=1, T=1, D=64, G=8, M=2, k=1), 65537, [65536], [1]),
    (Dims(B=2, T=20, D=64, G=1, M=8, k=4), 40100, [40001, 128], [20, 11]),
    (Dims(B=2, T=3, D=64, G=64, M=1, k=1), 6000, [5990, 4097], [3, 2]),
    (Dims(B=2, T=128, D=64, G=8, M=4, k=2), 20200, [20000, 9001], [128, 77]),
    (Dims(B=2, T=100, D=64, G=8, M=8, k=8), 8100, [8000, 2047], [100, 3]),
]


@pytest.mark.parametrize("d,cap,lens,acc", LONG, ids=[f"b{c[0].B}t{c[0].T}g{c[0].G}k{c[0].k}_{max(c[2])}" for c in LONG])
def test_sums_over_long_caches(d, cap, lens, acc):
    commit_and_check(d, cap, lens, acc, 52)


def test_sums_past_32_bit_offsets():
    """K of more than 2^31 elements: the second sequence's rows lie beyond."""
    d, cap = Dims(B=2, T=2, D=64, G=64, M=1, k=1), 270_000
    assert d.B * cap * d.G * 64 > 2 ** 31
    commit_and_check(d, cap, [1000, cap - 2], [0, 2], 53, groups=[0, 1, 37, 63])
