"""The serving operators around a GQE layer's key/value cache: real cases of each, their plain form, and the framework's calls.

One step of a server that drafts tokens runs, for every layer, the router and the projections on the drafted tokens, then
  rope    norms of each head's queries and keys, with the position rotation in the same pass;
  tree    attention of a tree of drafted tokens over the cache and over their own ancestors;
  commit  the accepted path appended to the cache, its attention weight added to every cached position's sum;
  evict   the positions with the least accumulated weight dropped, the cache closed up again in place.
Sizes are a layer's: G key/value groups, M experts in each, k of them selected per token, one shared head on group 0, heads of 64.
"""
import math
import random

import torch

own = False

DH = 64
HEADS = [(8, 2, 1), (8, 4, 2), (4, 2, 1), (2, 8, 4), (1, 8, 2), (8, 8, 4), (4, 4, 1), (16, 4, 1), (32, 2, 2), (64, 1, 1)]


def listed():
    g = dict(G=8, M=2, k=1)
    return [
        # one new token of one conversation: the call's latency
        dict(name="rope one token", op="rope", B=1, T=1, **g, layout="half", rot=64, norm=True, far=70000),
        # the main layer's prompt batch, 8 sequences of 2048 tokens
        dict(name="rope prompts 8x2048", op="rope", B=8, T=2048, **g, layout="half", rot=64, norm=True, far=0),
        # a long document in the pool of four experts, the first 32 dimensions rotated as neighbouring pairs
        dict(name="rope long 1x131072", op="rope", B=1, T=131072, G=8, M=4, k=2, layout="interleaved", rot=32, norm=True, far=0),
        # plain decoding of one conversation: a "tree" of one token
        dict(name="tree 1x1 over 4095", op="tree", B=1, T=1, **g, len=4095, len_min=4095, chain=True, ragged=False),
        # eight conversations of ragged length, 16 drafted tokens each, the caches at up to 32K
        dict(name="tree 8x16 over 32K", op="tree", B=8, T=16, **g, len=32767, len_min=20001, chain=False, ragged=True),
        # odd sizes in the pool of four experts: 13 drafts, short caches
        dict(name="tree 5x13 over 1500", op="tree", B=5, T=13, G=8, M=4, k=2, len=1500, len_min=0, chain=False, ragged=True),
        # a prompt's last 128 tokens as one chunk against the long cache of each of four sequences
        dict(name="tree 4x128 over 131K", op="tree", B=4, T=128, G=8, M=4, k=2, len=131072, len_min=131072, chain=True, ragged=False),
        # one accepted token of one conversation
        dict(name="commit 1 over 4095", op="commit", B=1, T=1, **g, len=4095, len_min=4095, acc=1),
        # up to 6 accepted of 16 drafted, weights accumulated over caches of up to 32K
        dict(name="commit 8x6 over 32K", op="commit", B=8, T=16, **g, len=32767, len_min=20001, acc=6),
        # a chunk of 128 prompt tokens in the pool of four experts (the window of queries that votes for the prompt's keys)
        dict(name="commit 2x128 over 64K", op="commit", B=2, T=128, G=8, M=4, k=2, len=65536, len_min=60000, acc=128),
        # the steady state: a few positions over the budget leave
        dict(name="evict 8x4100 to 4096", op="evict", B=8, **g, len=4100, len_min=4090, keep=4096, sink=4, recent=256),
        # a prompt's cache cut to an eighth
        dict(name="evict 8x32K to 4096", op="evict", B=8, **g, len=32768, len_min=30000, keep=4096, sink=4, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    G, M, k = rng.choice(HEADS)
    op = rng.choice(["rope", "tree", "tree", "commit", "evict"])
    c = dict(op=op, G=G, M=M, k=k)
    if op == "rope":
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, 2_000_000 // (B * (G * (k + 1) + 1))))
        layout = rng.choice(["half", "interleaved"])
        c.update(B=B, T=T, layout=layout, rot=rng.choice([64, 64, 32, 2 * rng.randint(1, 32)]), norm=rng.random() < 0.8,
                 far=rng.choice([0, _log(rng, 1, 1_000_000)]))
        return c
    B = _log(rng, 1, 32)
    if op == "evict":
        n = _log(rng, 16, max(17, min(131072, 2_000_000 // (B * G))))
        keep = max(3, n - _log(rng, 1, n - 3)) if rng.random() < 0.5 else max(3, n // rng.randint(2, 9))
        sink = rng.randint(0, min(8, keep // 3))
        c.update(B=B, len=n, len_min=rng.randint(0, n), keep=keep, sink=sink, recent=rng.randint(0, keep // 2))
        return c
    T = _log(rng, 1, 128)
    rows = B * T * (G * k + 1)
    n = _log(rng, 1, max(2, min(131072, 4_000_000 // (B * G), 500_000_000 // rows)))
    c.update(B=B, T=T, len=n, len_min=rng.randint(0, n))
    if op == "tree":
        c.update(chain=rng.random() < 0.3, ragged=rng.random() < 0.7)
    else:
        c.update(acc=rng.randint(1, T))
    return c


# ---- what follows from a case alone -----------------------------------------------------------------------------------
def _lens(c):
    """The sequences' cache lengths: evenly from len down to len_min."""
    n = max(1, c["B"] - 1)
    return [c["len"] - (c["len"] - c["len_min"]) * b // n for b in range(c["B"])]


def _drafts(c):
    """Drafted tokens of each sequence: all T, or ragged from T down to 0."""
    T = c["T"]
    return [T - (T * b) // max(1, c["B"]) if c["ragged"] else T for b in range(c["B"])]


def _accs(c):
    """Accepted tokens of each sequence: acc for the first, fewer for some of the others, none for every seventh."""
    return [0 if b % 7 == 6 else c["acc"] - (c["acc"] // 2 if b % 3 == 2 else 0) for b in range(c["B"])]


def _cap(c):
    return c["len"] + c.get("T", 0) + 7


def work(c):
    B, G, k = c["B"], c["G"], c["k"]
    Ha = G * k + 1
    if c["op"] == "rope":
        rows = B * c["T"]
        return {"bytes": rows * ((Ha + G) * 256 + 4 + (4 * G * k if c["norm"] else 0)), "flops": rows * (Ha + G) * 64 * (6 if c["norm"] else 3)}
    L = _lens(c)
    if c["op"] == "tree":
        n = _drafts(c)
        keys = sum((x + y) * G for x, y in zip(L, n) if y)
        pairs = sum(y * Ha * x + Ha * y * ((y + 1) / 2 if c["chain"] else math.log2(y + 1)) for x, y in zip(L, n))
        return {"bytes": keys * 256 + sum(n) * Ha * (256 + 4) + sum(n) * 4, "flops": 256 * pairs}
    if c["op"] == "commit":
        n = _accs(c)
        keys = sum((x + y) * G for x, y in zip(L, n) if y)
        pairs = sum(y * Ha * (x + (y + 1) / 2) for x, y in zip(L, n))
        return {"bytes": keys * (128 + 8) + sum(n) * (Ha * 132 + G * 516), "flops": 128 * pairs}
    keep = c["keep"]
    moved = sum((min(keep, x) * (1 - keep / x) if x > keep else 0) * G for x in L)
    return {"bytes": sum(L) * G * 8 + sum(min(x, keep) for x in L) * G * 8 + moved * 512, "flops": sum(L) * G}


# ---- inputs -----------------------------------------------------------------------------------------------------------
def _tree(c, seed):
    """Parents of the drafted tokens: a chain, or a tree whose nodes mostly continue one of the last few."""
    T = c["T"]
    r = random.Random(seed * 1000003 + T)
    if c["chain"]:
        return [[i - 1 for i in range(T)] for _ in range(c["B"])]
    return [[-1 if i == 0 or r.random() < 0.1 else r.randint(max(0, i - 5), i - 1) for i in range(T)] for _ in range(c["B"])]


def prepare(c, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    bf = torch.bfloat16

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(bf)

    B, G, M, k = c["B"], c["G"], c["M"], c["k"]
    Ha = G * k + 1
    # the layer's dimensions as the calls take them; the eviction has no new tokens, its T is the cache's capacity
    s = {"c": c, "dims": dict(B=B, T=_cap(c) if c["op"] == "evict" else c["T"], D=64, G=G, M=M, k=k, dh=DH)}
    if c["op"] == "rope":
        N = B * c["T"]
        s["Q"], s["K"] = normal(N, Ha, DH, std=0.64), normal(N, G, DH, std=0.64)
        s["wq"] = s["wk"] = None
        if c["norm"]:
            s["wq"], s["wk"] = 1 + normal(G * M + 1, DH, std=0.1), 1 + normal(G, DH, std=0.1)
        s["sel"] = torch.rand(N, G, M, generator=gen, device=dev).topk(k, dim=2).indices.sort(dim=2).values.int()
        half = max(1, c["rot"] // 2)
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(dev)
        s["scale"] = 1.0 if c["far"] == 0 else 0.1 * math.log(4.0) + 1.0
        start = torch.randint(0, c["far"] + 1, (B, 1), generator=gen, device=dev)
        s["positions"] = (start + torch.arange(c["T"], device=dev)).reshape(-1).int()
        s["Qo"], s["Ko"] = torch.zeros_like(s["Q"]), torch.zeros_like(s["K"])
        return s
    cap = _cap(c)
    s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device=dev)
    # rows at and past a sequence's length hold what an earlier user of the buffer left there
    s["Kc"], s["Vc"] = normal(B, cap, G, DH), normal(B, cap, G, DH)
    if c["op"] == "evict":
        # accumulated weights are heavy-tailed; in some places they are equal, and where they underflowed, zero
        m = torch.exp(2.0 * torch.randn(B, G, cap, generator=gen, device=dev) - 4.0)
        u = torch.rand(B, G, cap, generator=gen, device=dev)
        m = torch.where(u < 0.05, torch.zeros_like(m), torch.where(u < 0.3, (m * 256).round() / 256, m))
        s["mass"] = m
        # some positions were evicted before: those that are left, in an order of their own
        s["pos"] = (torch.rand(B, G, 2 * cap, generator=gen, device=dev).argsort(dim=2)[:, :, :cap]).int()
        s["next_pos"] = torch.full((B,), 2 * cap, dtype=torch.int32, device=dev)
        s["mass_out"], s["pos_out"] = torch.zeros_like(m), torch.zeros_like(s["pos"])
        s["new_len"] = torch.zeros_like(s["lens"])
        return s
    T = c["T"]
    s["Q"], s["Kn"], s["Vn"] = normal(B * T, Ha, DH, std=1.2), normal(B * T, G, DH), normal(B * T, G, DH)
    if c["op"] == "tree":
        s["parent"] = torch.tensor(_tree(c, seed), dtype=torch.int32, device=dev).reshape(-1)
        s["drafts"] = torch.tensor(_drafts(c), dtype=torch.int32, device=dev)
        s["O"] = torch.zeros(B * T, Ha, DH, dtype=bf, device=dev)
        s["lse"] = torch.zeros(B * T, Ha, device=dev)
        return s
    acc = _accs(c)
    r = random.Random(seed)
    path = [sorted(r.sample(range(T), n)) + [0] * (T - n) for n in acc]
    s["path"] = torch.tensor(path, dtype=torch.int32, device=dev)
    s["n_acc"] = torch.tensor(acc, dtype=torch.int32, device=dev)
    s["positions"] = (s["lens"][:, None] + 1000 + torch.arange(T, device=dev)[None, :]).int().reshape(-1)
    s["mass"] = torch.exp(torch.randn(B, G, cap, generator=gen, device=dev) - 2.0)
    s["mass_out"] = torch.zeros_like(s["mass"])
    s["pos"] = torch.arange(cap, device=dev, dtype=torch.int32).expand(B, G, cap).contiguous()
    s["new_len"] = torch.zeros_like(s["lens"])
    # the attention's log-sums for scores q.k / 8 of N(0, 1.2^2) over the cache, as far as this needs them
    near = torch.randn(B * T, Ha, generator=gen, device=dev) * 0.02
    s["lse"] = near + 0.72 + torch.log(s["lens"].float().clamp_min(0) + 2.0).repeat_interleave(T)[:, None]
    return s


# ---- plain forms ------------------------------------------------------------------------------------------------------
def _norm(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w


def _rotate(x, cos, sin, c):
    rot = c["rot"]
    a, rest = x[..., :rot], x[..., rot:]
    if c["layout"] == "half":
        lo, hi = a[..., :rot // 2], a[..., rot // 2:]
        a = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)
    else:
        lo, hi = a[..., 0::2], a[..., 1::2]
        a = torch.stack([lo * cos - hi * sin, hi * cos + lo * sin], -1).flatten(-2)
    return torch.cat([a, rest], -1)


def _rope(s):
    c = s["c"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = (torch.cos(angle) * s["scale"]).float()[:, None], (torch.sin(angle) * s["scale"]).float()[:, None]
    wq = wk = None
    if s["wq"] is not None:
        base = torch.arange(c["G"], device="cuda")[None, :, None] * c["M"]
        heads = (base + s["sel"]).flatten(1)
        heads = torch.cat([heads, torch.full_like(heads[:, :1], c["G"] * c["M"])], 1)
        wq, wk = s["wq"].float()[heads], s["wk"].float()
    return {"Q": _rotate(_norm(s["Q"], wq), cos, sin, c).to(torch.bfloat16), "K": _rotate(_norm(s["K"], wk), cos, sin, c).to(torch.bfloat16)}


def _grouped(x, c):
    """[B, T, G*k + 1, e] as [B, G, T, k + 1, e]: each group's selected rows, and in group 0 the shared row (zeros elsewhere)."""
    B, T, G, k = c["B"], c["T"], c["G"], c["k"]
    x = x.view(B, T, G * k + 1, -1)
    shared = torch.zeros(B, T, G, 1, x.shape[-1], dtype=x.dtype, device=x.device)
    shared[:, :, 0, 0] = x[:, :, G * k]
    return torch.cat([x[:, :, :G * k].reshape(B, T, G, k, -1), shared], 3).transpose(1, 2)


def _ungrouped(x, c):
    B, T, G, k = c["B"], c["T"], c["G"], c["k"]
    x = x.transpose(1, 2)
    return torch.cat([x[:, :, :, :k].reshape(B, T, G * k, -1), x[:, :, 0, k:]], 2).reshape(B * T, G * k + 1, -1)


def _tree_attn(s):
    c = s["c"]
    B, T, G, k = c["B"], c["T"], c["G"], c["k"]
    top = c["len"]
    q = _grouped(s["Q"].float(), c).reshape(B, G, T * (k + 1), DH)
    keys = torch.cat([s["Kc"][:, :top], s["Kn"].view(B, T, G, DH)], 1).float().transpose(1, 2)
    values = torch.cat([s["Vc"][:, :top], s["Vn"].view(B, T, G, DH)], 1).float().transpose(1, 2)
    step = torch.zeros(B, T, T + 1, dtype=torch.float64, device="cuda").scatter_(2, s["parent"].view(B, T, 1).long() + 1, 1.0)[:, :, 1:]
    sees = torch.linalg.matrix_power(step + torch.eye(T, dtype=torch.float64, device="cuda"), T) > 0
    cached = (torch.arange(top, device="cuda")[None, :] < s["lens"][:, None])[:, None, :].expand(B, T, top)
    mask = torch.cat([cached, sees], 2)[:, None].repeat_interleave(k + 1, 2)
    score = (q @ keys.transpose(2, 3) / 8.0).masked_fill(~mask, -math.inf)
    high = score.amax(-1, keepdim=True)
    p = torch.exp(score - high)
    total = p.sum(-1, keepdim=True)
    o = _ungrouped((p @ values / total).view(B, G, T, k + 1, DH), c)
    lse = _ungrouped((high + torch.log(total)).view(B, G, T, k + 1, 1), c)[..., 0]
    live = (torch.arange(T, device="cuda")[None, :] < s["drafts"][:, None]).reshape(-1, 1)
    s["O"].copy_(torch.where(live[:, :, None], o.to(torch.bfloat16), s["O"]))
    s["lse"].copy_(torch.where(live, lse, s["lse"]))
    return {"O": s["O"], "lse": s["lse"]}


def _commit(s):
    c = s["c"]
    B, T, G, k = c["B"], c["T"], c["G"], c["k"]
    top = c["len"] + c["T"]
    j = torch.arange(T, device="cuda")
    taken = j[None, :] < s["n_acc"][:, None]
    at = (torch.arange(B, device="cuda")[:, None] * T + s["path"]).reshape(-1).long()
    b, to = torch.arange(B, device="cuda")[:, None], s["lens"].long()[:, None] + j[None, :]
    keep = taken[:, :, None, None]
    s["Kc"][b, to] = torch.where(keep, s["Kn"][at].view(B, T, G, DH), s["Kc"][b, to])
    s["Vc"][b, to] = torch.where(keep, s["Vn"][at].view(B, T, G, DH), s["Vc"][b, to])
    s["pos"].scatter_(2, to[:, None].expand(-1, G, -1), torch.where(taken, s["positions"][at].view(B, T), to.int())[:, None].expand(-1, G, -1))
    s["new_len"].copy_(s["lens"] + s["n_acc"])
    q = _grouped(s["Q"][at].float(), c)
    lse = _grouped(s["lse"][at][..., None], c)
    keys = s["Kc"][:, :top].float().transpose(1, 2)
    slot = torch.arange(top, device="cuda")
    sees = (slot[None, None, :] <= s["lens"][:, None, None] + j[None, :, None]) & taken[:, :, None]
    score = (q.reshape(B, G, T * (k + 1), DH) @ keys.transpose(2, 3)) / 8.0
    p = torch.exp(score - lse.reshape(B, G, T * (k + 1), 1)).view(B, G, T, k + 1, top)
    p = p.masked_fill(~sees[:, None, :, None, :], 0.0)
    got = p[:, :, :, :k].sum((2, 3))
    got[:, 0] += p[:, 0, :, k].sum(1)
    got += s["mass"][:, :, :top].masked_fill((slot[None, :] >= s["lens"][:, None])[:, None], 0.0)
    live = (slot[None, :] < s["new_len"][:, None])[:, None]
    s["mass_out"][:, :, :top] = torch.where(live, got, s["mass_out"][:, :, :top])
    return {"K": s["Kc"], "V": s["Vc"], "pos": s["pos"], "mass": s["mass_out"], "len": s["new_len"]}


def _evict(s):
    c = s["c"]
    cap, keep = _cap(c), c["keep"]
    slot = torch.arange(cap, device="cuda")
    n = s["lens"][:, None, None]
    fixed = (s["pos"] < c["sink"]) | (s["pos"] >= s["next_pos"][:, None, None] - c["recent"])
    key = s["mass"].masked_fill(fixed, math.inf).masked_fill(slot >= n, -1.0)
    order = key.sort(dim=2, descending=True, stable=True).indices
    stays = torch.zeros_like(fixed).scatter_(2, order[:, :, :keep], True) & (slot < n)
    hole = ~stays & (slot < torch.minimum(n, torch.full_like(n, keep)))
    rank = (hole.cumsum(2) - 1).clamp_min(0)
    late = (stays & (slot >= keep)).int().sort(dim=2, descending=True, stable=True).indices
    src = torch.where(hole, late.gather(2, rank), slot)[:, :, :keep]
    s["new_len"].copy_(s["lens"].clamp_max(keep))
    live = slot[:keep] < s["new_len"][:, None, None]
    at = src.transpose(1, 2)[..., None].expand(-1, -1, -1, DH)
    s["Kc"][:, :keep] = s["Kc"].gather(1, at)
    s["Vc"][:, :keep] = s["Vc"].gather(1, at)
    s["mass_out"][:, :, :keep] = torch.where(live, s["mass"].gather(2, src), s["mass_out"][:, :, :keep])
    s["pos_out"][:, :, :keep] = torch.where(live, s["pos"].gather(2, src), s["pos_out"][:, :, :keep])
    return {"K": s["Kc"], "V": s["Vc"], "mass": s["mass_out"], "pos": s["pos_out"], "len": s["new_len"]}


def _ws(s, gqe, op):
    """The state's workspace, made before its first pass and kept."""
    if "ws" not in s:
        s["ws"] = gqe.workspace(s["dims"], op)
    return s["ws"]


def run(s):
    op = s["c"]["op"]
    if not own:
        return {"rope": _rope, "tree": _tree_attn, "commit": _commit, "evict": _evict}[op](s)
    import moe_gqa_query_gqe_b200 as gqe
    c = s["c"]
    if op == "rope":
        layout = gqe.ROPE_HALF if c["layout"] == "half" else gqe.ROPE_INTERLEAVED
        gqe.gqe_qk_rope(s["dims"], s["Q"], s["K"], s["wq"], s["wk"], s["sel"], s["inv_freq"], s["positions"], s["Qo"], s["Ko"],
                        layout=layout, rot=c["rot"], eps=1e-6, scale=s["scale"])
        return {"Q": s["Qo"], "K": s["Ko"]}
    if op == "tree":
        gqe.gqe_tree_attn(s["dims"], _cap(c), s["Q"], s["Kn"], s["Vn"], s["Kc"], s["Vc"], s["lens"], s["drafts"], s["parent"],
                          s["O"], s["lse"], _ws(s, gqe, gqe.OP_TREE_ATTN))
        return {"O": s["O"], "lse": s["lse"]}
    if op == "commit":
        gqe.gqe_tree_commit(s["dims"], _cap(c), s["path"], s["n_acc"], s["positions"], s["Q"], s["lse"], s["Kn"], s["Vn"],
                            s["lens"], s["Kc"], s["Vc"], s["pos"], s["mass"], s["mass_out"], s["new_len"])
        return {"K": s["Kc"], "V": s["Vc"], "pos": s["pos"], "mass": s["mass_out"], "len": s["new_len"]}
    gqe.gqe_cache_evict(s["dims"], c["keep"], c["sink"], c["recent"], s["lens"], s["next_pos"], s["Kc"], s["Vc"], s["mass"],
                        s["mass_out"], s["pos"], s["pos_out"], s["new_len"], _ws(s, gqe, gqe.OP_CACHE_EVICT))
    return {"K": s["Kc"], "V": s["Vc"], "mass": s["mass_out"], "pos": s["pos_out"], "len": s["new_len"]}


# ---- the definition, in 64 bits ---------------------------------------------------------------------------------------
def _exact_rope(s, c):
    angle = torch.outer(s["positions"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.full_like(angle, s["scale"]), angle)

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / DH + 1e-6) * w
        r = c["rot"]
        pair = x[..., :r].unflatten(-1, (2, r // 2)).movedim(-2, -1) if c["layout"] == "half" else x[..., :r].unflatten(-1, (r // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
        x[..., :r] = z.movedim(-1, -2).flatten(-2) if c["layout"] == "half" else z.flatten(-2)
        return x

    wq = wk = None
    if s["wq"] is not None:
        wq = torch.empty(s["Q"].shape, dtype=torch.float64, device="cuda")
        for h in range(c["G"] * c["k"]):
            wq[:, h] = s["wq"].double()[h // c["k"] * c["M"] + s["sel"].flatten(1)[:, h].long()]
        wq[:, -1] = s["wq"].double()[-1]
        wk = s["wk"].double()
    return {"Q": one(s["Q"], wq), "K": one(s["K"], wk)}


def _rows(c, g):
    """Query slots of group g."""
    return [g * c["k"] + j for j in range(c["k"])] + ([c["G"] * c["k"]] if g == 0 else [])


def _exact_tree(s, c):
    T, O, lse = c["T"], s["O"].double(), s["lse"].double()
    lens, drafts, parent = _lens(c), _drafts(c), s["parent"].view(c["B"], T).tolist()
    for b in range(c["B"]):
        n = drafts[b]
        if n == 0:
            continue
        sees = torch.zeros(n, n, dtype=torch.bool)
        for i in range(n):
            if parent[b][i] >= 0:
                sees[i] = sees[parent[b][i]]
            sees[i, i] = True
        own_rows = slice(b * T, b * T + n)
        for g in range(c["G"]):
            kk = torch.cat([s["Kc"][b, :lens[b], g], s["Kn"][own_rows, g]]).double()
            vv = torch.cat([s["Vc"][b, :lens[b], g], s["Vn"][own_rows, g]]).double()
            for h in _rows(c, g):
                a = s["Q"][own_rows, h].double() @ kk.T * 0.125
                a[:, lens[b]:][~sees.cuda()] = -math.inf
                lse[own_rows, h] = torch.logsumexp(a, 1)
                O[own_rows, h] = torch.softmax(a, 1) @ vv
    return {"O": O, "lse": lse}


def _exact_commit(s, c):
    T, K, V, mass = c["T"], s["Kc"].double(), s["Vc"].double(), s["mass_out"].double()
    lens, acc, path = _lens(c), _accs(c), s["path"].tolist()
    for b in range(c["B"]):
        n, L = acc[b], lens[b]
        rows = torch.tensor([b * T + i for i in path[b][:n]], dtype=torch.long, device="cuda")
        K[b, L:L + n], V[b, L:L + n] = s["Kn"][rows].double(), s["Vn"][rows].double()
        mass[b, :, :L] = s["mass"][b, :, :L].double()
        blocked = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        for g in range(c["G"] if n else 0):
            for h in _rows(c, g):
                p = torch.exp(s["Q"][rows, h].double() @ K[b, :L + n, g].T * 0.125 - s["lse"][rows, h].double()[:, None])
                p[:, L:][blocked] = 0.0
                mass[b, g, :L + n] += p.sum(0)
    return {"K": K, "V": V, "pos": None, "mass": mass, "len": None}


def _exact_evict(s, c):
    K, V, mass = s["Kc"].double(), s["Vc"].double(), s["mass_out"].double()
    lens, keep = _lens(c), c["keep"]
    m_all, p_all, nxt = s["mass"].double().cpu().numpy(), s["pos"].cpu().numpy(), s["next_pos"].cpu().numpy()
    import numpy as np
    for b in range(c["B"]):
        n = lens[b]
        for g in range(c["G"]):
            m, p = m_all[b, g, :n], p_all[b, g, :n]
            if n <= keep:
                mass[b, g, :n] = torch.from_numpy(m).cuda()
                continue
            fixed = (p < c["sink"]) | (p >= nxt[b] - c["recent"])
            best = np.lexsort((np.arange(n), -m, ~fixed))[:keep]
            holes = np.setdiff1d(np.arange(keep), best)
            late = np.sort(best[best >= keep])
            src = np.arange(keep)
            src[holes] = late
            mass[b, g, :keep] = torch.from_numpy(m[src]).cuda()
            at, fr = torch.from_numpy(holes).cuda(), torch.from_numpy(late).cuda()
            K[b, at, g], V[b, at, g] = K[b, fr, g], V[b, fr, g]
    return {"K": K, "V": V, "mass": mass, "pos": None, "len": None}


def exact(c, seed):
    if c["op"] == "tree" and c["B"] * c["T"] * (c["G"] * c["k"] + 1) * c["len"] > 2_000_000_000:
        return None
    s = prepare(c, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "commit": _exact_commit, "evict": _exact_evict}[c["op"]](s, c)
