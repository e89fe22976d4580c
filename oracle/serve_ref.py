"""fp64 CPU oracle of the operators around the key/value cache: norms with
rotation, attention of a tree of drafted tokens, commit, eviction.

TEST INFRASTRUCTURE: plain, slow restatements in float64, with nothing of the
CUDA library. Inputs are the bf16/fp32 values (exact in float64). Beside each
result stands what a tolerance needs: the size of the terms that were added.
"""
from __future__ import annotations

import numpy as np

from oracle.gqe_ref import _f64


def qk_rope(x, weights, inv_freq, positions, layout, rot, eps, scale):
    """x [N, H, 64]; weights [N, H, 64] or None; inv_freq [rot/2]; positions
    [N] ints; layout "half" or "interleaved". Returns (y, size): size [N, H, 1]
    bounds the magnitude of every term added in a rotation."""
    y = _f64(x).copy()
    if weights is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * _f64(weights)
    size = np.abs(y).max(-1, keepdims=True) * max(1.0, abs(scale)) * 2.0
    angle = np.asarray(positions, dtype=np.float64)[:, None] * _f64(inv_freq)[None, :]
    out = y.copy()
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = scale * np.cos(angle[:, i])[:, None], scale * np.sin(angle[:, i])[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out, size


def query_weights(wq, sel, G, M):
    """[N, G*k + 1, 64]: the weight row of each query slot, that of its expert,
    and for the last slot the shared head's."""
    wq, sel = _f64(wq), np.asarray(sel)
    N = sel.shape[0]
    rows = [wq[g * M + sel[:, g, j]] for g in range(G) for j in range(sel.shape[2])]
    return np.stack(rows + [np.broadcast_to(wq[G * M], (N, 64))], axis=1)


def ancestors(parent, n):
    """[n, n] truth values: token i sees token j (itself and its ancestors)."""
    sees = np.zeros((n, n), dtype=bool)
    for i in range(n):
        p = i - 1 if parent is None else int(parent[i])
        if p >= 0:
            sees[i] = sees[p]
        sees[i, i] = True
    return sees


def group_slots(g, G, k):
    return [g * k + j for j in range(k)] + ([G * k] if g == 0 else [])


def tree_attn(Q, K_new, V_new, K_cache, V_cache, cache_len, draft_len, parent, B, T, G, k):
    """Q [B*T, G*k+1, 64], K_new, V_new [B*T, G, 64], caches [B, cap, G, 64].
    Returns a dict of O, lse, and for tolerances `terms` = sum_s p_s |v_s| and
    `score` = max_s sum_d |q_d k_sd| / 8 of every row; rows at and past
    draft_len[b] are NaN."""
    Ha = G * k + 1
    Q, Kn, Vn, Kc, Vc = _f64(Q), _f64(K_new), _f64(V_new), _f64(K_cache), _f64(V_cache)
    O, terms = np.full((B * T, Ha, 64), np.nan), np.full((B * T, Ha, 64), np.nan)
    lse, score = np.full((B * T, Ha), np.nan), np.full((B * T, Ha), np.nan)
    for b in range(B):
        L, n = int(cache_len[b]), T if draft_len is None else int(draft_len[b])
        par = None if parent is None else np.asarray(parent).reshape(B, T)[b]
        sees = ancestors(par, n)
        for i in range(n):
            row = b * T + i
            kin = b * T + np.flatnonzero(sees[i])
            for g in range(G):
                kk = np.concatenate([Kc[b, :L, g], Kn[kin, g]])
                vv = np.concatenate([Vc[b, :L, g], Vn[kin, g]])
                for h in group_slots(g, G, k):
                    a = kk @ Q[row, h] / 8.0
                    m = a.max()
                    p = np.exp(a - m)
                    l = p.sum()
                    O[row, h] = p @ vv / l
                    terms[row, h] = p @ np.abs(vv) / l
                    lse[row, h] = m + np.log(l)
                    score[row, h] = (np.abs(kk) @ np.abs(Q[row, h])).max() / 8.0
    return {"O": O, "lse": lse, "terms": terms, "score": score}


def tree_commit(path, n_acc, positions, Q, lse, K_new, V_new, cache_len, K_cache, V_cache, pos, mass, B, T, G, k):
    """The caches, positions, sums and lengths after the commit (copies).
    mass None: not accumulated. `score` as in tree_attn, the largest of all."""
    Kn, Vn, K, V = _f64(K_new), _f64(V_new), _f64(K_cache).copy(), _f64(V_cache).copy()
    pos = None if pos is None else np.array(pos, copy=True)
    out = None if mass is None else _f64(mass).copy()
    new_len, score = [], 0.0
    for b in range(B):
        L, n = int(cache_len[b]), T if n_acc is None else int(n_acc[b])
        toks = [j if path is None else int(np.asarray(path).reshape(B, T)[b, j]) for j in range(n)]
        for j, i in enumerate(toks):
            K[b, L + j], V[b, L + j] = Kn[b * T + i], Vn[b * T + i]
            if pos is not None:
                pos[b, :, L + j] = L + j if positions is None else int(np.asarray(positions).reshape(B, T)[b, i])
        new_len.append(L + n)
        if out is None:
            continue
        out[b, :, L:L + n] = 0.0
        q, ls = _f64(Q), _f64(lse)
        for j, i in enumerate(toks):
            for g in range(G):
                for h in group_slots(g, G, k):
                    kk = K[b, :L + j + 1, g]
                    out[b, g, :L + j + 1] += np.exp(kk @ q[b * T + i, h] / 8.0 - ls[b * T + i, h])
                    score = max(score, (np.abs(kk) @ np.abs(q[b * T + i, h])).max() / 8.0)
    return {"K": K, "V": V, "pos": pos, "mass": out, "len": np.array(new_len), "score": score}


def cache_evict(keep, sink, recent, cache_len, next_pos, mass, pos, B, G):
    """src[b][g]: for each row of the cache after the eviction, the row it came
    from. Rows that stay are chosen one by one: the lowest row among the best."""
    src = []
    for b in range(B):
        n = int(cache_len[b])
        per = []
        for g in range(G):
            if n <= keep:
                per.append(list(range(n)))
                continue
            m, p = np.asarray(mass[b][g][:n], dtype=np.float64), np.asarray(pos[b][g][:n])
            fixed = (p < sink) | (p >= int(next_pos[b]) - recent)
            # protected rows first, then by mass, those without a number last; the lower row of equal ones
            order = [(0, 0.0, s) if fixed[s] else ((2, 0.0, s) if np.isnan(m[s]) else (1, -m[s], s)) for s in range(n)]
            rank = [o[2] for o in sorted(order)]
            stays = set(rank[:keep])
            holes = [s for s in range(keep) if s not in stays]
            late = sorted(s for s in stays if s >= keep)
            rows = list(range(keep))
            for to, fr in zip(holes, late, strict=True):
                rows[to] = fr
            per.append(rows)
        src.append(per)
    return src
