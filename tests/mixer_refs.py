"""Plain 64-bit forms of the token mixers and the token log probabilities
(numpy, from their formulas), for the tests."""
import numpy as np

HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step of the type, relative to the value


def attention(q, k_pool, v_pool, table, lens, scale, cap=None):
    """out [B][Hq][d], lse [B][Hq], and per output the bound's parts: the
    absolute weighted values and the largest sum |q||k| of a head."""
    B, Hq, d = q.shape
    n_pages, Hkv, page, _ = k_pool.shape
    out, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf)
    mass, reach = np.zeros((B, Hq, d)), np.zeros((B, Hq))
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * page, cap if cap else 1 << 62))
        j = np.arange(n)
        pg = table[b, j // page]
        ok = (pg >= 0) & (pg < n_pages)
        j, pg = j[ok], pg[ok]
        if not len(j):
            continue
        for h in range(Hq):
            kh = h // (Hq // Hkv)
            k, v = k_pool[pg, kh, j % page].astype(np.float64), v_pool[pg, kh, j % page].astype(np.float64)
            x = (k @ q[b, h].astype(np.float64)) * scale
            m = x.max()
            p = np.exp(x - m)
            out[b, h], lse[b, h] = (p @ v) / p.sum(), m + np.log(p.sum())
            mass[b, h] = (p @ np.abs(v)) / p.sum()
            reach[b, h] = (np.abs(k) @ np.abs(q[b, h].astype(np.float64))).max() * abs(scale)
    return out, lse, mass, reach


def delta_rule(q, k, v, g, beta, state, at, scale, eps):
    """out (NaN in rows of no sequence) and the new state."""
    T, Hv, dv = v.shape
    rep = Hv // q.shape[1]
    q, k = (x.astype(np.float64) for x in (q, k))
    if eps is not None:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + eps) for x in (q, k))
    q, k = np.repeat(q, rep, 1), np.repeat(k, rep, 1)
    out, S = np.full((T, Hv, dv), np.nan), state.astype(np.float64).copy()
    for s in range(len(at) - 1):
        t0 = min(max(int(at[s]), 0), T)
        for t in range(t0, max(t0, min(int(at[s + 1]), T))):
            x = S[s] * np.exp(g[t].astype(np.float64))[:, None, None]
            u = beta[t].astype(np.float64)[:, None] * (v[t].astype(np.float64) - np.einsum("hij,hi->hj", x, k[t]))
            S[s] = x + k[t][:, :, None] * u[:, None]
            out[t] = scale * np.einsum("hij,hi->hj", S[s], q[t])
    return out, S


def logprobs(x, ids, top):
    """dict like native.token_logprobs's, in 64 bits."""
    x = x.astype(np.float64)
    M, V = x.shape
    r = {"lse": np.empty(M), "entropy": np.empty(M), "top_ids": np.empty((M, top), np.int64),
         "logprobs": np.empty(ids.shape), "top_logprobs": np.empty((M, top))}
    for i in range(M):
        y = x[i]
        rank = np.where(np.isnan(y), np.inf, y)
        order = np.lexsort((np.arange(V), -rank, ~np.isnan(y)))[:top]
        r["top_ids"][i] = order
        if np.isnan(y).any() or np.isposinf(y).any():
            lse, lp, ent = np.nan, np.full(V, np.nan), np.nan
        elif np.isneginf(y).all():
            lse, lp, ent = -np.inf, np.full(V, -np.inf), 0.0
        else:
            m = y.max()
            e = np.exp(y - m)
            lse = m + np.log(e.sum())
            lp = (y - m) - np.log(e.sum())
            p = np.exp(lp)
            ent = -np.sum(p[p > 0] * lp[p > 0])
        r["lse"][i], r["entropy"][i] = lse, ent
        r["top_logprobs"][i] = lp[order]
        for j, t in enumerate(ids[i]):
            r["logprobs"][i, j] = 0.0 if t == -1 else lp[t] if 0 <= t < V else np.nan
    return r
