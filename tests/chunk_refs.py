"""Plain 64-bit forms of the rotation and append, the attention of a chunk of
tokens and the adjusted logits (numpy, from their formulas), for the tests."""
import numpy as np


def places(at, lens, T):
    """(sequence, position) of each token; -1 where it belongs to none."""
    seq, pos = np.full(T, -1), np.zeros(T, np.int64)
    for s in range(len(lens)):
        a, b = (min(max(int(x), 0), T) for x in at[s:s + 2])
        seq[a:b] = s
        pos[a:b] = int(lens[s]) - (b - a) + np.arange(b - a)
    return seq, pos


def rotate(x, angle, factor, interleaved):
    """x [T][H][d] turned by angle [T][rot / 2]."""
    y, rot = x.astype(np.float64).copy(), 2 * angle.shape[1]
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    c, s = (factor * f(angle)[:, None] for f in (np.cos, np.sin))
    a, b = y[..., one].copy(), y[..., two].copy()
    y[..., one], y[..., two] = a * c - b * s, a * s + b * c
    return y


def append(k_pool, v_pool, k, v, table, at, lens):
    """Stores the tokens of k and v [T][Hkv][d] in the pools (changed)."""
    n_pages, _, page, _ = k_pool.shape
    seq, pos = places(at, lens, len(k))
    for t in range(len(k)):
        if seq[t] < 0 or not 0 <= pos[t] < table.shape[1] * page:
            continue
        pg = int(table[seq[t], pos[t] // page])
        if 0 <= pg < n_pages:
            k_pool[pg, :, pos[t] % page], v_pool[pg, :, pos[t] % page] = k[t], v[t]


def chunk_attention(q, k_pool, v_pool, table, at, lens, scale, cap=None):
    """out (NaN in rows of no sequence), lse, and the parts of an output's bound:
    the absolute weighted values, the largest sum |q||k| of a head, and the
    number of keys times the largest |value|."""
    T, Hq, d = q.shape
    n_pages, Hkv, page, _ = k_pool.shape
    group = Hq // Hkv
    out, lse = np.full((T, Hq, d), np.nan), np.full((T, Hq), np.nan)
    mass, reach, most = np.zeros((T, Hq, d)), np.zeros((T, Hq)), np.zeros((T, Hq))
    seq, pos = places(at, lens, T)
    for s in range(len(lens)):
        t = np.flatnonzero(seq == s)
        if not len(t):
            continue
        n = max(0, min(int(lens[s]), table.shape[1] * page, cap if cap else 1 << 62))
        j = np.arange(n)
        pg = table[s, j // page]
        ok = (pg >= 0) & (pg < n_pages)
        j, pg = j[ok], pg[ok]
        seen = j <= pos[t][:, None]
        for h in range(Hq):
            k, v = (x[pg, h // group, j % page].astype(np.float64) for x in (k_pool, v_pool))
            qh = q[t, h].astype(np.float64)
            with np.errstate(all="ignore"):
                x = np.where(seen, qh @ k.T * scale, -np.inf)
                m = x.max(1, initial=-np.inf, keepdims=True)
                p = np.where(seen, np.exp(x - np.where(np.isneginf(m), 0, m)), 0)
                total = p.sum(1, keepdims=True)
                # a key that is not seen adds nothing, whatever its value is
                odd = ~np.isfinite(v).all(1)
                y = p[:, ~odd] @ v[~odd]
                for i in np.flatnonzero(odd):
                    y[seen[:, i]] += p[seen[:, i], i, None] * v[i]
                some = np.where(total == 0, 1, total)
                out[t, h] = y / some
                lse[t, h] = np.where(total == 0, -np.inf, m + np.log(some))[:, 0]
                mass[t, h] = (p[:, ~odd] @ np.abs(v[~odd])) / some
                if len(j):
                    reach[t, h] = np.where(seen, np.abs(qh) @ np.abs(k).T, 0).max(1) * abs(scale)
                    most[t, h] = seen.sum(1) * np.abs(v[~odd]).max(initial=0)
    return out, lse, mass, reach, most


def adjust_logits(x, ids, at, prompt, repetition, frequency, presence, bias_ids, bias, bias_at, allowed, allowed_rows):
    y = x.astype(np.float64).copy()
    M, V = y.shape
    for m in range(M):
        if ids is not None:
            a, b = (min(max(int(i), 0), len(ids)) for i in at[m:m + 2])
            mine = ids[a:b]
            late = mine[max(0, int(prompt[m])) if prompt is not None else 0:]
            some = np.unique(mine[(mine >= 0) & (mine < V)])
            r = 1.0 if repetition is None else float(repetition[m])
            with np.errstate(all="ignore"):
                y[m, some] = np.where(y[m, some] > 0, y[m, some] / r, y[m, some] * r)
                some, c = np.unique(late[(late >= 0) & (late < V)], return_counts=True)
                f = 0.0 if frequency is None else float(frequency[m])
                y[m, some] -= f * c + (0.0 if presence is None else float(presence[m]))
        if bias_ids is not None:
            for j in range(*(min(max(int(i), 0), len(bias_ids)) for i in bias_at[m:m + 2])):
                if 0 <= bias_ids[j] < V:
                    y[m, bias_ids[j]] += float(bias[j])
        if allowed is not None:
            r = m if allowed_rows is None else int(allowed_rows[m])
            if 0 <= r < len(allowed):
                i = np.arange(V)
                y[m, (allowed[r].view(np.uint32)[i // 32] >> (i % 32).astype(np.uint32)) & 1 == 0] = -np.inf
    return y
