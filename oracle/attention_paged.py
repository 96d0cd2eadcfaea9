"""fp64 restatement of the target-side attention operators over a paged cache.

Per-head RMSNorm with rotate-half rotation, the paged append, and the attention
of ragged chunks over their pages, request by request and head by head, from
the formulas.  Test infrastructure only (see the package's docstring).
"""

import numpy as np


def norm_rope(x, gain, pos, base, eps):
    """x [n, heads, hd] at positions pos [n]; gain None: no norm, base None: no rotation."""
    y = np.asarray(x, dtype=np.float64)
    hd = y.shape[-1]
    if gain is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    if base is None:
        return y
    half = hd // 2
    ang = np.asarray(pos, np.float64)[:, None] * base ** (-2.0 * np.arange(half) / hd)
    c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
    a, b = y[..., :half], y[..., half:]
    return np.concatenate((a * c - b * s, b * c + a * s), -1)


def rotated_bound(x, gain, eps):
    """|a| + |b| of every rotation pair (normalised), the scale of a rotation's fp32 error."""
    y = np.abs(norm_rope(x, gain, None, None, eps))
    half = y.shape[-1] // 2
    t = y[..., :half] + y[..., half:]
    return np.concatenate((t, t), -1)


def positions(cu_rows, start_pos):
    """Position of every row below cu_rows[-1]."""
    return np.concatenate([np.arange(n) + s for n, s in
                           zip(np.diff(cu_rows), start_pos)] or [np.zeros(0, int)])


def append(k, v, k_pool, v_pool, table, cu_rows, start_pos):
    """Writes rows k, v [n, n_kv, hd] into float64 copies of the pools [pages, n_kv, P, hd]."""
    P = k_pool.shape[2]
    for r in range(len(start_pos)):
        for i in range(cu_rows[r], cu_rows[r + 1]):
            p = start_pos[r] + i - cu_rows[r]
            k_pool[table[r][p // P], :, p % P] = k[i]
            v_pool[table[r][p // P], :, p % P] = v[i]


def gather(pool, pages, length):
    """The first `length` positions of a request: [n_kv, length, hd] (slots read only below it)."""
    P = pool.shape[2]
    out = np.zeros((pool.shape[1], length, pool.shape[3]))
    for j in range(0, length, P):
        n = min(P, length - j)
        if 0 <= pages[j // P] < pool.shape[0]:
            out[:, j:j + n] = pool[pages[j // P], :, :n]
    return out


def attention(q, k_pool, v_pool, table, cu_rows, start_pos, kv_len, scale, causal=True, window=0):
    """(out, lse, mass): mass[row, head, d] = sum_j p_j |v_jd|, the scale of the weights'
    rounding.  Masked keys do not take part at all (whatever their values)."""
    q = np.asarray(q, np.float64)
    n, nq, hd = q.shape
    nkv = k_pool.shape[1]
    out, mass = np.zeros((n, nq, hd)), np.zeros((n, nq, hd))
    lse = np.full((n, nq), -np.inf)
    for r in range(len(start_pos)):
        K, V = (gather(p, table[r], int(kv_len[r])) for p in (k_pool, v_pool))
        for i in range(cu_rows[r], cu_rows[r + 1]):
            p = start_pos[r] + i - cu_rows[r]
            hi = min(kv_len[r], p + 1) if causal else kv_len[r]
            lo = max(0, p - window + 1) if window else 0
            if hi <= lo:
                continue
            for h in range(nkv):
                G = nq // nkv
                z = scale * (q[i, h * G:(h + 1) * G] @ K[h, lo:hi].T)  # [G, keys]
                m = z.max(-1, keepdims=True)
                e = np.exp(z - m)
                l = e.sum(-1, keepdims=True)
                with np.errstate(invalid="ignore"):  # infinities in visible keys
                    out[i, h * G:(h + 1) * G] = (e / l) @ V[h, lo:hi]
                    mass[i, h * G:(h + 1) * G] = (e / l) @ np.abs(V[h, lo:hi])
                lse[i, h * G:(h + 1) * G] = (m + np.log(l))[:, 0]
    return out, lse, mass


def score_error(q, k_pool, table, cu_rows, start_pos, kv_len, scale):
    """Largest sum_d |q_d k_d| * scale of any row and key: times a step, the fp32 error of a score."""
    q = np.abs(np.asarray(q, np.float64))
    worst = 0.0
    nkv = k_pool.shape[1]
    G = q.shape[1] // nkv
    for r in range(len(start_pos)):
        K = np.abs(gather(k_pool, table[r], int(kv_len[r])))
        for h in range(nkv):
            qq = q[cu_rows[r]:cu_rows[r + 1], h * G:(h + 1) * G].reshape(-1, q.shape[2])
            if qq.size and K.shape[1]:
                s = qq @ np.nan_to_num(K[h], nan=0.0, posinf=0.0, neginf=0.0).T
                worst = max(worst, float(np.nanmax(s)) * scale)
    return worst
