"""Float64 definitions of the attention layer's operators (NumPy only; shares no code with the HIP library).

Every row is computed over exactly the keys it sees, so what it does not see cannot reach it.
"""
from __future__ import annotations

import numpy as np


def rotation(cos, sin, pos, rot, d, interleaved):
    """R(p) as a [..., d, d] matrix for positions pos [...]: NaN rows for a position outside the table."""
    pos = np.asarray(pos)
    R = np.zeros(pos.shape + (d, d))
    R[...] = np.eye(d)
    inside = (pos >= 0) & (pos < len(cos))
    p = np.where(inside, pos, 0)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c = np.where(inside, cos[p, i], np.nan)
        s = np.where(inside, sin[p, i], np.nan)
        R[..., a, a], R[..., a, b], R[..., b, a], R[..., b, b] = c, -s, s, c
    return R


def norm_rope(x, w, cos, sin, pos, rot, interleaved, norm, eps):
    """y = R(p) (x r w) for x [..., H, d] at positions pos [...]."""
    x = np.asarray(x, np.float64)
    z = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) if norm else x
    if w is not None:
        z = z * w
    if not rot:
        return z
    R = rotation(cos, sin, pos, rot, x.shape[-1], interleaved)
    turned = np.einsum("...ij,...hj->...hi", R[..., :rot, :rot], z[..., :rot])
    return np.concatenate([turned, z[..., rot:]], axis=-1)


def norm_rope_grad(x, w, dy, cos, sin, pos, rot, interleaved, norm, eps):
    """(dx, dw) of norm_rope from dy; dw None without weights."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    d = x.shape[-1]
    dz = dy
    if rot:
        R = rotation(cos, sin, pos, rot, d, interleaved)
        dz = np.concatenate([np.einsum("...ij,...hi->...hj", R[..., :rot, :rot], dy[..., :rot]), dy[..., rot:]], axis=-1)
    if not norm:
        return dz, None
    s = np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    dw = np.sum((dz * x / s).reshape(-1, d), axis=0) if w is not None else None
    u = dz * (1.0 if w is None else w)
    # d/dx_i of sum_j u_j x_j / s:  u_i / s - x_i (u . x) / (d s^3)
    return u / s - x * np.sum(u * x, axis=-1, keepdims=True) / (d * s ** 3), dw


def token_places(cu, kv_lens, N):
    """For each of N packed tokens (sequence, position), or None behind the last sequence."""
    out = []
    for n in range(N):
        s = next((s for s in range(len(kv_lens)) if cu[s] <= n < cu[s + 1]), None)
        out.append(None if s is None else (s, max(int(kv_lens[s]), 0) - int(cu[s + 1] - cu[s]) + n - int(cu[s])))
    return out


def place(table, s, pos, page_size, pages):
    """(page, offset) of position pos of sequence s, or None when the cache does not hold it."""
    if pos < 0 or pos // page_size >= table.shape[1]:
        return None
    page = int(table[s, pos // page_size])
    return (page, pos % page_size) if 0 <= page < pages else None


def paged_append(k, v, k_cache, v_cache, table, kv_lens, cu, page_size, turn=lambda k, pos: k):
    """Caches after the append (copies); turn(k_rows, pos) norms and rotates one token's keys."""
    kc, vc = np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    for n, at in enumerate(token_places(cu, kv_lens, len(k))):
        if at is None:
            continue
        cell = place(table, at[0], at[1], page_size, len(kc))
        if cell is not None:
            kc[cell], vc[cell] = turn(k[n], at[1]), v[n]
    return kc, vc


def paged_attention(q, k_cache, v_cache, table, kv_lens, cu, scale, window):
    """(o, lse, mean_abs, reach, keys): o and lse with NaN rows behind the last sequence; the softmax mean of |v|,
    the largest sum_i |q_i k_ji| over the visible keys, and their number, for error bounds."""
    N, Hq, d = q.shape
    pages, page_size, Hk = k_cache.shape[:3]
    G = Hq // Hk
    o, A = np.full((N, Hq, d), np.nan), np.zeros((N, Hq, d))
    lse, reach, keys = np.full((N, Hq), np.nan), np.zeros((N, Hq)), np.zeros(N, int)
    for n, at in enumerate(token_places(cu, kv_lens, N)):
        if at is None:
            continue
        s, p = at
        first = max(0, p - window + 1) if window else 0
        cells = [place(table, s, j, page_size, pages) for j in range(first, p + 1)]
        cells = [c for c in cells if c is not None]
        o[n], lse[n], keys[n] = 0.0, -np.inf, len(cells)
        if not cells:
            continue
        pg, off = np.array(cells).T
        K, V = k_cache[pg, off], v_cache[pg, off]          # [keys, Hk, d]
        for h in range(Hq):
            x = scale * (K[:, h // G] @ q[n, h])
            m = np.max(x)
            e = np.exp(x - m)
            o[n, h] = e @ V[:, h // G] / e.sum()
            A[n, h] = e @ np.abs(V[:, h // G]) / e.sum()
            lse[n, h] = m + np.log(e.sum())
            reach[n, h] = np.max(np.abs(K[:, h // G]) @ np.abs(q[n, h]))
    return o, lse, A, reach, keys
