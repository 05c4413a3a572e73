"""Float64 definitions of the 4-bit paged cache and of the room in a paged cache (NumPy only; shares no code with the
HIP library)."""
from __future__ import annotations

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6.0])
BLOCK = 32


def encode_block(x):
    """(codes [32], scale byte) of one block."""
    x = np.asarray(x, np.float64)
    if not np.isfinite(x).all():
        return np.zeros(BLOCK, np.uint8), 255
    top = np.abs(x).max()
    e = -125
    while e < 125 and top > 7 * 2.0 ** e:
        e += 1
    codes = np.zeros(BLOCK, np.uint8)
    for i, v in enumerate(x):
        far = np.abs(abs(v) / 2.0 ** e - GRID)
        near = np.flatnonzero(far == far.min())
        codes[i] = near[0] if len(near) == 1 else near[near % 2 == 0][0]
        if np.signbit(v):
            codes[i] |= 8
    return codes, e + 127


def encode(x):
    """(packed codes [..., d / 2], scales [..., d / 32]) of x [..., d]."""
    x = np.asarray(x, np.float64)
    flat = x.reshape(-1, BLOCK)
    codes, scales = np.zeros(flat.shape, np.uint8), np.zeros(len(flat), np.uint8)
    for i, b in enumerate(flat):
        codes[i], scales[i] = encode_block(b)
    codes = codes.reshape(x.shape)
    return codes[..., ::2] | codes[..., 1::2] << 4, scales.reshape(*x.shape[:-1], -1)


def decode(codes, scales):
    codes, scales = np.asarray(codes), np.asarray(scales).astype(np.float64)
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales - 127))
    return np.where(c & 8, -1.0, 1.0) * GRID[c & 7] * np.repeat(s, BLOCK, -1)


def assign(table, kv_lens, new_lens, free_pages, free_count, page_size, tokens, done=None):
    """(cu, lengths, positions, slots, free count, table, free pages) after room was made for new_lens."""
    table, free = np.array(table, np.int64), [int(x) for x in free_pages]
    width, cap = table.shape[1], len(free)
    top, lacking = min(max(int(free_count[0]), 0), cap), int(free_count[1])
    pages = lambda n: min(-(-n // page_size), width)  # noqa: E731
    old = [max(int(n), 0) for n in kv_lens]
    if done is not None:
        for s in range(len(old)):
            if done[s]:
                for p in table[s, :pages(old[s])]:
                    if p >= 0 and top < cap:
                        free[top] = int(p)
                        top += 1
                old[s] = 0
    cu, lens, positions, slots = [0], [], np.zeros(tokens, np.int64), np.full(tokens, -1, np.int64)
    for s, n in enumerate(max(int(n), 0) for n in new_lens):
        for i in range(pages(old[s]), pages(old[s] + n)):
            if top > 0:
                top -= 1
                table[s, i] = free[top]
            else:
                lacking += 1
                table[s, i] = -1
        for i in range(n):
            t, p = cu[-1] + i, old[s] + i
            if t < tokens:
                positions[t] = p
                if p // page_size < width and table[s, p // page_size] >= 0:
                    slots[t] = table[s, p // page_size] * page_size + p % page_size
        lens.append(old[s] + n)
        cu.append(cu[-1] + n)
    return cu, lens, positions, slots, (top, lacking), table, free
