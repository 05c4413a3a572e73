"""PyTorch-facing binding of the paged cache in 4 bits, and of the room in a paged cache of either kind.

`paged_assign` works out on the GPU which pages the next tokens of a batch go to: block table, lengths, offsets,
positions and slots, for these calls and for `paged_append` and `paged_attention` alike. `paged_append_fp4` and
`paged_attention_fp4` are the latter two over a cache of 4-bit codes (4.25 bits a value with the scales, 17/64 of the
bf16 cache's bytes), and `paged_read_fp4` gives the values back. `paged_fp4_cache` makes such a cache. Argument
marshalling only: every step runs in the HIP library.

A cache is four uint8 tensors, k_cache and v_cache [pages, page_size, Hk, d / 2] and k_scale and v_scale [pages,
page_size, Hk, d / 32]. Every 32 channels of a head share one scale 2^(byte - 127) (2 to 252; 255: NaN); a code is a
sign and 0, 0.5, 1, 1.5, 2, 3, 4 or 6, two to a byte with the even channel in the low half. Page, token and head
strides are free.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _lib
from .api import _DTYPES
from .attention import (_I32, _MOST, _angles, _dense, _first, _flags, _flat, _like, _on, _rows, _sequences, _window,
                        _workspace)

_U8 = torch.uint8


def _pack(*values):
    try:
        return _lib.pack_fp4(*values)
    except struct.error as e:            # a size past its bits, or a scale or eps that is no float
        raise ValueError(f"a value that the configuration does not hold: {e}") from None


def paged_fp4_cache(pages, page_size, heads, d, device="cuda"):
    """(k_cache, k_scale, v_cache, v_scale) for `pages` pages, the order in which the other functions take them. In
    memory a head's tokens of a page follow each other, which is the fastest to read. Not initialised: entries that
    no token was stored in are read by nobody but paged_read_fp4."""
    if d not in (64, 128):
        raise ValueError(f"d: expected 64 or 128, got {d}")
    if page_size < 1 or page_size & (page_size - 1):
        raise ValueError(f"page_size: expected a power of two, got {page_size}")
    return tuple(torch.empty((pages, heads, page_size, n), dtype=_U8, device=device).transpose(1, 2)
                 for n in (d // 2, d // 32) * 2)


def _fp4_cache(k_cache, k_scale, v_cache, v_scale, Hk, d, dev):
    """(pages, page size, strides of the codes as a paged config has them, strides of the scales)."""
    shape, small = k_cache.shape, k_scale.shape
    if len(shape) != 4 or shape[2] != Hk or 2 * shape[3] != d:
        raise ValueError(f"k_cache: expected [pages, page_size, {Hk}, {d // 2}], got {tuple(shape)}")
    pages, page_size = shape[0], shape[1]
    if pages > _MOST or page_size > _MOST:
        raise ValueError(f"k_cache: sizes past 32 bits: {tuple(shape)}")
    want = (pages, page_size, Hk, d // 32)
    at = dev.index
    if not (v_cache.shape == shape and small == want and v_scale.shape == small
            and k_cache.dtype is _U8 and k_scale.dtype is _U8 and v_cache.dtype is _U8 and v_scale.dtype is _U8
            and k_cache.get_device() == at and k_scale.get_device() == at and v_cache.get_device() == at
            and v_scale.get_device() == at):
        for t, name, s in ((k_cache, "k_cache", shape), (k_scale, "k_scale", want), (v_cache, "v_cache", shape),
                           (v_scale, "v_scale", want)):
            if t.shape != s:
                raise ValueError(f"{name}: expected shape {tuple(s)}, got {tuple(t.shape)}")
            _like(t, name, _U8, dev)
    kp, kt, kh, k1 = k_cache.stride()
    sp, st, sh, s1 = k_scale.stride()
    vp, vt, vh, v1 = v_cache.stride()
    tp, tt, th, t1 = v_scale.stride()
    if k1 != 1 or s1 != 1 or v1 != 1 or t1 != 1:
        raise ValueError("the bytes of a head must be contiguous in codes and scales")
    return pages, page_size, (kp, kt, kh, vp, vt, vh), (sp, st, sh, tp, tt, th)


def paged_append_fp4(k, v, k_cache, k_scale, v_cache, v_scale, block_table, kv_lens, cu_seqlens=None, cos=None,
                     sin=None, q=None, q_weight=None, k_weight=None, norm=False, eps=1e-6, interleaved=False, q_out=None,
                     stream=None):
    """paged_append into a cache in 4 bits: the same arguments, checks and result, with the cache's four tensors in the
    place of two (see the module's text). A block of 32 channels takes the smallest scale 2^e with max |x| <= 7 2^e
    (-125 <= e <= 125), a value the nearest code, the even one of two; a block with an infinity or NaN is stored as NaN.
    Keys are normed and rotated first where that is asked for, and rounded to the input's type as qk_norm_rope_fwd does."""
    dt, dev = _first(k, "k", "paged_append_fp4")
    sk = k.shape
    if len(sk) != 3:
        raise ValueError(f"k: expected [tokens, heads, d], got {tuple(sk)}")
    N, Hk, d = sk
    pages, page_size, codes, scales = _fp4_cache(k_cache, k_scale, v_cache, v_scale, Hk, d, dev)
    S, width, table_row, step, cu, lens, table = _sequences(block_table, kv_lens, cu_seqlens, N, dev)
    pc, ps, rot, table_len = _angles(cos, sin, dev)
    flags = step | _flags(norm, interleaved, q_weight, k_weight)
    wq, wk = _flat(q_weight, "q_weight", (d,), dt, dev), _flat(k_weight, "k_weight", (d,), dt, dev)
    Hq = q_row = o_row = 0
    pq = po = None
    with _on(dev, stream):
        if q is not None:
            sq = q.shape
            if len(sq) != 3 or sq[0] != N or sq[2] != d:
                raise ValueError(f"q: expected shape {(N, 'heads', d)}, got {tuple(sq)}")
            Hq, q_row, pq = sq[1], _rows(q, "q", sq, dt, dev), q.data_ptr()
            q_out = _dense(q) if q_out is None else q_out
            o_row, po = _rows(q_out, "q_out", sq, dt, dev), q_out.data_ptr()
        elif q_weight is not None or q_out is not None:
            raise ValueError("q_weight and q_out belong to q")
        c = _pack(N, S, Hq, Hk, d, page_size, pages, width, rot, table_len, 0, _DTYPES[dt], flags, eps, 1.0, q_row,
                  _rows(k, "k", sk, dt, dev), _rows(v, "v", sk, dt, dev), o_row, table_row, *codes, *scales)
        code = _lib.lib().carve_paged_append_fp4(c, k.data_ptr(), v.data_ptr(), pq, wq, wk, pc, ps, cu, lens, table,
                                                 k_cache.data_ptr(), k_scale.data_ptr(), v_cache.data_ptr(),
                                                 v_scale.data_ptr(), po, torch._C._cuda_getCurrentRawStream(dev.index))
    if code:
        _lib.check(code)
    return q_out


def paged_read_fp4(k_cache, k_scale, v_cache, v_scale, slots, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """The values that cache entries stand for: (k, v), each [*slots.shape, Hk, d] of `dtype` (bf16 and fp32 hold them
    exactly), from entry slots % page_size of page slots // page_size. slots int64; one outside the cache gives zeros."""
    if k_cache.device.type != "cuda":
        raise ValueError("paged_read_fp4 runs on the GPU only; move the inputs to a cuda device")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    dev = k_cache.device
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache: expected [pages, page_size, heads, d / 2], got {tuple(k_cache.shape)}")
    Hk, d = k_cache.shape[2], 2 * k_cache.shape[3]
    pages, page_size, codes, scales = _fp4_cache(k_cache, k_scale, v_cache, v_scale, Hk, d, dev)
    lead = slots.shape
    N = slots.numel()
    if N > _MOST or Hk > _MOST:
        raise ValueError(f"sizes past 32 bits: {N} slots of {Hk} heads")
    at = _flat(slots, "slots", lead, torch.int64, dev)
    shape = (*lead, Hk, d)
    k_row = v_row = Hk * d
    with _on(dev, stream):
        if k_out is None and v_out is None:
            k_out, v_out = torch.empty((2, *shape), dtype=dtype, device=dev).unbind()    # one allocation
        else:
            shape = torch.Size(shape)
            k_out = torch.empty(shape, dtype=dtype, device=dev) if k_out is None else k_out
            v_out = torch.empty(shape, dtype=dtype, device=dev) if v_out is None else v_out
            k_row, v_row = _rows(k_out, "k_out", shape, dtype, dev), _rows(v_out, "v_out", shape, dtype, dev)
        c = _pack(N, 0, 0, Hk, d, page_size, pages, 0, 0, 0, 0, _DTYPES[dtype], 0, 0.0, 0.0, 0, k_row, v_row, 0, 0,
                  *codes, *scales)
        code = _lib.lib().carve_paged_read_fp4(c, k_cache.data_ptr(), k_scale.data_ptr(), v_cache.data_ptr(),
                                               v_scale.data_ptr(), at, k_out.data_ptr(), v_out.data_ptr(),
                                               torch._C._cuda_getCurrentRawStream(dev.index))
    if code:
        _lib.check(code)
    return k_out, v_out


def paged_attention_fp4(q, k_cache, k_scale, v_cache, v_scale, block_table, kv_lens, cu_seqlens=None, scale=None,
                        window=0, out=None, return_lse=False, workspace=None, stream=None):
    """paged_attention over a cache in 4 bits: the same arguments, checks and result, with the cache's four tensors in
    the place of two. workspace: device scratch to use (paged_fp4_workspace_bytes of it); allocated when None."""
    dt, dev = _first(q, "q", "paged_attention_fp4")
    sq = q.shape
    if len(sq) != 3:
        raise ValueError(f"q: expected [tokens, heads, d], got {tuple(sq)}")
    N, Hq, d = sq
    Hk = k_cache.shape[2] if k_cache.dim() == 4 else 0
    pages, page_size, codes, scales = _fp4_cache(k_cache, k_scale, v_cache, v_scale, Hk, d, dev)
    S, width, table_row, step, cu, lens, table = _sequences(block_table, kv_lens, cu_seqlens, N, dev)
    L = _lib.lib()
    lse = pl = None
    with _on(dev, stream):
        if out is None:
            out, o_row = _dense(q), Hq * d
        else:
            o_row = _rows(out, "out", sq, dt, dev)
        c = _pack(N, S, Hq, Hk, d, page_size, pages, width, 0, 0, _window(window), _DTYPES[dt], step, 0.0,
                  d ** -0.5 if scale is None else scale, _rows(q, "q", sq, dt, dev), 0, 0, o_row, table_row, *codes,
                  *scales)
        if return_lse:
            lse = torch.empty((N, Hq), dtype=torch.float32, device=dev)
            pl = lse.data_ptr()
        need = ctypes.c_int64()
        code = L.carve_paged_workspace_fp4(c, need)
        if code:
            _lib.check(code)
        workspace, ws = _workspace(workspace, need.value, dev)
        code = L.carve_paged_attention_fp4(c, q.data_ptr(), k_cache.data_ptr(), k_scale.data_ptr(), v_cache.data_ptr(),
                                           v_scale.data_ptr(), cu, lens, table, out.data_ptr(), pl, ws, need.value,
                                           torch._C._cuda_getCurrentRawStream(dev.index))
    if code:
        _lib.check(code)
    return (out, lse) if return_lse else out


def paged_fp4_workspace_bytes(N, S, Hq, Hk, d, page_size, width, dtype=torch.bfloat16, window=0, step=False):
    """Bytes of workspace paged_attention_fp4 needs for N new tokens of S sequences (step: one each) with a block table
    `width` pages wide."""
    for name, n in (("N", N), ("S", S), ("Hq", Hq), ("Hk", Hk), ("d", d), ("page_size", page_size), ("width", width)):
        if not 0 <= n <= _MOST:
            raise ValueError(f"{name}: expected a size of 32 bits, got {n}")
    half, small = d // 2, d // 32
    c = _pack(N, S, Hq, Hk, d, page_size, 1, width, 0, 0, _window(window), _DTYPES[dtype],
              _lib.CARVE_PAGED_STEP if step else 0, 0.0, 1.0, 0, 0, 0, 0, width, *(half,) * 6, *(small,) * 6)
    need = ctypes.c_int64()
    _lib.check(_lib.lib().carve_paged_workspace_fp4(c, need))
    return need.value


def paged_assign(block_table, kv_lens, new_lens, free_pages, free_count, page_size, tokens, done=None, kv_lens_out=None,
                 free_count_out=None, stream=None):
    """Room in a paged cache for the next tokens of S requests, worked out on the GPU (nothing is read by the host, so a
    captured step goes on from the last one). Shapes, int32: block_table [S, pages each], written in place; kv_lens
    [S], tokens held before; new_lens [S], tokens to come; done [S] or None: nonzero where the request that held the
    slot has ended (its pages are freed first, its length starts at 0); free_pages [capacity], a stack whose entries
    [0, free_count[0]) nobody holds, written in place above them; free_count [2]: pages free, pages lacking so far.
    tokens: rows of positions and slots, at least the sum of new_lens (what is past it gets none).
    Returns (cu_seqlens [S + 1], kv_lens_out [S], positions [tokens], slots [tokens] int64, free_count_out [2]):
    kv_lens_out and cu_seqlens as paged_append and paged_attention take them, positions as qk_norm_rope_fwd does (0 behind
    the last token), slots as paged_read_fp4 does (page * page_size + offset; -1 behind the last token and where no page
    is). Requests are served in their order; one that finds the stack empty has -1 in its table, which is counted in
    free_count_out[1], and those tokens are neither stored nor seen. kv_lens_out may be kv_lens, free_count_out
    free_count. A page that several requests hold must not be in the table of one that has ended. Entries past
    ceil(kv_lens / page_size) are taken for empty: where a length is set back (drafted tokens that were rejected), the
    pages past it have to be put on the stack first, or they are lost."""
    dev = block_table.device
    if dev.type != "cuda":
        raise ValueError("paged_assign runs on the GPU only; move the inputs to a cuda device")
    if block_table.dim() != 2:
        raise ValueError(f"block_table: expected [requests, pages each], got {tuple(block_table.shape)}")
    S, width = block_table.shape
    if block_table.dtype is not _I32:
        _like(block_table, "block_table", _I32, dev)
    row, step = block_table.stride()
    if S and width > 1 and step != 1:
        raise ValueError("block_table: a request's entries must be contiguous")
    if free_pages.dim() != 1:
        raise ValueError(f"free_pages: expected one dimension, got {tuple(free_pages.shape)}")
    if not 0 <= tokens <= _MOST:
        raise ValueError(f"tokens: expected a size of 32 bits, got {tokens}")
    if not 0 <= page_size <= _MOST or S > _MOST or width > _MOST:
        raise ValueError(f"sizes past 32 bits: pages of {page_size}, a block_table of {tuple(block_table.shape)}")
    args = [_flat(kv_lens, "kv_lens", (S,), _I32, dev), _flat(new_lens, "new_lens", (S,), _I32, dev),
            _flat(done, "done", (S,), _I32, dev), block_table.data_ptr(),
            _flat(free_pages, "free_pages", free_pages.shape, _I32, dev), _flat(free_count, "free_count", (2,), _I32, dev)]
    with _on(dev, stream):
        # one allocation for what has 32 bits
        cu, positions, lens, count = torch.empty(2 * S + tokens + 3, dtype=_I32, device=dev).split_with_sizes(
            (S + 1, tokens, S, 2))
        kv_lens_out = lens if kv_lens_out is None else kv_lens_out
        free_count_out = count if free_count_out is None else free_count_out
        slots = torch.empty(tokens, dtype=torch.int64, device=dev)
        c = _lib.pack_assign(S, tokens, page_size, width, row if S > 1 else width, free_pages.numel())
        code = _lib.lib().carve_paged_assign(
            c, *args, _flat(kv_lens_out, "kv_lens_out", (S,), _I32, dev), cu.data_ptr(), positions.data_ptr(),
            slots.data_ptr(), _flat(free_count_out, "free_count_out", (2,), _I32, dev),
            torch._C._cuda_getCurrentRawStream(dev.index))
    if code:
        _lib.check(code)
    return cu, kv_lens_out, positions, slots, free_count_out
