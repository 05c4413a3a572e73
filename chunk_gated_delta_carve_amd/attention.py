"""PyTorch-facing binding of the attention layer that stands beside the CARVE mixer in a hybrid model.

`qk_norm_rope_fwd` and `qk_norm_rope_bwd` norm and rotate queries and keys, `paged_append` puts new
keys and values into a paged cache with both applied on the way, and `paged_attention` lets new
tokens attend to that cache, a prompt chunk or a single token per sequence. `rope_tables` makes the
tables of angles. Argument marshalling only: every step runs in the HIP library.

Tensors may be views as long as a head's channels are contiguous and its neighbours follow it: q and
k may be parts of one projection's output, a cache may have its pages, tokens and heads in any order.
Lengths, offsets and block tables stay on the device and are not read by the host, so a captured
graph follows them when they change.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import _lib
from .api import _DTYPES

_I32 = torch.int32
_MOST = 2**31 - 1                        # the library's sizes have 32 bits


def rope_tables(length, rot, base=10000.0, device="cuda"):
    """(cos, sin), each [length, rot / 2] fp32: the angles p base^(-2i / rot) of positions p, formed in
    64 bits (at position 10^5 a 32-bit angle would be off by up to 2^-8)."""
    if rot <= 0 or rot % 16:
        raise ValueError(f"rot: expected a positive multiple of 16, got {rot}")
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(length, dtype=torch.float64, device=device)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def _like(t, name, dtype, device):
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")


def _flat(t, name, shape, dtype, device):
    """A dense tensor's address (None for None)."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype or t.device != device:
        _like(t, name, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _rows(t, name, shape, dtype, device):
    """Elements from one token of t [*lead, H, d] to the next."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype or t.device != device:
        _like(t, name, dtype, device)
    H, d = shape[-2], shape[-1]
    if t.is_contiguous() or t.numel() == 0:
        return H * d
    stride = t.stride()
    if stride[-1] != 1 or (H > 1 and stride[-2] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    row, size = H * d, 0                 # the token dimensions must step evenly
    for i in range(len(shape) - 3, -1, -1):
        n = shape[i]
        if n == 1:
            continue
        if not size:
            row, size = stride[i], 1
        elif stride[i] != row * size:
            raise ValueError(f"{name}: tokens must be evenly spaced")
        size *= n
    return row


def _dense(like):
    return torch.empty_like(like, memory_format=torch.contiguous_format)


class _On:
    """The given stream and the tensors' device made current: temporaries belong to the stream that the kernels
    run on."""

    def __init__(self, device, stream):
        handle = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream
        self.stack = contextlib.ExitStack()
        self.stack.enter_context(torch.cuda.device(device))
        if handle is not None and handle != torch._C._cuda_getCurrentRawStream(device.index):
            s = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
            self.stack.enter_context(torch.cuda.stream(s))

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return self.stack.__exit__(*exc)


_HERE = contextlib.nullcontext()         # nothing to change: the usual case, on the device and stream that are current


def _on(device, stream):
    return _HERE if stream is None and device.index == torch._C._cuda_getDevice() else _On(device, stream)


def _first(t, name, what):
    device, dtype = t.device, t.dtype
    if device.type != "cuda":
        raise ValueError(f"{what} runs on the GPU only; move the inputs to a cuda device")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    if t.dim() < 3:
        raise ValueError(f"{name}: expected [..., heads, d], got {tuple(t.shape)}")
    return dtype, device


def _angles(cos, sin, device):
    if cos is None and sin is None:
        return None, None, 0, 0
    if cos is None or sin is None:
        raise ValueError("cos and sin come together")
    shape = cos.shape
    if len(shape) != 2:
        raise ValueError(f"cos: expected [positions, rot / 2], got {tuple(shape)}")
    if shape[0] > _MOST or 2 * shape[1] > _MOST:
        raise ValueError(f"cos: sizes past 32 bits: {tuple(shape)}")
    return (_flat(cos, "cos", shape, torch.float32, device), _flat(sin, "sin", shape, torch.float32, device),
            2 * shape[1], shape[0])


def _flags(norm, interleaved, q_weight, k_weight):
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("weights belong to the norm")
    return (_lib.CARVE_ROPE_NORM if norm else 0) | (_lib.CARVE_ROPE_INTERLEAVED if interleaved else 0)


def _rope_call(what, q, k, cos, sin, positions, q_weight, k_weight, norm, eps, interleaved):
    dt, dev = _first(q, "q", what)
    sq, sk = q.shape, k.shape
    lead, d = sq[:-2], sq[-1]
    if sk[:-2] != lead or sk[-1] != d:
        raise ValueError(f"k: expected shape {(*lead, 'heads', d)}, got {tuple(sk)}")
    pc, ps, rot, table_len = _angles(cos, sin, dev)
    c = _lib.CarveRopeConfig(math.prod(lead), _rows(q, "q", sq, dt, dev), _rows(k, "k", sk, dt, dev), 0, 0, 0, 0,
                             lead[-1] or 1, sq[-2], sk[-2], d, rot, table_len, _DTYPES[dt],
                             _flags(norm, interleaved, q_weight, k_weight), eps)
    args = (q.data_ptr(), k.data_ptr(), _flat(q_weight, "q_weight", (d,), dt, dev),
            _flat(k_weight, "k_weight", (d,), dt, dev), pc, ps, _flat(positions, "positions", lead, _I32, dev))
    return c, args, sq, sk, dt, dev


def qk_norm_rope_fwd(q, k, cos=None, sin=None, positions=None, q_weight=None, k_weight=None, norm=True, eps=1e-6,
                     interleaved=False, q_out=None, k_out=None, stream=None):
    """Norm and rotation of queries and keys in one pass: y = R(p) (x / sqrt(mean(x^2) + eps) * weight) for
    each head x. Shapes: q [..., Hq, d], k [..., Hk, d] with equal leading (token) dimensions; weights [d] in the
    input dtype; cos, sin [P, rot / 2] fp32 (see rope_tables; rot is a multiple of 16 up to d, None for no
    rotation); positions int32 over the token dimensions (None: the index in the last of them). A position
    outside the table gives NaN. norm=False leaves the norm out. q_out, k_out may be q and k themselves.
    Returns (q_out, k_out)."""
    c, args, sq, sk, dt, dev = _rope_call("qk_norm_rope_fwd", q, k, cos, sin, positions, q_weight, k_weight, norm,
                                          eps, interleaved)
    with _on(dev, stream):
        q_out = _dense(q) if q_out is None else q_out
        k_out = _dense(k) if k_out is None else k_out
        c.qo_row, c.ko_row = _rows(q_out, "q_out", sq, dt, dev), _rows(k_out, "k_out", sk, dt, dev)
        code = _lib.lib().carve_qk_norm_rope_fwd(c, *args, q_out.data_ptr(), k_out.data_ptr(),
                                                 torch._C._cuda_getCurrentRawStream(dev.index))
    if code:
        _lib.check(code)
    return q_out, k_out


def qk_norm_rope_bwd(q, k, d_q_out, d_k_out, cos=None, sin=None, positions=None, q_weight=None, k_weight=None,
                     norm=True, eps=1e-6, interleaved=False, dq=None, dk=None, workspace=None, stream=None):
    """Gradients of qk_norm_rope_fwd's q, k and weights from those of its outputs; the other arguments as given to
    the forward pass. dq may be d_q_out or q itself, dk likewise. Returns a dict with dq, dk (input dtype) and
    dq_weight, dk_weight (fp32, None without the weight)."""
    c, args, sq, sk, dt, dev = _rope_call("qk_norm_rope_bwd", q, k, cos, sin, positions, q_weight, k_weight, norm,
                                          eps, interleaved)
    c.qo_row, c.ko_row = _rows(d_q_out, "d_q_out", sq, dt, dev), _rows(d_k_out, "d_k_out", sk, dt, dev)
    L = _lib.lib()
    with _on(dev, stream):
        dq = _dense(q) if dq is None else dq
        dk = _dense(k) if dk is None else dk
        c.dq_row, c.dk_row = _rows(dq, "dq", sq, dt, dev), _rows(dk, "dk", sk, dt, dev)
        dqw = None if q_weight is None else torch.empty_like(q_weight, dtype=torch.float32)
        dkw = None if k_weight is None else torch.empty_like(k_weight, dtype=torch.float32)
        need = ctypes.c_int64()
        code = L.carve_qk_norm_rope_workspace(c, dqw is not None or dkw is not None, need)
        if code:
            _lib.check(code)
        workspace, ws = _workspace(workspace, need.value, dev)
        code = L.carve_qk_norm_rope_bwd(
            c, *args, d_q_out.data_ptr(), d_k_out.data_ptr(), dq.data_ptr(), dk.data_ptr(),
            None if dqw is None else dqw.data_ptr(), None if dkw is None else dkw.data_ptr(), ws, need.value,
            torch._C._cuda_getCurrentRawStream(dev.index))
    if code:
        _lib.check(code)
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _workspace(given, need, dev):
    if not need:
        return None, None
    if given is None:
        given = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        if given.device != dev or not given.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on {dev}")
        if given.numel() * given.element_size() < need:
            raise ValueError(f"workspace: {need} bytes are needed, got {given.numel() * given.element_size()}")
    return given, given.data_ptr()


def _caches(k_cache, v_cache, Hk, d, dt, dev):
    shape = k_cache.shape
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dim() != 4 or t.shape[2] != Hk or t.shape[3] != d:
            raise ValueError(f"{name}: expected [pages, page_size, {Hk}, {d}], got {tuple(t.shape)}")
        if t.dtype is not dt or t.device != dev:
            _like(t, name, dt, dev)
        if t.stride(3) != 1:
            raise ValueError(f"{name}: the channels of a head must be contiguous")
    if v_cache.shape != shape:
        raise ValueError(f"v_cache: expected shape {tuple(shape)}, got {tuple(v_cache.shape)}")
    return shape, k_cache.stride(), v_cache.stride()


def _sequences(block_table, kv_lens, cu_seqlens, N, dev):
    """(S, table width, elements between its rows, flags, addresses of cu_seqlens, kv_lens and the table)."""
    if block_table.dim() != 2:
        raise ValueError(f"block_table: expected [sequences, pages each], got {tuple(block_table.shape)}")
    S, width = block_table.shape
    if S > _MOST or width > _MOST or N > _MOST:
        raise ValueError(f"sizes past 32 bits: {N} tokens, a block_table of {tuple(block_table.shape)}")
    row, step = block_table.stride()
    if block_table.dtype is not _I32 or block_table.device != dev:
        _like(block_table, "block_table", _I32, dev)
    if width > 1 and step != 1:
        raise ValueError("block_table: a sequence's entries must be contiguous")
    if cu_seqlens is None and N != S:
        raise ValueError(f"without cu_seqlens every sequence has one new token: {N} tokens, {S} sequences")
    return (S, width, row if S > 1 else width, _lib.CARVE_PAGED_STEP if cu_seqlens is None else 0,
            _flat(cu_seqlens, "cu_seqlens", (S + 1,), _I32, dev), _flat(kv_lens, "kv_lens", (S,), _I32, dev),
            block_table.data_ptr())


def _window(n):
    """A window as the library takes it: beyond 32 bits it hides nothing that one of 32 bits shows."""
    return max(-1, min(n, _MOST))


def paged_append(k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None, cos=None, sin=None, q=None,
                 q_weight=None, k_weight=None, norm=False, eps=1e-6, interleaved=False, q_out=None, stream=None):
    """Stores new tokens in a paged cache, their keys (and q, where given) normed and rotated on the way as by
    qk_norm_rope_fwd, at their own positions. Shapes: k, v [N, Hk, d], packed sequence after sequence; caches
    [pages, page_size, Hk, d], page_size a power of two; block_table int32 [S, pages each]; kv_lens int32 [S], the
    lengths with the new tokens counted; cu_seqlens int32 [S + 1], where each sequence's new tokens start (None:
    one each); q [N, Hq, d], q_out may be q itself. No two entries of the caches may overlap. A token whose position
    is negative or past its table, or whose page number is not in [0, pages), is not stored; tokens behind
    cu_seqlens[S] are left alone. Returns q_out (None without q)."""
    dt, dev = _first(k, "k", "paged_append")
    sk = k.shape
    if len(sk) != 3:
        raise ValueError(f"k: expected [tokens, heads, d], got {tuple(sk)}")
    N, Hk, d = sk
    cache, ks, vs = _caches(k_cache, v_cache, Hk, d, dt, dev)
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
        c = _lib.CarvePagedConfig(N, S, Hq, Hk, d, cache[1], cache[0], width, rot, table_len, 0, _DTYPES[dt], flags,
                                  eps, 1.0, q_row, _rows(k, "k", sk, dt, dev), _rows(v, "v", sk, dt, dev), o_row,
                                  table_row, *ks[:3], *vs[:3])
        code = _lib.lib().carve_paged_append(c, k.data_ptr(), v.data_ptr(), pq, wq, wk, pc, ps, cu, lens, table,
                                             k_cache.data_ptr(), v_cache.data_ptr(), po,
                                             torch._C._cuda_getCurrentRawStream(dev.index))
    if code:
        _lib.check(code)
    return q_out


def paged_attention(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None, scale=None, window=0, out=None,
                    return_lse=False, workspace=None, stream=None):
    """Causal attention of new tokens over a paged cache that holds them already (see paged_append for the cache
    and the lengths). q [N, Hq, d], Hq a multiple of the cache's heads (query head h reads head h // (Hq / Hk)). A
    token at position p sees the keys j <= p and, with a window, j > p - window. scale: 1 / sqrt(d) when None.
    A token that sees no key has o = 0 and lse = -inf; tokens behind cu_seqlens[S] are left as they were in `out`.
    One kernel serves the call: a long prompt chunk beside many single tokens is faster in a call of its own.
    workspace: device scratch to use (paged_workspace_bytes of it); allocated when None. Returns o [N, Hq, d], and
    lse [N, Hq] fp32 when return_lse."""
    dt, dev = _first(q, "q", "paged_attention")
    sq = q.shape
    if len(sq) != 3:
        raise ValueError(f"q: expected [tokens, heads, d], got {tuple(sq)}")
    N, Hq, d = sq
    Hk = k_cache.shape[2] if k_cache.dim() == 4 else 0
    cache, ks, vs = _caches(k_cache, v_cache, Hk, d, dt, dev)
    S, width, table_row, step, cu, lens, table = _sequences(block_table, kv_lens, cu_seqlens, N, dev)
    L = _lib.lib()
    lse = pl = None
    with _on(dev, stream):
        out = _dense(q) if out is None else out
        c = _lib.CarvePagedConfig(N, S, Hq, Hk, d, cache[1], cache[0], width, 0, 0, _window(window), _DTYPES[dt],
                                  step, 0.0, d ** -0.5 if scale is None else scale, _rows(q, "q", sq, dt, dev), 0, 0,
                                  _rows(out, "out", sq, dt, dev), table_row, *ks[:3], *vs[:3])
        if return_lse:
            lse = torch.empty((N, Hq), dtype=torch.float32, device=dev)
            pl = lse.data_ptr()
        need = ctypes.c_int64()
        code = L.carve_paged_workspace(c, need)
        if code:
            _lib.check(code)
        workspace, ws = _workspace(workspace, need.value, dev)
        code = L.carve_paged_attention(c, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), cu, lens, table,
                                       out.data_ptr(), pl, ws, need.value,
                                       torch._C._cuda_getCurrentRawStream(dev.index))
    if code:
        _lib.check(code)
    return (out, lse) if return_lse else out


def paged_workspace_bytes(N, S, Hq, Hk, d, page_size, width, dtype=torch.bfloat16, window=0, step=False):
    """Bytes of workspace paged_attention needs for N new tokens of S sequences (step: one each) with a block table
    `width` pages wide."""
    for name, n in (("N", N), ("S", S), ("Hq", Hq), ("Hk", Hk), ("d", d), ("page_size", page_size), ("width", width)):
        if not 0 <= n <= _MOST:
            raise ValueError(f"{name}: expected a size of 32 bits, got {n}")
    c = _lib.CarvePagedConfig()
    c.N, c.S, c.Hq, c.Hk, c.d, c.page_size, c.pages, c.width = N, S, Hq, Hk, d, page_size, 1, width
    c.window, c.dtype, c.scale = _window(window), _DTYPES[dtype], 1.0
    c.flags = _lib.CARVE_PAGED_STEP if step else 0
    c.table_row = width
    c.kc_page = c.kc_tok = c.kc_head = c.vc_page = c.vc_tok = c.vc_head = d
    need = ctypes.c_int64()
    _lib.check(_lib.lib().carve_paged_workspace(c, need))
    return need.value
