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
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    _like(t, name, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _rows(t, name, lead, H, d, dtype, device):
    """Elements from one token of t [*lead, H, d] to the next."""
    shape, stride = t.shape, t.stride()
    if tuple(shape) != (*lead, H, d):
        raise ValueError(f"{name}: expected shape {(*lead, H, d)}, got {tuple(shape)}")
    _like(t, name, dtype, device)
    if t.numel() == 0:
        return H * d
    if stride[-1] != 1 or (H > 1 and stride[-2] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    row, size = None, 1                  # the token dimensions must step evenly
    for n, s in zip(reversed(lead), reversed(stride[:-2])):
        if n == 1:
            continue
        if row is None:
            row = s
        elif s != row * size:
            raise ValueError(f"{name}: tokens must be evenly spaced")
        size *= n
    return H * d if row is None else row


class _Call:
    """Stream and device of one call: temporaries belong to the stream that the kernels run on, and the
    tensors' device is current for the launch."""

    def __init__(self, device, stream):
        self.device, self.given = device, stream

    def __enter__(self):
        dev = self.device
        self.stack = None
        if torch.cuda.current_device() != dev.index:
            self.stack = contextlib.ExitStack()
            self.stack.enter_context(torch.cuda.device(dev))
        if self.given is None:
            self.stream = torch.cuda.current_stream(dev).cuda_stream
        else:
            self.stream = self.given.cuda_stream if isinstance(self.given, torch.cuda.Stream) else int(self.given)
            if self.stream != torch.cuda.current_stream(dev).cuda_stream:
                self.stack = self.stack or contextlib.ExitStack()
                self.stack.enter_context(torch.cuda.stream(torch.cuda.ExternalStream(self.stream, device=dev)))
        return self

    def __exit__(self, *exc):
        if self.stack is not None:
            self.stack.close()
        return False


def _first(t, name, what):
    if t.device.type != "cuda":
        raise ValueError(f"{what} runs on the GPU only; move the inputs to a cuda device")
    if t.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {t.dtype}")
    if t.dim() < 3:
        raise ValueError(f"{name}: expected [..., heads, d], got {tuple(t.shape)}")
    return t.dtype, t.device


def _angles(cos, sin, device):
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is None:
        return None, None, 0, 0
    if cos.dim() != 2:
        raise ValueError(f"cos: expected [positions, rot / 2], got {tuple(cos.shape)}")
    return (_flat(cos, "cos", cos.shape, torch.float32, device), _flat(sin, "sin", cos.shape, torch.float32, device),
            2 * cos.shape[1], cos.shape[0])


def _rope_call(what, q, k, cos, sin, positions, q_weight, k_weight, norm, eps, interleaved):
    dt, dev = _first(q, "q", what)
    lead, Hq, d = tuple(q.shape[:-2]), q.shape[-2], q.shape[-1]
    Hk = k.shape[-2] if k.dim() >= 2 else -1
    c = _lib.CarveRopeConfig()
    c.q_row, c.k_row = _rows(q, "q", lead, Hq, d, dt, dev), _rows(k, "k", lead, Hk, d, dt, dev)
    c.N, c.T, c.Hq, c.Hk, c.d = math.prod(lead), max(lead[-1], 1), Hq, Hk, d
    pc, ps, c.rot, c.table_len = _angles(cos, sin, dev)
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("weights belong to the norm")
    c.dtype = _DTYPES[dt]
    c.flags = (_lib.CARVE_ROPE_NORM if norm else 0) | (_lib.CARVE_ROPE_INTERLEAVED if interleaved else 0)
    c.eps = eps
    args = (q.data_ptr(), k.data_ptr(), _flat(q_weight, "q_weight", (d,), dt, dev),
            _flat(k_weight, "k_weight", (d,), dt, dev), pc, ps, _flat(positions, "positions", lead, _I32, dev))
    return c, args, lead, Hq, Hk, d, dt, dev


def qk_norm_rope_fwd(q, k, cos=None, sin=None, positions=None, q_weight=None, k_weight=None, norm=True, eps=1e-6,
                     interleaved=False, q_out=None, k_out=None, stream=None):
    """Norm and rotation of queries and keys in one pass: y = R(p) (x / sqrt(mean(x^2) + eps) * weight) for
    each head x. Shapes: q [..., Hq, d], k [..., Hk, d] with equal leading (token) dimensions; weights [d] in the
    input dtype; cos, sin [P, rot / 2] fp32 (see rope_tables; rot is a multiple of 16 up to d, None for no
    rotation); positions int32 over the token dimensions (None: the index in the last of them). A position
    outside the table gives NaN. norm=False leaves the norm out. q_out, k_out may be q and k themselves.
    Returns (q_out, k_out)."""
    c, args, lead, Hq, Hk, d, dt, dev = _rope_call("qk_norm_rope_fwd", q, k, cos, sin, positions, q_weight, k_weight,
                                                   norm, eps, interleaved)
    with _Call(dev, stream) as call:
        if q_out is None:
            q_out = torch.empty((*lead, Hq, d), dtype=dt, device=dev)
        if k_out is None:
            k_out = torch.empty((*lead, Hk, d), dtype=dt, device=dev)
        c.qo_row, c.ko_row = (_rows(q_out, "q_out", lead, Hq, d, dt, dev), _rows(k_out, "k_out", lead, Hk, d, dt, dev))
        _lib.check(_lib.lib().carve_qk_norm_rope_fwd(ctypes.byref(c), *args, q_out.data_ptr(), k_out.data_ptr(),
                                                     call.stream))
    return q_out, k_out


def qk_norm_rope_bwd(q, k, d_q_out, d_k_out, cos=None, sin=None, positions=None, q_weight=None, k_weight=None,
                     norm=True, eps=1e-6, interleaved=False, dq=None, dk=None, workspace=None, stream=None):
    """Gradients of qk_norm_rope_fwd's q, k and weights from those of its outputs; the other arguments as given to
    the forward pass. dq may be d_q_out or q itself, dk likewise. Returns a dict with dq, dk (input dtype) and
    dq_weight, dk_weight (fp32, None without the weight)."""
    c, args, lead, Hq, Hk, d, dt, dev = _rope_call("qk_norm_rope_bwd", q, k, cos, sin, positions, q_weight, k_weight,
                                                   norm, eps, interleaved)
    c.qo_row, c.ko_row = (_rows(d_q_out, "d_q_out", lead, Hq, d, dt, dev),
                          _rows(d_k_out, "d_k_out", lead, Hk, d, dt, dev))
    with _Call(dev, stream) as call:
        if dq is None:
            dq = torch.empty((*lead, Hq, d), dtype=dt, device=dev)
        if dk is None:
            dk = torch.empty((*lead, Hk, d), dtype=dt, device=dev)
        c.dq_row, c.dk_row = _rows(dq, "dq", lead, Hq, d, dt, dev), _rows(dk, "dk", lead, Hk, d, dt, dev)
        dqw = torch.empty(d, dtype=torch.float32, device=dev) if q_weight is not None else None
        dkw = torch.empty(d, dtype=torch.float32, device=dev) if k_weight is not None else None
        need = ctypes.c_int64()
        _lib.check(_lib.lib().carve_qk_norm_rope_workspace(ctypes.byref(c), int(dqw is not None or dkw is not None),
                                                           ctypes.byref(need)))
        workspace, ws = _workspace(workspace, need.value, dev)
        _lib.check(_lib.lib().carve_qk_norm_rope_bwd(
            ctypes.byref(c), *args, d_q_out.data_ptr(), d_k_out.data_ptr(), dq.data_ptr(), dk.data_ptr(),
            None if dqw is None else dqw.data_ptr(), None if dkw is None else dkw.data_ptr(), ws, need.value,
            call.stream))
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


def _paged_call(N, Hq, Hk, d, k_cache, v_cache, block_table, kv_lens, cu_seqlens, dt, dev):
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dim() != 4 or t.shape[2] != Hk or t.shape[3] != d:
            raise ValueError(f"{name}: expected [pages, page_size, {Hk}, {d}], got {tuple(t.shape)}")
        _like(t, name, dt, dev)
        if t.stride(3) != 1:
            raise ValueError(f"{name}: the channels of a head must be contiguous")
    if v_cache.shape != k_cache.shape:
        raise ValueError(f"v_cache: expected shape {tuple(k_cache.shape)}, got {tuple(v_cache.shape)}")
    if block_table.dim() != 2:
        raise ValueError(f"block_table: expected [sequences, pages each], got {tuple(block_table.shape)}")
    _like(block_table, "block_table", _I32, dev)
    S, width = block_table.shape
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table: a sequence's entries must be contiguous")
    c = _lib.CarvePagedConfig()
    c.N, c.S, c.Hq, c.Hk, c.d = N, S, Hq, Hk, d
    c.pages, c.page_size = k_cache.shape[0], k_cache.shape[1]
    c.width, c.table_row = width, block_table.stride(0) if S > 1 else width
    c.kc_page, c.kc_tok, c.kc_head = k_cache.stride()[:3]
    c.vc_page, c.vc_tok, c.vc_head = v_cache.stride()[:3]
    c.dtype = _DTYPES[dt]
    c.scale = 1.0
    if cu_seqlens is None:
        if N != S:
            raise ValueError(f"without cu_seqlens every sequence has one new token: {N} tokens, {S} sequences")
        c.flags = _lib.CARVE_PAGED_STEP
    return (c, _flat(cu_seqlens, "cu_seqlens", (S + 1,), _I32, dev), _flat(kv_lens, "kv_lens", (S,), _I32, dev),
            block_table.data_ptr())


def paged_append(k, v, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None, cos=None, sin=None, q=None,
                 q_weight=None, k_weight=None, norm=False, eps=1e-6, interleaved=False, q_out=None, stream=None):
    """Stores new tokens in a paged cache, their keys (and q, where given) normed and rotated on the way as by
    qk_norm_rope_fwd, at their own positions. Shapes: k, v [N, Hk, d], packed sequence after sequence; caches
    [pages, page_size, Hk, d], page_size a power of two; block_table int32 [S, pages each]; kv_lens int32 [S], the
    lengths with the new tokens counted; cu_seqlens int32 [S + 1], where each sequence's new tokens start (None:
    one each); q [N, Hq, d], q_out may be q itself. A token whose position is negative or past its table, or whose
    page number is not in [0, pages), is not stored; tokens behind cu_seqlens[S] are left alone. Returns q_out
    (None without q)."""
    dt, dev = _first(k, "k", "paged_append")
    N, Hk, d = k.shape[0], k.shape[-2], k.shape[-1]
    Hq = 0 if q is None else q.shape[-2]
    c, cu, lens, table = _paged_call(N, Hq, Hk, d, k_cache, v_cache, block_table, kv_lens, cu_seqlens, dt, dev)
    c.k_row, c.v_row = _rows(k, "k", (N,), Hk, d, dt, dev), _rows(v, "v", (N,), Hk, d, dt, dev)
    pc, ps, c.rot, c.table_len = _angles(cos, sin, dev)
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("weights belong to the norm")
    if q is None and (q_weight is not None or q_out is not None):
        raise ValueError("q_weight and q_out belong to q")
    c.flags |= (_lib.CARVE_ROPE_NORM if norm else 0) | (_lib.CARVE_ROPE_INTERLEAVED if interleaved else 0)
    c.eps = eps
    wq, wk = _flat(q_weight, "q_weight", (d,), dt, dev), _flat(k_weight, "k_weight", (d,), dt, dev)
    with _Call(dev, stream) as call:
        if q is not None:
            c.q_row = _rows(q, "q", (N,), Hq, d, dt, dev)
            if q_out is None:
                q_out = torch.empty((N, Hq, d), dtype=dt, device=dev)
            c.o_row = _rows(q_out, "q_out", (N,), Hq, d, dt, dev)
        _lib.check(_lib.lib().carve_paged_append(
            ctypes.byref(c), k.data_ptr(), v.data_ptr(), None if q is None else q.data_ptr(), wq, wk, pc, ps, cu, lens,
            table, k_cache.data_ptr(), v_cache.data_ptr(), None if q is None else q_out.data_ptr(), call.stream))
    return q_out


def paged_attention(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens=None, scale=None, window=0, out=None,
                    return_lse=False, workspace=None, stream=None):
    """Causal attention of new tokens over a paged cache that holds them already (see paged_append for the cache
    and the lengths). q [N, Hq, d], Hq a multiple of the cache's heads (query head h reads head h // (Hq / Hk)). A
    token at position p sees the keys j <= p and, with a window, j > p - window. scale: 1 / sqrt(d) when None.
    A token that sees no key has o = 0 and lse = -inf; tokens behind cu_seqlens[S] are left as they were in `out`.
    workspace: device scratch to use (paged_workspace_bytes of it); allocated when None. Returns o [N, Hq, d], and
    lse [N, Hq] fp32 when return_lse."""
    dt, dev = _first(q, "q", "paged_attention")
    N, Hq, d = q.shape[0], q.shape[-2], q.shape[-1]
    Hk = k_cache.shape[2] if k_cache.dim() == 4 else 0
    c, cu, lens, table = _paged_call(N, Hq, Hk, d, k_cache, v_cache, block_table, kv_lens, cu_seqlens, dt, dev)
    c.q_row = _rows(q, "q", (N,), Hq, d, dt, dev)
    c.scale = d ** -0.5 if scale is None else scale
    c.window = window
    L = _lib.lib()
    with _Call(dev, stream) as call:
        if out is None:
            out = torch.empty((N, Hq, d), dtype=dt, device=dev)
        c.o_row = _rows(out, "out", (N,), Hq, d, dt, dev)
        lse = torch.empty((N, Hq), dtype=torch.float32, device=dev) if return_lse else None
        need = ctypes.c_int64()
        _lib.check(L.carve_paged_workspace(ctypes.byref(c), ctypes.byref(need)))
        workspace, ws = _workspace(workspace, need.value, dev)
        _lib.check(L.carve_paged_attention(
            ctypes.byref(c), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), cu, lens, table, out.data_ptr(),
            None if lse is None else lse.data_ptr(), ws, need.value, call.stream))
    return (out, lse) if return_lse else out


def paged_workspace_bytes(N, S, Hq, Hk, d, page_size, width, dtype=torch.bfloat16, window=0, step=False):
    """Bytes of workspace paged_attention needs for N new tokens of S sequences (step: one each) with a block table
    `width` pages wide."""
    c = _lib.CarvePagedConfig()
    c.N, c.S, c.Hq, c.Hk, c.d, c.page_size, c.pages, c.width = N, S, Hq, Hk, d, page_size, 1, width
    c.window, c.dtype, c.scale = window, _DTYPES[dtype], 1.0
    c.flags = _lib.CARVE_PAGED_STEP if step else 0
    c.table_row = width
    c.kc_page = c.kc_tok = c.kc_head = c.vc_page = c.vc_tok = c.vc_head = d
    need = ctypes.c_int64()
    _lib.check(_lib.lib().carve_paged_workspace(ctypes.byref(c), ctypes.byref(need)))
    return need.value
