"""The attention layer's operators without a GPU: the float64 oracle against closed forms and differences, and the
C ABI's argument checks, which all run before the first HIP call."""
import ctypes
import os

import numpy as np
import pytest

from chunk_gated_delta_carve_amd import _lib
from oracle import attention_oracle as orc

FAKE = 0x10000000            # never dereferenced: validation fails before any use
MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from chunk_gated_delta_carve_amd.build import build_library
        build_library(verbose=False)
    return _lib.lib()


def tables(P, rot):
    ang = np.arange(P)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.cos(ang), np.sin(ang)


# the oracle

@pytest.mark.parametrize("rot,inter", [(0, False), (16, False), (16, True), (32, False), (32, True)])
def test_rotation_keeps_lengths_and_depends_on_distance_alone(rot, inter):
    rng = np.random.default_rng(rot + inter)
    d, P = 32, 40
    cos, sin = tables(P, max(rot, 2))
    q, k = rng.standard_normal((2, 1, d))
    dots = []
    for a, b in ((3, 1), (12, 10), (39, 37)):
        y = orc.norm_rope(q[None], None, cos, sin, np.array([a]), rot, inter, False, 0.0)[0]
        z = orc.norm_rope(k[None], None, cos, sin, np.array([b]), rot, inter, False, 0.0)[0]
        assert np.allclose(np.linalg.norm(y), np.linalg.norm(q), rtol=1e-13)
        dots.append(float(np.sum(y * z)))
    assert np.allclose(dots, dots[0], rtol=1e-12)
    if rot == 0:
        assert np.array_equal(y, q)


def test_rotation_pairs():
    cos, sin = tables(8, 32)
    x = np.zeros((1, 1, 64))
    x[0, 0, 1] = 1.0
    half = orc.norm_rope(x, None, cos, sin, np.array([5]), 32, False, False, 0.0)[0, 0]
    assert np.allclose(half[[1, 17]], [cos[5, 1], sin[5, 1]]) and np.count_nonzero(half) == 2
    near = orc.norm_rope(x, None, cos, sin, np.array([5]), 32, True, False, 0.0)[0, 0]
    assert np.allclose(near[[0, 1]], [-sin[5, 0], cos[5, 0]]) and np.count_nonzero(near) == 2
    assert np.isnan(orc.norm_rope(x, None, cos, sin, np.array([8]), 32, True, False, 0.0)[0, 0, :32]).all()


def test_norm_closed_form():
    x = np.full((1, 1, 16), 3.0)
    y = orc.norm_rope(x, np.arange(16.0), None, None, None, 0, False, True, 0.0)
    assert np.allclose(y[0, 0], np.arange(16.0))


@pytest.mark.parametrize("rot,inter,norm,weighted", [(16, False, True, True), (32, True, True, True),
                                                     (16, True, True, False), (32, False, False, False)])
def test_gradient_against_differences(rot, inter, norm, weighted):
    rng = np.random.default_rng(5)
    T, H, d, eps = 3, 2, 32, 1e-6
    cos, sin = tables(9, rot)
    pos = np.array([0, 4, 8])
    x, dy = rng.standard_normal((2, T, H, d))
    w = rng.standard_normal(d) if weighted else None
    f = lambda x, w: float(np.sum(dy * orc.norm_rope(x, w, cos, sin, pos, rot, inter, norm, eps)))  # noqa: E731
    dx, dw = orc.norm_rope_grad(x, w, dy, cos, sin, pos, rot, inter, norm, eps)
    h = 1e-6          # central differences: error h^2 f''' + 2^-53 f / h, far below 1e-7
    for at in ((0, 0, 0), (1, 1, 7), (2, 0, 31), (1, 0, 16)):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    if weighted:
        for i in (0, 9, 31):
            e = np.zeros(d)
            e[i] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_attention_is_plain_softmax_over_the_gathered_sequence():
    rng = np.random.default_rng(3)
    kv, n, G, Hk, d, page = 13, 5, 2, 2, 16, 4
    kc, vc = rng.standard_normal((2, 7, page, Hk, d))
    table = np.array([[5, 2, 6, 0]])
    q = rng.standard_normal((n, G * Hk, d))
    o, lse, A, reach, keys = orc.paged_attention(q, kc, vc, table, [kv], [0, n], 0.3, 0)
    K, V = (c[table[0]].reshape(-1, Hk, d)[:kv] for c in (kc, vc))
    for i in range(n):
        for h in range(G * Hk):
            x = 0.3 * K[:, h // G] @ q[i, h]
            x[kv - n + i + 1:] = -np.inf
            e = np.exp(x)
            assert np.allclose(o[i, h], e @ V[:, h // G] / e.sum(), rtol=1e-12)
            assert np.isclose(lse[i, h], np.log(e.sum()), rtol=1e-12)
    assert list(keys) == [9, 10, 11, 12, 13]
    o1 = orc.paged_attention(q, kc, vc, table, [kv], [0, n], 0.3, 1)[0]      # a window of one: its own value
    assert np.allclose(o1[2, 3], V[kv - n + 2, 1])


def test_append_then_places():
    rng = np.random.default_rng(4)
    kc = np.zeros((4, 4, 1, 2))
    table = np.array([[3, 1], [0, -1]])
    k = rng.standard_normal((7, 1, 2))
    got, _ = orc.paged_append(k, k, kc, kc, table, [6, 3], [0, 2, 6], 4)
    assert np.array_equal(got[1, 0], k[0]) and np.array_equal(got[1, 1], k[1])   # positions 4, 5
    assert np.array_equal(got[0, :3], k[3:6]) and not got[3].any()               # -1 is dropped, 0, 1, 2 stored


# argument checks

def rope_cfg(**kw):
    base = dict(N=10, T=10, Hq=4, Hk=2, d=64, rot=64, table_len=10, dtype=_lib.CARVE_BF16, flags=_lib.CARVE_ROPE_NORM,
                eps=1e-6)
    base.update(kw)
    lq, lk = base["Hq"] * base["d"], base["Hk"] * base["d"]
    for n, v in (("q_row", lq), ("k_row", lk), ("qo_row", lq), ("ko_row", lk), ("dq_row", lq), ("dk_row", lk)):
        base.setdefault(n, v)
    c = _lib.CarveRopeConfig()
    for n, v in base.items():
        setattr(c, n, v)
    return c


FWD = ("q", "k", "q_weight", "k_weight", "cos", "sin", "positions", "q_out", "k_out")
BWD = ("q", "k", "q_weight", "k_weight", "cos", "sin", "positions", "d_q_out", "d_k_out", "dq", "dk", "dq_weight",
       "dk_weight", "workspace")


def fwd(L, c, **ptr):
    base = {n: FAKE + i * MB for i, n in enumerate(FWD)}
    base.update(ptr)
    return L.carve_qk_norm_rope_fwd(None if c is None else ctypes.byref(c), *(base[n] for n in FWD), None)


def bwd(L, c, ws=None, **ptr):
    base = {n: FAKE + i * MB for i, n in enumerate(BWD)}
    base.update(ptr)
    if ws is None:
        need = ctypes.c_int64()
        ok = c is not None and L.carve_qk_norm_rope_workspace(ctypes.byref(c), 1, ctypes.byref(need)) == 0
        ws = need.value if ok else 0
    return L.carve_qk_norm_rope_bwd(None if c is None else ctypes.byref(c), *(base[n] for n in BWD), ws, None)


BAD_ROPE = [
    (dict(d=96), _lib.CARVE_EUNSUPPORTED), (dict(d=32), _lib.CARVE_EUNSUPPORTED),
    (dict(rot=24), _lib.CARVE_EUNSUPPORTED), (dict(rot=80), _lib.CARVE_EUNSUPPORTED),
    (dict(rot=-16), _lib.CARVE_EINVAL), (dict(N=-1), _lib.CARVE_EINVAL), (dict(Hq=-1), _lib.CARVE_EINVAL),
    (dict(dtype=2), _lib.CARVE_EINVAL), (dict(flags=8), _lib.CARVE_EINVAL),
    (dict(flags=_lib.CARVE_PAGED_STEP), _lib.CARVE_EINVAL), (dict(eps=0.0), _lib.CARVE_EINVAL),
    (dict(eps=float("nan")), _lib.CARVE_EINVAL), (dict(q_row=-256), _lib.CARVE_EINVAL),
    (dict(q_row=260), _lib.CARVE_EALIGN), (dict(k_row=129), _lib.CARVE_EALIGN), (dict(qo_row=252), _lib.CARVE_EALIGN),
    (dict(N=1 << 31), _lib.CARVE_EUNSUPPORTED), (dict(N=1 << 29, Hq=64), _lib.CARVE_EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_ROPE, ids=[str(i) for i in range(len(BAD_ROPE))])
def test_rope_config_refused(L, kw, code):
    assert fwd(L, rope_cfg(**kw)) == code
    assert bwd(L, rope_cfg(**kw)) == code


def test_rope_arguments_refused(L):
    c = rope_cfg()
    assert fwd(L, None) == _lib.CARVE_EINVAL and bwd(L, None) == _lib.CARVE_EINVAL
    for n in ("q", "k", "cos", "sin", "q_out", "k_out"):
        assert fwd(L, c, **{n: None}) == _lib.CARVE_EINVAL, n
    for n in ("q", "k", "cos", "d_q_out", "d_k_out", "dq", "dk", "dq_weight", "dk_weight", "workspace"):
        assert bwd(L, c, **{n: None}) == _lib.CARVE_EINVAL, n
    for n in FWD:
        assert fwd(L, c, **{n: FAKE + 9 * MB + (2 if n == "positions" else 8)}) == _lib.CARVE_EALIGN, n
    assert fwd(L, rope_cfg(T=0), positions=None) == _lib.CARVE_EINVAL
    assert fwd(L, rope_cfg(flags=0)) == _lib.CARVE_EINVAL                    # weights without the norm
    assert fwd(L, c, q_out=FAKE + 16) == _lib.CARVE_EINVAL                   # a shifted view of q
    assert fwd(L, c, q_out=FAKE + MB) == _lib.CARVE_EINVAL                   # over k
    assert fwd(L, c, k_out=FAKE + 7 * MB) == _lib.CARVE_EINVAL               # over q_out
    assert fwd(L, c, q_out=FAKE + 4 * MB) == _lib.CARVE_EINVAL               # over cos
    assert fwd(L, rope_cfg(qo_row=128)) == _lib.CARVE_EINVAL                 # output tokens on top of each other
    # the two parts of one projection's output interleave without overlapping, one channel further they overlap
    part = dict(q_row=384, k_row=384, qo_row=384, ko_row=384)
    assert fwd(L, rope_cfg(**part), q=FAKE, k=FAKE + 512, q_out=FAKE + 16, k_out=FAKE + 512) == _lib.CARVE_EINVAL
    assert fwd(L, rope_cfg(**part), q=FAKE, k=FAKE + 496, q_out=FAKE, k_out=FAKE + 496) == _lib.CARVE_EINVAL
    need = ctypes.c_int64()
    assert L.carve_qk_norm_rope_workspace(ctypes.byref(c), 1, ctypes.byref(need)) == _lib.CARVE_OK and need.value > 0
    assert bwd(L, c, ws=need.value - 4) == _lib.CARVE_EWORKSPACE
    assert L.carve_qk_norm_rope_workspace(ctypes.byref(c), 0, ctypes.byref(need)) == _lib.CARVE_OK and need.value == 0
    assert L.carve_qk_norm_rope_workspace(ctypes.byref(c), 1, None) == _lib.CARVE_EINVAL
    assert bwd(L, c, dq=FAKE + 8 * MB) == _lib.CARVE_EINVAL                  # over d_k_out
    assert bwd(L, c, dq=FAKE + 7 * MB + 16) == _lib.CARVE_EINVAL             # a shifted view of d_q_out
    assert bwd(L, c, dk=FAKE + 13 * MB) == _lib.CARVE_EINVAL                 # in the workspace
    # nothing to do: no HIP call
    assert fwd(L, rope_cfg(N=0)) == _lib.CARVE_OK
    assert fwd(L, rope_cfg(Hq=0, Hk=0)) == _lib.CARVE_OK
    assert bwd(L, rope_cfg(N=0, flags=0), q_weight=None, k_weight=None) == _lib.CARVE_OK


def paged_cfg(**kw):
    base = dict(N=20, S=3, Hq=4, Hk=2, d=64, page_size=16, pages=12, width=4, rot=64, table_len=64, window=0,
                dtype=_lib.CARVE_BF16, flags=_lib.CARVE_ROPE_NORM, eps=1e-6, scale=0.125)
    base.update(kw)
    lq, lk, d = base["Hq"] * base["d"], base["Hk"] * base["d"], base["d"]
    for n, v in (("q_row", lq), ("k_row", lk), ("v_row", lk), ("o_row", lq), ("table_row", base["width"]),
                 ("kc_page", lk * base["page_size"]), ("kc_tok", lk), ("kc_head", d),
                 ("vc_page", lk * base["page_size"]), ("vc_tok", lk), ("vc_head", d)):
        base.setdefault(n, v)
    c = _lib.CarvePagedConfig()
    for n, v in base.items():
        setattr(c, n, v)
    return c


APP = ("k", "v", "q", "q_weight", "k_weight", "cos", "sin", "cu", "kv_lens", "table", "k_cache", "v_cache", "q_out")
ATT = ("q", "k_cache", "v_cache", "cu", "kv_lens", "table", "o", "lse", "workspace")


def append(L, c, **ptr):
    base = {n: FAKE + i * MB for i, n in enumerate(APP)}
    base.update(ptr)
    return L.carve_paged_append(None if c is None else ctypes.byref(c), *(base[n] for n in APP), None)


def attention(L, c, ws=None, **ptr):
    base = {n: FAKE + i * 64 * MB for i, n in enumerate(ATT)}
    base.update(ptr)
    if ws is None:
        need = ctypes.c_int64()
        ok = c is not None and L.carve_paged_workspace(ctypes.byref(c), ctypes.byref(need)) == 0
        ws = need.value if ok else 0
    return L.carve_paged_attention(None if c is None else ctypes.byref(c), *(base[n] for n in ATT), ws, None)


BAD_PAGED = [
    (dict(d=96), _lib.CARVE_EUNSUPPORTED), (dict(page_size=24), _lib.CARVE_EUNSUPPORTED),
    (dict(page_size=0), _lib.CARVE_EINVAL), (dict(page_size=-16), _lib.CARVE_EINVAL),
    (dict(N=-1), _lib.CARVE_EINVAL), (dict(S=-1), _lib.CARVE_EINVAL), (dict(width=-1), _lib.CARVE_EINVAL),
    (dict(pages=-1), _lib.CARVE_EINVAL), (dict(window=-1), _lib.CARVE_EINVAL), (dict(dtype=5), _lib.CARVE_EINVAL),
    (dict(flags=16), _lib.CARVE_EINVAL), (dict(flags=_lib.CARVE_PAGED_STEP), _lib.CARVE_EINVAL),   # N != S
    (dict(width=1 << 27), _lib.CARVE_EUNSUPPORTED), (dict(table_row=3), _lib.CARVE_EINVAL),
    (dict(kc_tok=32), _lib.CARVE_EINVAL), (dict(vc_page=0), _lib.CARVE_EINVAL), (dict(kc_head=-64), _lib.CARVE_EINVAL),
    (dict(kc_tok=132), _lib.CARVE_EALIGN), (dict(vc_head=68), _lib.CARVE_EALIGN), (dict(q_row=260), _lib.CARVE_EALIGN),
    (dict(q_row=-256), _lib.CARVE_EINVAL), (dict(o_row=128), _lib.CARVE_EINVAL),
    (dict(N=1 << 30, Hq=4, Hk=2), _lib.CARVE_EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_PAGED, ids=[str(i) for i in range(len(BAD_PAGED))])
def test_paged_config_refused(L, kw, code):
    assert append(L, paged_cfg(**kw)) == code
    assert attention(L, paged_cfg(**kw)) == code


def test_append_arguments_refused(L):
    c = paged_cfg()
    assert append(L, None) == _lib.CARVE_EINVAL
    for n in ("k", "v", "q", "q_out", "cos", "sin", "cu", "kv_lens", "table", "k_cache", "v_cache"):
        assert append(L, c, **{n: None}) == _lib.CARVE_EINVAL, n
    for n in ("k", "v", "q", "q_weight", "k_weight", "cos", "sin", "k_cache", "v_cache", "q_out"):
        assert append(L, c, **{n: FAKE + 20 * MB + 8}) == _lib.CARVE_EALIGN, n
    for n in ("cu", "kv_lens", "table"):
        assert append(L, c, **{n: FAKE + 20 * MB + 2}) == _lib.CARVE_EALIGN, n
    assert append(L, paged_cfg(rot=8)) == _lib.CARVE_EUNSUPPORTED
    assert append(L, paged_cfg(eps=0.0)) == _lib.CARVE_EINVAL
    assert append(L, paged_cfg(flags=0)) == _lib.CARVE_EINVAL                  # weights without the norm
    assert append(L, c, q_out=FAKE) == _lib.CARVE_EINVAL                       # over k
    assert append(L, c, q_out=FAKE + 2 * MB + 16) == _lib.CARVE_EINVAL         # a shifted view of q
    assert append(L, c, q_out=FAKE + 9 * MB) == _lib.CARVE_EINVAL              # over the table
    assert append(L, c, k=FAKE + 10 * MB + 4096) == _lib.CARVE_EINVAL          # inside the cache
    assert append(L, c, v_cache=FAKE + 10 * MB) == _lib.CARVE_EINVAL           # both caches the same
    assert append(L, paged_cfg(N=0)) == _lib.CARVE_OK
    assert append(L, paged_cfg(S=0)) == _lib.CARVE_OK


def test_attention_arguments_refused(L):
    c = paged_cfg()
    assert attention(L, None) == _lib.CARVE_EINVAL
    for n in ("q", "o", "cu", "kv_lens", "table", "k_cache", "v_cache"):
        assert attention(L, c, **{n: None}) == _lib.CARVE_EINVAL, n
    for n in ("q", "k_cache", "v_cache", "o", "workspace"):
        assert attention(L, c, **{n: FAKE + 900 * MB + 8}) == _lib.CARVE_EALIGN, n
    for n in ("cu", "kv_lens", "table", "lse"):
        assert attention(L, c, **{n: FAKE + 900 * MB + 2}) == _lib.CARVE_EALIGN, n
    for s in (0.0, -0.1, float("nan")):
        assert attention(L, paged_cfg(scale=s)) == _lib.CARVE_EINVAL
    assert attention(L, paged_cfg(scale=17.0)) == _lib.CARVE_EUNSUPPORTED
    assert attention(L, paged_cfg(Hq=5)) == _lib.CARVE_EINVAL                  # not a multiple of Hk
    assert attention(L, paged_cfg(Hk=0)) == _lib.CARVE_EINVAL
    assert attention(L, paged_cfg(pages=0)) == _lib.CARVE_EINVAL
    assert attention(L, c, o=FAKE) == _lib.CARVE_EINVAL                        # over q
    assert attention(L, c, o=FAKE + 64 * MB + 4096) == _lib.CARVE_EINVAL       # in the cache
    assert attention(L, c, lse=FAKE + 6 * 64 * MB) == _lib.CARVE_EINVAL        # over o
    need = ctypes.c_int64()
    assert L.carve_paged_workspace(ctypes.byref(c), None) == _lib.CARVE_EINVAL
    long = paged_cfg(width=4096, pages=4096)
    assert L.carve_paged_workspace(ctypes.byref(long), ctypes.byref(need)) == _lib.CARVE_OK and need.value > 0
    assert attention(L, long, ws=need.value - 4) == _lib.CARVE_EWORKSPACE
    assert attention(L, long, workspace=None) == _lib.CARVE_EINVAL
    assert attention(L, long, workspace=FAKE + 6 * 64 * MB) == _lib.CARVE_EINVAL   # over o
    assert attention(L, paged_cfg(N=0)) == _lib.CARVE_OK
    assert attention(L, paged_cfg(S=0)) == _lib.CARVE_OK
    assert attention(L, paged_cfg(Hq=0)) == _lib.CARVE_OK


def test_paged_workspace_is_bounded(L):
    """Partial results belong to workgroups, not to sequences: a larger batch or a longer table asks for no more
    than fills the GPU, and a call that one workgroup does asks for none."""
    need = ctypes.c_int64()
    size = {}
    for S, width in ((1, 1), (1, 512), (64, 512), (4096, 512), (64, 65536)):
        c = paged_cfg(N=S, S=S, width=width, flags=_lib.CARVE_PAGED_STEP, Hq=1, Hk=1)
        assert L.carve_paged_workspace(ctypes.byref(c), ctypes.byref(need)) == _lib.CARVE_OK
        size[S, width] = need.value
    assert 0 < size[1, 512] <= size[64, 512] == size[4096, 512] == size[64, 65536]
    assert size[64, 512] <= 32 * MB
    # more blocks of keys than 32 bits count
    c = paged_cfg(N=1 << 20, S=1 << 20, width=1 << 26, flags=_lib.CARVE_PAGED_STEP)
    assert L.carve_paged_workspace(ctypes.byref(c), ctypes.byref(need)) == _lib.CARVE_EUNSUPPORTED


def test_sizes_past_the_launches_refused(L):
    """A wave per token in workgroups of four: 2^26 tokens are 2^32 threads, one more than a launch counts. The tile
    kernels' workgroups are counted the same way."""
    most = (1 << 26) - 4
    c = rope_cfg(N=most + 1, Hq=1, Hk=0)
    assert fwd(L, c, k=None, k_out=None) == _lib.CARVE_EUNSUPPORTED
    assert bwd(L, c, k=None, d_k_out=None, dk=None) == _lib.CARVE_EUNSUPPORTED
    assert append(L, paged_cfg(N=most + 1, Hq=0, Hk=1, flags=0), q=None, q_out=None, q_weight=None,
                  k_weight=None) == _lib.CARVE_EUNSUPPORTED
    need = ctypes.c_int64()
    for d, tiles in ((64, (1 << 24) - 1), (128, (1 << 23) - 1)):
        rows = 33                                                    # per sequence: one tile and the numbering's slack
        S = tiles * 128 * (d // 64) // (rows + 128 * (d // 64))
        for more, code in ((0, _lib.CARVE_OK), (S // 50, _lib.CARVE_EUNSUPPORTED)):
            c = paged_cfg(N=(S + more) * rows, S=S + more, Hq=1, Hk=1, d=d)
            assert L.carve_paged_workspace(ctypes.byref(c), ctypes.byref(need)) == code, (d, more)


@pytest.mark.parametrize("name", ["q_row", "k_row", "qo_row", "ko_row", "dq_row", "dk_row"])
def test_far_rope_strides_refused(L, name):
    c = rope_cfg(**{name: 1 << 31})
    assert fwd(L, c) == bwd(L, c) == _lib.CARVE_EUNSUPPORTED


@pytest.mark.parametrize("name", ["q_row", "k_row", "v_row", "o_row", "table_row", "kc_page", "vc_tok"])
def test_far_paged_strides_refused(L, name):
    c = paged_cfg(**{name: 1 << 31})
    assert append(L, c) == attention(L, c) == _lib.CARVE_EUNSUPPORTED


def test_denormal_eps_refused(L):
    """The inverse root takes a denormal as 0, so a row of zeros would come out as NaN."""
    assert fwd(L, rope_cfg(eps=1e-39)) == bwd(L, rope_cfg(eps=1e-39)) == _lib.CARVE_EINVAL
    assert append(L, paged_cfg(eps=1e-39)) == _lib.CARVE_EINVAL
    assert fwd(L, rope_cfg(eps=1.2e-38, N=0)) == _lib.CARVE_OK


def test_append_refuses_caches_whose_entries_overlap(L):
    for kw in (dict(kc_tok=128, kc_head=128), dict(vc_page=1024, vc_tok=128), dict(kc_page=64, kc_tok=768, kc_head=64),
               dict(vc_head=1024)):
        assert append(L, paged_cfg(**kw)) == _lib.CARVE_EINVAL, kw
    # heads before tokens, tokens before pages, and gaps are fine (refused later, for the missing k)
    for kw in (dict(kc_head=1024, kc_tok=64), dict(kc_page=128, kc_tok=12 * 128), dict(vc_page=4096, vc_tok=192)):
        assert append(L, paged_cfg(N=0, **kw)) == _lib.CARVE_OK, kw


def test_sizes_past_32_bits_in_python():
    from chunk_gated_delta_carve_amd import paged_workspace_bytes
    from chunk_gated_delta_carve_amd.attention import _window
    assert [_window(n) for n in (-2**32, -1, 0, 7, 2**31, 2**32 + 5)] == [-1, -1, 0, 7, 2**31 - 1, 2**31 - 1]
    ok = dict(N=64, S=64, Hq=8, Hk=2, d=64, page_size=16, width=256)
    assert paged_workspace_bytes(**ok) > 0
    for name in ok:
        with pytest.raises(ValueError):
            paged_workspace_bytes(**{**ok, name: 2**32 + ok[name]})


def test_the_row_kernels_blocks_fit_32_bits(L):
    """What the host accepts the row kernel counts in 32 bits: an item (16 rows of a key/value head) has the blocks of
    128 keys that its sequence's rows see, and with a window no more than 16 rows can."""
    need = ctypes.c_int64()
    rng = np.random.default_rng(31)
    codes = set()
    cases = [(524288, w, 64) for w in (0, 256, 1024)] + [(1 << 20, 1024, 64), (700000, 1024, 128)]
    cases += [(int(2.0 ** rng.uniform(10, 22)), int(rng.choice([0, 2.0 ** rng.uniform(0, 22)])), 64)
              for _ in range(200)]
    for N, window, page in cases:
        c = paged_cfg(N=N, S=1, Hq=16, Hk=4, page_size=page, pages=N // page + 1, width=N // page + 1, window=window,
                      dtype=_lib.CARVE_F32)
        code = L.carve_paged_workspace(ctypes.byref(c), ctypes.byref(need))
        codes.add(code)
        items, blocks = -(-N * 4 // 16) * 4, -(-N // 128)
        if window:
            blocks = min(blocks, (window + 16 + 128 - 3) // 128 + 1)
        if code == _lib.CARVE_OK:
            assert items * blocks < 2 ** 31, (N, window)
        else:
            assert code == _lib.CARVE_EUNSUPPORTED and items * (blocks + 3) >= 2 ** 31, (N, window)
    assert codes == {_lib.CARVE_OK, _lib.CARVE_EUNSUPPORTED}


def test_tensors_past_32_bits_in_python():
    """Sizes that the library would take modulo 2^32: a table of 2^32 + 4 pages is none of four."""
    torch = pytest.importorskip("torch")
    from chunk_gated_delta_carve_amd.attention import _angles, _sequences
    meta = torch.device("meta")
    ints = lambda *shape: torch.empty(shape, dtype=torch.int32, device=meta)  # noqa: E731
    f32 = lambda *shape: torch.empty(shape, device=meta)  # noqa: E731
    assert _sequences(ints(3, 4), ints(3), ints(4), 9, meta)[:3] == (3, 4, 4)
    for table, lens, cu, N in ((ints(3, 2**32 + 4), ints(3), ints(4), 9), (ints(2**31, 1), ints(2**31), None, 2**31),
                               (ints(3, 4), ints(3), ints(4), 2**32 + 9)):
        with pytest.raises(ValueError):
            _sequences(table, lens, cu, N, meta)
    assert _angles(f32(10, 32), f32(10, 32), meta)[2:] == (64, 10)
    for shape in ((2**32 + 10, 8), (1, 2**31 + 32)):
        with pytest.raises(ValueError):
            _angles(f32(*shape), f32(*shape), meta)


@pytest.mark.parametrize("kw", [
    dict(), dict(kc_page=4096, vc_page=4096), dict(kc_tok=256, vc_tok=256, kc_page=4096, vc_page=4096),
    dict(kc_tok=64, vc_tok=64, kc_head=1024, vc_head=1024), dict(kc_tok=1536, vc_tok=1536, kc_page=128, vc_page=128),
    dict(kc_head=192, vc_head=192, kc_tok=576, vc_tok=576, kc_page=9216, vc_page=9216),
    dict(pages=1, kc_page=0, vc_page=64),
    dict(Hk=1, Hq=4, kc_head=0, vc_head=64, kc_tok=192, vc_tok=192, kc_page=4096, vc_page=4096)],
    ids=[str(i) for i in range(8)])
def test_append_refuses_caches_that_share_channels(L, kw):
    """v_cache at every distance of a step of 16 bytes from k_cache, against the entries themselves: refused where two
    share a channel, and only there (N = 0: nothing is launched)."""
    c = paged_cfg(N=0, **kw)
    at = [(c.pages, c.kc_page), (c.page_size, c.kc_tok), (c.Hk, c.kc_head)]
    starts = np.zeros(1, np.int64)
    for n, s in at:
        starts = (starts[:, None] + np.arange(n)[None] * s).ravel()
    taken = np.zeros(int(starts.max()) + c.d, bool)
    taken[(starts[:, None] + np.arange(c.d)[None]).ravel()] = True
    mid = FAKE + 64 * MB
    got = want = 0
    for apart in [*range(-len(taken) - 64, len(taken) + 65, 8 if len(taken) < 10000 else 56)]:
        a, b = max(0, apart), max(0, -apart)
        meet = bool(np.any(taken[a:len(taken) - b] & taken[b:len(taken) - a])) if abs(apart) < len(taken) else False
        code = append(L, c, k_cache=mid, v_cache=mid + 2 * apart)
        assert (code == _lib.CARVE_EINVAL) == meet and code in (_lib.CARVE_OK, _lib.CARVE_EINVAL), apart
        got, want = got + (code != _lib.CARVE_OK), want + meet
    assert got == want > 0


def test_append_refuses_caches_that_start_alike(L):
    """Whatever their strides, two caches whose first entries meet."""
    c = paged_cfg(N=0, vc_page=4096, vc_tok=192, vc_head=64)
    for apart, code in ((0, _lib.CARVE_EINVAL), (112, _lib.CARVE_EINVAL), (-112, _lib.CARVE_EINVAL),
                        (MB, _lib.CARVE_OK)):
        assert append(L, c, k_cache=FAKE + 64 * MB, v_cache=FAKE + 64 * MB + apart) == code, apart
