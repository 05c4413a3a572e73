"""The 4-bit paged cache without a GPU: its float64 oracle against its definition, and the argument checks of the C ABI,
which all run before the first HIP call."""
import ctypes

import numpy as np
import pytest

from chunk_gated_delta_carve_amd import _lib
from oracle import fp4_oracle as orc
from test_attention_cpu import FAKE, L, MB, paged_cfg  # noqa: F401


# the oracle

def test_codes_are_the_nearest_and_the_scale_the_smallest():
    rng = np.random.default_rng(1)
    for size in (1e-30, 1e-3, 1.0, 5.9, 6.5, 7.5, 1e30):
        x = rng.standard_normal((9, 64)) * size
        codes, scales = orc.encode(x)
        y, s = orc.decode(codes, scales), np.repeat(2.0 ** (scales.astype(float) - 127), 32, -1)
        assert np.all(np.abs(x - y) <= s) and np.all(np.abs(x - y)[np.abs(x) <= 2 * s] <= s[np.abs(x) <= 2 * s] / 4)
        top = np.abs(x).reshape(9, 2, 32).max(-1)
        e = 2.0 ** (scales.astype(float) - 127)
        assert np.all(top <= 7 * e) and np.all(top > 3.5 * e)


def test_values_of_the_grid_survive():
    c = np.arange(16, dtype=np.uint8)
    codes = np.tile(c[::2] | c[1::2] << 4, 2)
    for byte in (2, 100, 127, 252):
        x = orc.decode(codes, np.array([byte]))
        again, scale = orc.encode(x)
        assert np.array_equal(again, codes) and scale[0] == byte
        assert sorted(set(np.abs(x) / 2.0 ** (byte - 127))) == list(orc.GRID)


def test_ties_go_to_the_even_code():
    x = np.zeros(32)
    x[:8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]     # the last one makes the scale 1
    codes, byte = orc.encode_block(x)
    assert byte == 127 and list(codes[:8]) == [0, 2, 2, 4, 4, 6, 6, 7]
    x[7] = 7.0001
    assert orc.encode_block(x)[1] == 128
    assert orc.encode_block(-x)[0][0] == 8 | orc.encode_block(x)[0][0]


def test_blocks_that_are_not_finite_and_ends_of_the_range():
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones(32)
        x[5] = bad
        codes, byte = orc.encode_block(x)
        assert byte == 255 and not codes.any() and np.isnan(orc.decode(np.zeros(16, np.uint8), np.array([byte]))).all()
    assert orc.encode_block(np.zeros(32))[1] == 2
    big = np.full(32, float(np.finfo(np.float32).max))
    codes, byte = orc.encode_block(big)
    assert byte == 252 and np.all(codes == 7)


def test_assign_by_hand():
    table = [[5, 6, -1, -1], [7, -1, -1, -1], [8, 9, -1, -1]]
    free = [0, 1, 2, 3, -9, -9, -9]
    out = orc.assign(table, [8, 3, 7], [1, 1, 6], free, [4, 0], 4, 10, [0, 0, 1])
    cu, lens, pos, slots, count, tab, stack = out
    assert cu == [0, 1, 2, 8] and lens == [9, 4, 6] and count == (3, 0)
    # 8 and 9 are freed, request 0 takes 9, request 2 takes 8 and 3
    assert tab.tolist() == [[5, 6, 9, -1], [7, -1, -1, -1], [8, 3, -1, -1]]
    assert stack == [0, 1, 2, 3, 8, 9, -9]
    assert pos.tolist() == [8, 3, 0, 1, 2, 3, 4, 5, 0, 0]
    assert slots.tolist() == [36, 31, 32, 33, 34, 35, 12, 13, -1, -1]


# refusals

def fp4_cfg(**kw):
    base = dict(kw)
    d, Hk, page = base.get("d", 64), max(base.get("Hk", 2), 1), base.get("page_size", 16)
    for n, v in (("kc_page", Hk * d // 2 * page), ("kc_tok", Hk * d // 2), ("kc_head", d // 2),
                 ("vc_page", Hk * d // 2 * page), ("vc_tok", Hk * d // 2), ("vc_head", d // 2)):
        base.setdefault(n, v)
    small = {n: base.pop(n, v) for n, v in (
        ("ks_page", Hk * d // 32 * page), ("ks_tok", Hk * d // 32), ("ks_head", d // 32),
        ("vs_page", Hk * d // 32 * page), ("vs_tok", Hk * d // 32), ("vs_head", d // 32))}
    c = _lib.CarveFp4Config()
    c.paged = paged_cfg(**base)
    for n, v in small.items():
        setattr(c, n, v)
    return c


APP = ("k", "v", "q", "q_weight", "k_weight", "cos", "sin", "cu", "kv_lens", "table", "k_codes", "k_scales", "v_codes",
       "v_scales", "q_out")
ATT = ("q", "k_codes", "k_scales", "v_codes", "v_scales", "cu", "kv_lens", "table", "o", "lse", "workspace")
READ = ("k_codes", "k_scales", "v_codes", "v_scales", "slots", "k", "v")


def ptrs(names, given):
    base = {n: FAKE + i * 64 * MB for i, n in enumerate(names)}
    base.update(given)
    return [base[n] for n in names]


def ref(c):
    return None if c is None else ctypes.byref(c)


def append(L, c, **ptr):
    return L.carve_paged_append_fp4(ref(c), *ptrs(APP, ptr), None)


def read(L, c, **ptr):
    return L.carve_paged_read_fp4(ref(c), *ptrs(READ, ptr), None)


def attention(L, c, ws=None, **ptr):
    if ws is None:
        need = ctypes.c_int64()
        ok = c is not None and L.carve_paged_workspace_fp4(ctypes.byref(c), ctypes.byref(need)) == 0
        ws = need.value if ok else 0
    return L.carve_paged_attention_fp4(ref(c), *ptrs(ATT, ptr), ws, None)


BAD = [
    (dict(d=96), _lib.CARVE_EUNSUPPORTED), (dict(page_size=24), _lib.CARVE_EUNSUPPORTED),
    (dict(page_size=0), _lib.CARVE_EINVAL), (dict(N=-1), _lib.CARVE_EINVAL), (dict(S=-1), _lib.CARVE_EINVAL),
    (dict(pages=-1), _lib.CARVE_EINVAL), (dict(dtype=5), _lib.CARVE_EINVAL), (dict(flags=16), _lib.CARVE_EINVAL),
    (dict(flags=_lib.CARVE_PAGED_STEP), _lib.CARVE_EINVAL), (dict(width=1 << 27), _lib.CARVE_EUNSUPPORTED),
    (dict(table_row=3), _lib.CARVE_EINVAL), (dict(kc_tok=16), _lib.CARVE_EINVAL), (dict(vc_page=0), _lib.CARVE_EINVAL),
    (dict(kc_head=-32), _lib.CARVE_EINVAL), (dict(kc_tok=68), _lib.CARVE_EALIGN), (dict(vc_head=40), _lib.CARVE_EALIGN),
    (dict(ks_tok=1), _lib.CARVE_EINVAL), (dict(ks_tok=5), _lib.CARVE_EALIGN), (dict(vs_head=-2), _lib.CARVE_EINVAL),
    (dict(d=128, vs_page=258), _lib.CARVE_EALIGN), (dict(kc_page=1 << 31), _lib.CARVE_EUNSUPPORTED),
    (dict(vs_page=1 << 31), _lib.CARVE_EUNSUPPORTED), (dict(N=1 << 30, Hq=4, Hk=2), _lib.CARVE_EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD, ids=[str(i) for i in range(len(BAD))])
def test_config_refused(L, kw, code):  # noqa: F811
    assert append(L, fp4_cfg(**kw)) == code
    assert read(L, fp4_cfg(**kw)) == code
    assert attention(L, fp4_cfg(**kw)) == code


def test_append_arguments_refused(L):  # noqa: F811
    c = fp4_cfg()
    at = {n: FAKE + i * 64 * MB for i, n in enumerate(APP)}
    assert append(L, None) == _lib.CARVE_EINVAL
    for n in APP:
        if "weight" not in n:
            assert append(L, c, **{n: None}) == _lib.CARVE_EINVAL, n
    for n in APP:
        small = n in ("cu", "kv_lens", "table", "k_scales", "v_scales")
        assert append(L, c, **{n: FAKE + 2000 * MB + (2 if small else 8)}) == _lib.CARVE_EALIGN, n
    assert append(L, fp4_cfg(rot=8)) == _lib.CARVE_EUNSUPPORTED
    assert append(L, fp4_cfg(eps=0.0)) == _lib.CARVE_EINVAL
    assert append(L, fp4_cfg(flags=0)) == _lib.CARVE_EINVAL                         # weights without the norm
    assert append(L, c, q_out=at["k"]) == _lib.CARVE_EINVAL
    assert append(L, c, q_out=at["q"] + 16) == _lib.CARVE_EINVAL                    # a shifted view of q
    assert append(L, c, k=at["k_codes"] + 4096) == _lib.CARVE_EINVAL                # inside the cache
    assert append(L, c, table=at["v_scales"] + 64) == _lib.CARVE_EINVAL
    for a, b in (("k_codes", "v_codes"), ("k_scales", "v_scales"), ("k_codes", "k_scales"), ("v_codes", "k_scales")):
        assert append(L, c, **{b: at[a]}) == _lib.CARVE_EINVAL, (a, b)
    assert append(L, c, v_codes=at["k_codes"] + 12 * 1024 - 16) == _lib.CARVE_EINVAL     # its last entry's second half
    for kw in (dict(kc_tok=32, kc_head=32), dict(ks_tok=2, ks_head=2), dict(vs_page=16)):   # entries in one place
        assert append(L, fp4_cfg(**kw)) == _lib.CARVE_EINVAL, kw
    assert append(L, fp4_cfg(N=1 << 26)) == _lib.CARVE_EUNSUPPORTED
    assert append(L, fp4_cfg(N=0)) == _lib.CARVE_OK
    assert append(L, fp4_cfg(S=0)) == _lib.CARVE_OK


def test_read_arguments_refused(L):  # noqa: F811
    c = fp4_cfg()
    at = {n: FAKE + i * 64 * MB for i, n in enumerate(READ)}
    assert read(L, None) == _lib.CARVE_EINVAL
    for n in READ[:5]:
        assert read(L, c, **{n: None}) == _lib.CARVE_EINVAL, n
    for n in READ:
        small = n in ("k_scales", "v_scales")
        assert read(L, c, **{n: FAKE + 2000 * MB + (2 if small else 4)}) == _lib.CARVE_EALIGN, n
    assert read(L, fp4_cfg(k_row=64)) == _lib.CARVE_EINVAL                           # rows of 128
    assert read(L, c, k=at["v"]) == _lib.CARVE_EINVAL
    assert read(L, c, v=at["slots"]) == _lib.CARVE_EINVAL
    assert read(L, c, k=at["k_codes"]) == _lib.CARVE_EINVAL
    assert read(L, fp4_cfg(N=1 << 26)) == _lib.CARVE_EUNSUPPORTED
    assert read(L, fp4_cfg(N=0)) == _lib.CARVE_OK
    assert read(L, fp4_cfg(Hk=0, Hq=0)) == _lib.CARVE_OK
    assert read(L, c, k=None, v=None, slots=None) == _lib.CARVE_OK                   # nothing is asked for


def test_attention_arguments_refused(L):  # noqa: F811
    c = fp4_cfg()
    at = {n: FAKE + i * 64 * MB for i, n in enumerate(ATT)}
    assert attention(L, None) == _lib.CARVE_EINVAL
    for n in ATT[:9]:
        assert attention(L, c, **{n: None}) == _lib.CARVE_EINVAL, n
    for n in ATT:
        small = n in ("cu", "kv_lens", "table", "lse", "k_scales", "v_scales")
        assert attention(L, c, **{n: FAKE + 2000 * MB + (2 if small else 8)}) == _lib.CARVE_EALIGN, n
    for s in (0.0, -0.1, float("nan")):
        assert attention(L, fp4_cfg(scale=s)) == _lib.CARVE_EINVAL
    assert attention(L, fp4_cfg(scale=17.0)) == _lib.CARVE_EUNSUPPORTED
    assert attention(L, fp4_cfg(Hq=5)) == _lib.CARVE_EINVAL
    assert attention(L, fp4_cfg(Hk=0)) == _lib.CARVE_EINVAL
    assert attention(L, fp4_cfg(pages=0)) == _lib.CARVE_EINVAL
    for n in ("q", "k_codes", "v_scales", "table"):
        assert attention(L, c, o=at[n]) == _lib.CARVE_EINVAL, n
    assert attention(L, c, lse=at["o"]) == _lib.CARVE_EINVAL
    need = ctypes.c_int64()
    assert L.carve_paged_workspace_fp4(ctypes.byref(c), None) == _lib.CARVE_EINVAL
    assert L.carve_paged_workspace_fp4(None, ctypes.byref(need)) == _lib.CARVE_EINVAL
    for kw in (dict(N=0), dict(S=0), dict(Hq=0)):
        assert attention(L, fp4_cfg(**kw)) == _lib.CARVE_OK


ASSIGN = ("kv_lens", "new_lens", "done", "table", "free_pages", "free_count", "kv_lens_out", "cu", "positions", "slots",
          "free_count_out")


def assign(L, ptr=(), **kw):
    base = dict(S=5, N=40, page_size=16, width=8, table_row=8, capacity=64)
    base.update(kw)
    return L.carve_paged_assign(ctypes.byref(_lib.CarveAssignConfig(**base)), *ptrs(ASSIGN, dict(ptr)), None)


def test_more_blocks_than_the_row_kernel_counts(L):  # noqa: F811
    """Few rows a sequence under a table of 2^23 keys each: the tile kernels take them, fp32 is refused."""
    need = ctypes.c_int64()
    for dtype, code in ((_lib.CARVE_BF16, _lib.CARVE_OK), (_lib.CARVE_F32, _lib.CARVE_EUNSUPPORTED)):
        c = fp4_cfg(N=8192, S=256, Hq=128, Hk=32, d=128, width=1 << 19, pages=1 << 19, dtype=dtype)
        assert L.carve_paged_workspace_fp4(ctypes.byref(c), ctypes.byref(need)) == code
    c = fp4_cfg(N=8192, S=256, Hq=128, Hk=32, d=128, width=1 << 12, pages=1 << 12)
    assert L.carve_paged_workspace_fp4(ctypes.byref(c), ctypes.byref(need)) == _lib.CARVE_OK and need.value > 0


def test_assign_refused(L):  # noqa: F811
    at = {n: FAKE + i * 64 * MB for i, n in enumerate(ASSIGN)}
    assert L.carve_paged_assign(None, *ptrs(ASSIGN, {}), None) == _lib.CARVE_EINVAL
    for kw in (dict(S=-1), dict(N=-1), dict(page_size=0), dict(width=-1), dict(table_row=7), dict(table_row=-8),
               dict(capacity=-1)):
        assert assign(L, **kw) == _lib.CARVE_EINVAL, kw
    for kw in (dict(page_size=12), dict(width=1 << 27, table_row=1 << 27), dict(capacity=1 << 31), dict(table_row=1 << 31)):
        assert assign(L, **kw) == _lib.CARVE_EUNSUPPORTED, kw
    for n in ASSIGN:
        if n not in ("done", "positions", "slots"):
            assert assign(L, {n: None}) == _lib.CARVE_EINVAL, n
        assert assign(L, {n: FAKE + 2000 * MB + (4 if n == "slots" else 2)}) == _lib.CARVE_EALIGN, n
    for n, m in (("cu", "kv_lens"), ("table", "free_pages"), ("positions", "new_lens"), ("slots", "positions"),
                 ("kv_lens_out", "new_lens"), ("kv_lens_out", "cu"), ("free_count_out", "free_pages"),
                 ("free_pages", "done"), ("free_count_out", "kv_lens"), ("cu", "free_count")):
        assert assign(L, {n: at[m]}) == _lib.CARVE_EINVAL, (n, m)
    assert assign(L, {"kv_lens_out": at["kv_lens"] + 4}) == _lib.CARVE_EINVAL     # shifted, not in place


def test_a_cache_of_its_own():
    torch = pytest.importorskip("torch")
    from chunk_gated_delta_carve_amd import paged_fp4_cache
    kc, ks, vc, vs = paged_fp4_cache(5, 16, 3, 128, device="cpu")
    assert kc.shape == vc.shape == (5, 16, 3, 64) and ks.shape == vs.shape == (5, 16, 3, 4)
    assert kc.dtype == torch.uint8 and kc.stride() == (3 * 16 * 64, 64, 16 * 64, 1) and ks.stride(1) == 4
    for kw in (dict(d=96), dict(page_size=12), dict(page_size=0)):
        with pytest.raises(ValueError):
            paged_fp4_cache(**{**dict(pages=2, page_size=16, heads=1, d=64, device="cpu"), **kw})


def test_sizes_past_32_bits_in_python():
    from chunk_gated_delta_carve_amd import paged_fp4_workspace_bytes
    base = dict(N=4, S=4, Hq=8, Hk=2, d=64, page_size=16, width=10)
    for n in base:
        with pytest.raises(ValueError):
            paged_fp4_workspace_bytes(**{**base, n: 2 ** 31})
    assert paged_fp4_workspace_bytes(**base, window=2 ** 40) == paged_fp4_workspace_bytes(**base)


def test_what_a_read_is_limited_to(L):  # noqa: F811
    """The whole configuration has to hold, and the outputs have at most 2^24 - 1 workgroups of 2^14 bytes."""
    c = fp4_cfg(N=20, S=3, flags=_lib.CARVE_PAGED_STEP, k_row=256, v_row=256)
    assert read(L, c) == _lib.CARVE_EINVAL
    far = dict(zip(READ, (FAKE + i * (1 << 42) for i in range(len(READ)))))
    for d, dtype, Hk, N in ((128, _lib.CARVE_F32, 64, 1 << 22), (128, _lib.CARVE_BF16, 256, 1 << 21)):
        c = fp4_cfg(N=N, S=0, Hq=0, Hk=Hk, d=d, dtype=dtype, width=0, flags=0, rot=0)
        assert 2 * N * Hk * d * (4 if dtype == _lib.CARVE_F32 else 2) > 2 ** 38 - 2 ** 14
        assert read(L, c, **far) == _lib.CARVE_EUNSUPPORTED


def test_values_that_do_not_fit_the_configuration():
    """Sizes past 32 bits and what is no float are refused, the latter not as a size; a float past fp32's range goes through as infinity, which
    the library refuses by its own range, as in the calls over the other caches."""
    from chunk_gated_delta_carve_amd.fp4 import _pack
    ok = [1] * 13 + [1e-6, 0.125] + [0] * 17
    c = _lib.CarveFp4Config.from_buffer_copy(_pack(*ok))
    assert c.paged.scale == 0.125 and c.paged.N == 1
    for at, name in ((13, "eps"), (14, "scale")):
        c = _lib.CarveFp4Config.from_buffer_copy(_pack(*ok[:at], 1e300, *ok[at + 1:]))
        assert getattr(c.paged, name) == getattr(_lib.CarvePagedConfig(**{name: 1e300}), name) == float("inf")
        for bad in ("x", 10 ** 400):
            with pytest.raises(ValueError, match="not a float") as e:
                _pack(*ok[:at], bad, *ok[at + 1:])
            assert "size" not in str(e.value)
    with pytest.raises(ValueError):
        _pack(1 << 31, *ok[1:])
