"""The attention layer's operators on the GPU against their float64 definitions (oracle/attention_oracle.py).

Bounds, derived per element (h: half a step of the type relative to a value, 2^-24 for fp32 and 2^-8 for bf16):
  norm and rotation   h |y| for the one rounding of the output, and 2^-19 of the row's largest |z| for the fp32
                      arithmetic: the mean's error (a tree and a chain, under 20 additions of 2^-24 relative each,
                      halved by the root), the root and reciprocal, three products and the two terms of the turn
  its gradient        the same two terms around the largest |r dz w| of the row; weight sums add n 2^-24 of the sum
                      of their terms' magnitudes in the worst order
  attention           each score is off by at most e = scale (d + 4) 2^-24 max_j sum|q k| (the product) plus 2^-20
                      (the exponential's argument and result); with A the softmax mean of |v| a row is off by
                      (2 e + (keys + 64) 2^-24) A for numerator and denominator, by h A for the weights' rounding
                      (bf16) and by h |o| for its own; lse by e + (keys + 64) 2^-24 + 2^-22 |lse|
"""
import numpy as np
import pytest

from oracle import attention_oracle as orc

pytestmark = pytest.mark.gpu
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def say(*a):
    print(*a, flush=True)


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from chunk_gated_delta_carve_amd import _lib
    _lib.lib()                                   # loud failure if the library is missing
    return torch


def dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def rand(torch, seed, shape, dtype, scale=1.0, add=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + add).to(dt(torch, dtype)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(torch, x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def close(name, got, ref, bound):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= bound)          # NaN counts as off
    worst = np.max(np.abs(got - ref) / np.maximum(bound, 1e-300)) if got.size else 0.0
    say(f"  {name}: {worst:.3f} of the bound")
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {worst:.3f} of the bound at {np.argwhere(bad)[0]}"


# norm and rotation

ROPE = [
    # dtype, lead, Hq, Hk, d, rot, interleaved, norm, weights, positions
    ("bf16", (1,), 1, 1, 64, 64, False, True, True, False),
    ("bf16", (2, 33), 12, 12, 64, 64, False, True, True, False),
    ("bf16", (3, 17), 12, 4, 64, 32, True, True, True, True),
    ("bf16", (5, 7), 16, 2, 128, 128, False, True, True, True),
    ("bf16", (41,), 3, 1, 128, 16, False, True, False, False),
    ("bf16", (9,), 2, 5, 128, 128, True, False, False, True),
    ("bf16", (6,), 4, 4, 64, 0, False, True, True, False),
    ("f32", (2, 19), 12, 4, 64, 64, False, True, True, True),
    ("f32", (77,), 5, 1, 128, 128, True, True, True, False),
    ("f32", (4, 3), 2, 2, 128, 48, False, True, True, True),
    ("f32", (1,), 1, 1, 128, 128, False, False, False, True),
]
ROPE_IDS = ["-".join(str(x).replace(" ", "") for x in c) for c in ROPE]


def rope_inputs(torch, case, seed):
    dtype, lead, Hq, Hk, d, rot, inter, norm, weights, positions = case
    both = rand(torch, seed, (*lead, Hq + Hk, d), dtype, 1.5)     # two parts of one tensor: strided tokens
    t = dict(q=both[..., :Hq, :], k=both[..., Hq:, :])
    from chunk_gated_delta_carve_amd import rope_tables
    P = 200
    kw = dict(norm=norm, interleaved=inter, eps=1e-5)
    if rot:
        kw["cos"], kw["sin"] = rope_tables(P, rot)
    if weights:
        kw["q_weight"], kw["k_weight"] = (rand(torch, seed + i, (d,), dtype, 0.3, 1.0) for i in (1, 2))
    pos = np.broadcast_to(np.arange(lead[-1]), lead)
    if positions:
        pos = np.random.default_rng(seed).integers(0, P, lead)
        kw["positions"] = ints(torch, pos)
    orc_kw = dict(cos=f64(kw["cos"]) if rot else None, sin=f64(kw["sin"]) if rot else None, pos=pos, rot=rot,
                  interleaved=inter, norm=norm, eps=1e-5)
    return t, kw, orc_kw


def row_max(x):
    return np.max(np.abs(x), axis=-1, keepdims=True)


@pytest.mark.parametrize("case", ROPE, ids=ROPE_IDS)
def test_norm_rope(torch, case):
    from chunk_gated_delta_carve_amd import qk_norm_rope_fwd
    t, kw, ok = rope_inputs(torch, case, 10)
    say("case", case)
    out = qk_norm_rope_fwd(t["q"], t["k"], **kw)
    torch.cuda.synchronize()
    for n, got in zip("qk", out):
        w = kw.get(n + "_weight")
        ref = orc.norm_rope(f64(t[n]), None if w is None else f64(w), **ok)
        close(n, got, ref, HALF[case[0]] * np.abs(ref) + 2.0 ** -19 * row_max(ref))


@pytest.mark.parametrize("case", ROPE, ids=ROPE_IDS)
def test_norm_rope_gradient(torch, case):
    from chunk_gated_delta_carve_amd import qk_norm_rope_bwd
    t, kw, ok = rope_inputs(torch, case, 20)
    say("case", case)
    dy = {n: rand(torch, 30 + i, tuple(t[n].shape), case[0]) for i, n in enumerate("qk")}
    got = qk_norm_rope_bwd(t["q"], t["k"], dy["q"], dy["k"], **kw)
    torch.cuda.synchronize()
    for n in "qk":
        w = kw.get(n + "_weight")
        x, w64 = f64(t[n]), None if w is None else f64(w)
        dx, dw = orc.norm_rope_grad(x, w64, f64(dy[n]), **ok)
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-5) if case[7] else 1.0
        size = row_max(f64(dy[n])) * np.sqrt(2) * np.max(r * (1 if w is None else np.max(np.abs(w64))), -1, keepdims=True)
        # the row's dot product is a mean of d terms, each at most size times |x r| <= sqrt(d)
        size = size * np.maximum(1.0, row_max(x * r) ** 2)
        close("d" + n, got["d" + n], dx, HALF[case[0]] * np.abs(dx) + 2.0 ** -19 * size)
        if w is None:
            assert got[f"d{n}_weight"] is None
        else:
            dz = orc.norm_rope_grad(x, None, f64(dy[n]), **{**ok, "norm": False})[0]
            terms = np.sum(np.abs(dz * x * r).reshape(-1, x.shape[-1]), axis=0)
            turned = np.sqrt(2) * np.sum((row_max(f64(dy[n])) * np.abs(x * r)).reshape(-1, x.shape[-1]), axis=0)
            rows = x.size // x.shape[-1]
            close(f"d{n}_weight", got[f"d{n}_weight"], dw, rows * 2.0 ** -24 * terms + 2.0 ** -20 * turned)


def test_norm_rope_in_place_and_bits(torch):
    """Outputs over their inputs (the two parts of one projection's output), and gradients over the output gradients,
    have the bits of separate buffers; two calls of the gradient have the same bits."""
    from chunk_gated_delta_carve_amd import qk_norm_rope_bwd, qk_norm_rope_fwd
    case = ("bf16", (7, 300), 12, 4, 64, 64, False, True, True, False)
    t, kw, _ = rope_inputs(torch, (*case[:5], 64, *case[6:]), 40)
    from chunk_gated_delta_carve_amd import rope_tables
    kw["cos"], kw["sin"] = rope_tables(300, 64)
    ref = qk_norm_rope_fwd(t["q"], t["k"], **kw)
    g = [rand(torch, 41 + i, tuple(t[n].shape), "bf16") for i, n in enumerate("qk")]
    a = qk_norm_rope_bwd(t["q"], t["k"], *g, **kw)
    b = qk_norm_rope_bwd(t["q"], t["k"], *g, dq=g[0], dk=g[1], **kw)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    assert b["dq"].data_ptr() == g[0].data_ptr()
    out = qk_norm_rope_fwd(t["q"], t["k"], q_out=t["q"], k_out=t["k"], **kw)
    for x, y in zip(ref, out):
        assert torch.equal(x, y)
    with pytest.raises(Exception):
        qk_norm_rope_fwd(t["q"], t["k"], q_out=t["q"], k_out=t["q"], **kw)


def test_position_outside_the_table_is_nan(torch):
    from chunk_gated_delta_carve_amd import qk_norm_rope_fwd, rope_tables
    q = rand(torch, 1, (4, 2, 64), "bf16")
    cos, sin = rope_tables(10, 32)
    out, _ = qk_norm_rope_fwd(q, q.clone(), cos, sin, ints(torch, [9, 10, -1, 2 ** 31 - 1]))
    assert torch.isfinite(out[0]).all()
    assert torch.isnan(out[1:, :, :32]).all() and torch.isfinite(out[1:, :, 32:]).all()


def test_gradient_without_tokens_is_zero(torch):
    from chunk_gated_delta_carve_amd import qk_norm_rope_bwd
    q = torch.empty(0, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    got = qk_norm_rope_bwd(q, q.clone(), q.clone(), q.clone(), q_weight=w, k_weight=w)
    assert got["dq"].shape == (0, 2, 64) and not got["dq_weight"].any() and not got["dk_weight"].any()


# the paged cache

def ragged(torch, seed, S, n, kv, page, spare=2, width=None):
    """cu, kv_lens and a block table of shuffled pages for sequences of n[s] new tokens out of kv[s]."""
    rng = np.random.default_rng(seed)
    need = [-(-max(x, 0) // page) for x in kv]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((S, width or max(max(need), 1)), -1)
    at = 0
    for s in range(S):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
    return np.concatenate([[0], np.cumsum(n)]), np.array(kv), table, pages


def cache(torch, layout, pages, page, Hk, d, dtype, seed):
    """A pair of caches [pages, page, Hk, d] in one of the layouts a program may keep."""
    if layout == "plain":
        return tuple(rand(torch, seed + i, (pages, page, Hk, d), dtype) for i in range(2))
    if layout == "joint":                        # one tensor for both
        both = rand(torch, seed, (pages, 2, page, Hk, d), dtype)
        return both[:, 0], both[:, 1]
    both = rand(torch, seed, (2, pages, Hk, page, d), dtype)          # heads before tokens
    return both[0].transpose(1, 2), both[1].transpose(1, 2)


APPEND = [
    # dtype, Hq, Hk, d, page, n, kv, rot, interleaved, norm, layout, step
    ("bf16", 12, 4, 64, 16, [5, 0, 33, 1], [5, 7, 40, 100], 64, False, True, "plain", False),
    ("bf16", 16, 2, 128, 64, [100, 1], [163, 64], 128, True, False, "joint", False),
    ("bf16", 16, 4, 128, 16, [1] * 9, [1, 16, 17, 31, 32, 33, 200, 2, 48], 128, False, True, "heads", True),
    ("bf16", 0, 3, 64, 1, [3, 2], [4, 2], 16, False, False, "plain", False),
    ("bf16", 1, 1, 128, 256, [300], [300], 0, False, True, "plain", False),
    ("f32", 12, 4, 64, 16, [9, 14], [20, 14], 64, False, True, "heads", False),
    ("f32", 3, 3, 128, 32, [1, 1], [33, 1], 64, True, True, "joint", True),
]


@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
def test_append(torch, case):
    from chunk_gated_delta_carve_amd import paged_append, rope_tables
    dtype, Hq, Hk, d, page, n, kv, rot, inter, norm, layout, step = case
    say("case", case)
    S, N = len(n), sum(n)
    cu, lens, table, pages = ragged(torch, 5, S, n, kv, page)
    kc, vc = cache(torch, layout, pages, page, Hk, d, dtype, 50)
    k, v = rand(torch, 52, (N, Hk, d), dtype, 1.5), rand(torch, 53, (N, Hk, d), dtype)
    q = rand(torch, 54, (N, Hq, d), dtype, 1.5) if Hq else None
    kw = {}
    if rot:
        kw["cos"], kw["sin"] = rope_tables(max(kv), rot)
    if norm:
        kw["k_weight"] = rand(torch, 55, (d,), dtype, 0.3, 1.0)
        if Hq:
            kw["q_weight"] = rand(torch, 56, (d,), dtype, 0.3, 1.0)
    before = f64(kc), f64(vc)
    ok = dict(cos=f64(kw["cos"]) if rot else None, sin=f64(kw["sin"]) if rot else None, rot=rot, interleaved=inter,
              norm=norm, eps=1e-6)
    out = paged_append(k, v, kc, vc, ints(torch, table), ints(torch, lens), None if step else ints(torch, cu), q=q,
                       norm=norm, interleaved=inter, **kw)
    torch.cuda.synchronize()
    w = f64(kw["k_weight"]) if norm else None
    turn = lambda row, pos: orc.norm_rope(row[None], w, pos=np.array([pos]), **ok)[0]  # noqa: E731
    ref_k, ref_v = orc.paged_append(f64(k), f64(v), *before, table, lens, cu, page, turn)
    new = ref_v != before[1]                     # entries that were stored
    close("k_cache", kc, ref_k, np.where(new.any(-1, keepdims=True), HALF[dtype] * np.abs(ref_k)
                                         + 2.0 ** -19 * row_max(ref_k), 0.0))
    close("v_cache", vc, ref_v, np.zeros(()))
    if Hq:
        pos = np.array([p[1] for p in orc.token_places(cu, lens, N)])
        ref_q = orc.norm_rope(f64(q), f64(kw["q_weight"]) if norm else None, pos=pos, **ok)
        close("q", out, ref_q, HALF[dtype] * np.abs(ref_q) + 2.0 ** -19 * row_max(ref_q))
    else:
        assert out is None


def test_append_drops_what_has_no_place(torch):
    """Negative positions, positions past the table, page numbers outside the cache and tokens behind the last
    sequence leave the cache (and q_out of the latter) as they were."""
    from chunk_gated_delta_carve_amd import paged_append
    page, Hk, d, pages = 16, 2, 64, 5
    n, kv = [4, 4, 20, 3], [2, 64, 20, 3]        # two negative positions; past the table; through bad pages; good
    cu = np.concatenate([[0], np.cumsum(n)])
    table = np.array([[0, -1], [1, 2], [-5, 99], [3, 4]])
    N = sum(n) + 6
    kc, vc = cache(torch, "plain", pages, page, Hk, d, "bf16", 60)
    k, v, q = (rand(torch, 61 + i, (N, Hk, d), "bf16") for i in range(3))
    before = f64(kc), f64(vc)
    out = torch.full_like(q, 7.0)
    paged_append(k, v, kc, vc, ints(torch, table), ints(torch, kv), ints(torch, cu), q=q, q_out=out)
    ref = orc.paged_append(f64(k), f64(v), *before, table, kv, cu, page)
    assert np.array_equal(f64(kc), ref[0]) and np.array_equal(f64(vc), ref[1])
    assert (ref[0] != before[0]).any(-1).sum() == Hk * (2 + 3)
    assert torch.equal(out[:31], q[:31]) and (out[31:] == 7.0).all()


# attention

ATTENTION = [
    # dtype, Hq, Hk, d, page, n, kv, window, layout, step
    ("bf16", 1, 1, 64, 16, [1], [1], 0, "plain", True),
    ("bf16", 12, 12, 64, 16, [1, 1, 1], [1, 130, 17], 0, "plain", True),
    ("bf16", 16, 2, 128, 16, [1, 1, 1, 1], [0, 33, 700, 128], 0, "joint", True),
    ("bf16", 16, 4, 128, 64, [1, 1], [2000, 5], 100, "heads", True),
    ("bf16", 64, 2, 64, 32, [1, 1], [90, 31], 0, "plain", True),          # more heads in a group than a tile has rows
    ("bf16", 12, 4, 64, 16, [5, 0, 3], [5, 9, 300], 0, "plain", False),
    ("bf16", 6, 2, 128, 1, [3, 2], [40, 2], 7, "plain", False),
    ("bf16", 12, 4, 64, 16, [200, 1, 65], [200, 77, 333], 0, "plain", False),
    ("bf16", 16, 2, 128, 64, [130, 64], [259, 64], 0, "joint", False),
    ("bf16", 4, 4, 128, 16, [257], [600], 50, "heads", False),
    ("bf16", 3, 1, 64, 256, [150], [1500], 0, "plain", False),
    ("bf16", 2, 1, 128, 16, [129], [129], 1, "plain", False),
    ("bf16", 2, 2, 64, 32, [300, 40], [100, 40], 0, "plain", False),      # more new tokens than the length: empty rows
    # more than 128 tiles of 256 rows at d = 128
    ("bf16", 130, 130, 128, 16, [40], [40], 0, "plain", False),
    ("bf16", 16, 16, 128, 1, [40, 9, 70, 0, 33, 64, 33, 41, 36, 39], [300, 9, 70, 5, 65, 200, 64, 500, 30, 39], 0,
     "joint", False),
    ("bf16", 32, 16, 128, 64, [257, 129, 20, 1, 2, 50, 33, 64], [700, 129, 400, 90, 2, 64, 100, 333], 90, "heads",
     False),
    ("bf16", 64, 32, 128, 8, [513], [600], 0, "plain", False),
    ("f32", 12, 4, 64, 16, [5, 1, 40], [5, 129, 140], 0, "plain", False),
    ("f32", 4, 2, 128, 32, [17, 3], [200, 3], 33, "heads", False),
    ("f32", 16, 2, 128, 16, [1, 1, 1], [1, 400, 65], 0, "joint", True),
    ("f32", 5, 1, 64, 64, [70], [70], 0, "plain", False),
]


def attention_bounds(dtype, d, scale, o, lse, A, reach, keys):
    h = HALF[dtype]
    e = scale * (d + 4) * 2.0 ** -24 * reach + 2.0 ** -20
    acc = (keys[:, None] + 64) * 2.0 ** -24
    slack = 2 * e + acc + (h if dtype == "bf16" else 0.0)
    return h * np.abs(o) + slack[..., None] * A, e + acc + 2.0 ** -22 * np.abs(lse)


def check_attention(torch, got, got_lse, q, kc, vc, table, lens, cu, scale, window, dtype):
    d = q.shape[-1]
    o, lse, A, reach, keys = orc.paged_attention(f64(q), f64(kc), f64(vc), table, lens, cu, scale, window)
    live = ~np.isnan(lse[:, 0])
    with np.errstate(invalid="ignore"):
        bo, bl = attention_bounds(dtype, d, scale, o, lse, A, reach, keys)
    close("o", got[torch.tensor(live)] if live.any() else got[:0], o[live], bo[live])
    gl = f64(got_lse)[live]
    empty = np.isneginf(lse[live])
    assert np.array_equal(np.isneginf(gl), empty)
    assert np.all(np.abs(gl - lse[live])[~empty] <= bl[live][~empty])
    return o, keys


@pytest.mark.parametrize("case", ATTENTION, ids=[str(i) for i in range(len(ATTENTION))])
def test_attention(torch, case):
    """Every cache entry that no row sees holds NaN: other pages, the rest of the last page, keys before every
    window; block-table entries past a sequence's pages are -1."""
    from chunk_gated_delta_carve_amd import paged_attention
    dtype, Hq, Hk, d, page, n, kv, window, layout, step = case
    say("case", case)
    S, N = len(n), sum(n)
    cu, lens, table, pages = ragged(torch, 7, S, n, kv, page)
    kc, vc = cache(torch, layout, pages, page, Hk, d, dtype, 70)
    q = rand(torch, 72, (N, Hq, d), dtype)
    seen = np.zeros((pages, page), bool)
    for at in orc.token_places(cu, lens, N):
        s, p = at
        for j in range(max(0, p - window + 1) if window else 0, p + 1):
            seen[orc.place(table, s, j, page, pages)] = True
    hide = torch.tensor(~seen, device="cuda")[..., None, None]
    kc.masked_fill_(hide, float("nan"))
    vc.masked_fill_(hide, float("nan"))
    out, lse = paged_attention(q, kc, vc, ints(torch, table), ints(torch, lens), None if step else ints(torch, cu),
                               window=window, return_lse=True)
    torch.cuda.synchronize()
    check_attention(torch, out, lse, q, kc, vc, table, lens, cu, d ** -0.5, window, dtype)


@pytest.mark.parametrize("dtype,d,kv,n,Hq,Hk", [("bf16", 64, 9000, 1, 12, 12), ("bf16", 128, 20011, 1, 16, 2),
                                                ("bf16", 128, 5001, 300, 4, 1), ("f32", 64, 3001, 2, 4, 2),
                                                ("bf16", 64, 2000, 1999, 12, 4), ("bf16", 128, 2300, 1030, 16, 8)])
def test_attention_split_over_a_long_context(torch, dtype, d, kv, n, Hq, Hk):
    """Few rows over many keys are split over workgroups and joined; the same bits every time."""
    from chunk_gated_delta_carve_amd import paged_attention
    cu, lens, table, pages = ragged(torch, 8, 1, [n], [kv], 64)
    kc, vc = cache(torch, "plain", pages, 64, Hk, d, dtype, 80)
    q = rand(torch, 82, (n, Hq, d), dtype, 2.0)
    args = (q, kc, vc, ints(torch, table), ints(torch, lens), ints(torch, cu))
    out, lse = paged_attention(*args, return_lse=True)
    again, lse2 = paged_attention(*args, return_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    rows = [0, n // 2, n - 1] if n > 2 else list(range(n))
    sub = np.array(rows)
    o, l, A, reach, keys = (np.concatenate(x) for x in zip(*(
        orc.paged_attention(f64(q[r:r + 1]), f64(kc), f64(vc), table, [kv - n + 1 + r], [0, 1], d ** -0.5, 0)
        for r in rows)))
    bo, bl = attention_bounds(dtype, d, d ** -0.5, o, l, A, reach, keys)
    close("o", out[sub], o, bo)
    close("lse", lse[sub], l, bl)


@pytest.mark.parametrize("dtype,n,kv", [("bf16", 1, 40), ("bf16", 100, 100), ("f32", 9, 20), ("bf16", 3, 5000)])
def test_pages_that_are_not_there(torch, dtype, n, kv):
    """Page numbers outside the cache, in the middle of a sequence: their keys are not seen."""
    from chunk_gated_delta_carve_amd import paged_attention
    cu, lens, table, pages = ragged(torch, 9, 1, [n], [kv], 16)
    table[0, 1], table[0, -1] = pages + 3, -7
    kc, vc = cache(torch, "plain", pages, 16, 2, 64, dtype, 90)
    q = rand(torch, 92, (n, 4, 64), dtype)
    out, lse = paged_attention(q, kc, vc, ints(torch, table), ints(torch, lens), ints(torch, cu), return_lse=True)
    check_attention(torch, out, lse, q, kc, vc, table, lens, cu, 0.125, 0, dtype)


def test_nothing_to_see(torch):
    """A table that is too short or all holes gives zero outputs and -inf."""
    from chunk_gated_delta_carve_amd import paged_attention
    kc, vc = cache(torch, "plain", 2, 16, 2, 64, "bf16", 95)
    for n in (2, 100):
        q = rand(torch, 96, (n, 4, 64), "bf16")
        out, lse = paged_attention(q, kc, vc, ints(torch, [[-1, -1]]), ints(torch, [n]), ints(torch, [0, n]),
                                   return_lse=True)
        assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,n,Hk,d", [("bf16", 6, 2, 64), ("bf16", 150, 2, 64), ("f32", 6, 2, 64),
                                          ("bf16", 150, 2, 128), ("bf16", 150, 66, 128)])
def test_a_bad_value_reaches_only_the_rows_that_see_it(torch, bad, dtype, n, Hk, d):
    """A token's infinite or NaN key or value, inside the blocks that other rows of the same tile share, leaves the
    rows before it (and, with a window, those past it) as they are."""
    from chunk_gated_delta_carve_amd import paged_attention
    kv, window, Hq = n + 20, 10, 2 * Hk
    cu, lens, table, pages = ragged(torch, 11, 1, [n], [kv], 16)
    for which in (0, 1):
        pair = cache(torch, "plain", pages, 16, Hk, d, dtype, 100)
        q = rand(torch, 102, (n, Hq, d), dtype)
        args = (ints(torch, table), ints(torch, lens), ints(torch, cu))
        clean, clean_lse = paged_attention(q, *pair, *args, window=window, return_lse=True)
        j = kv - n // 2                          # that position's page entry
        pair[which][table[0, j // 16], j % 16, :, 3] = bad
        out, lse = paged_attention(q, *pair, *args, window=window, return_lse=True)
        p = np.arange(kv - n, kv)
        sees = (j <= p) & (j > p - window)
        ref = orc.paged_attention(f64(q), f64(pair[0]), f64(pair[1]), table, lens, cu, d ** -0.5, window)
        rows = torch.tensor(~sees)
        bo, bl = attention_bounds(dtype, d, d ** -0.5, *ref)
        close("rows that do not see it", out[rows], ref[0][~sees], bo[~sees])
        close("their lse", lse[rows], ref[1][~sees], bl[~sees])
        if which:                                # an infinite or NaN value shows in its channel alone
            seen = f64(out)[sees]
            assert not np.isfinite(seen[:, :, 3]).any() and np.isfinite(np.delete(seen, 3, 2)).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,n,d", [("bf16", 6, 64), ("bf16", 6, 128), ("bf16", 100, 64), ("bf16", 100, 128),
                                       ("f32", 6, 64), ("f32", 6, 128)])
def test_a_bad_value_in_a_context_that_is_split(torch, bad, dtype, n, d):
    """As above, with the context dealt to many workgroups: the part that holds the bad value is computed again by the
    row, the others join it."""
    from chunk_gated_delta_carve_amd import paged_attention
    kv, window = 4000, 2000
    cu, lens, table, pages = ragged(torch, 13, 1, [n], [kv], 16)
    pair = cache(torch, "plain", pages, 16, 1, d, dtype, 114)
    q = rand(torch, 116, (n, 2, d), dtype)
    args = (ints(torch, table), ints(torch, lens), ints(torch, cu))
    p = np.arange(kv - n, kv)
    first = p - window + 1
    edge = kv - n // 2 - window                  # falls out of the window half-way through the new tokens
    for j in (edge, 3000):
        _, vc = (x.clone() for x in pair)
        vc[table[0, j // 16], j % 16, :, 3] = bad
        out, lse = paged_attention(q, pair[0], vc, *args, window=window, return_lse=True)
        sees = j >= first
        ref = orc.paged_attention(f64(q), f64(pair[0]), f64(pair[1]), table, lens, cu, d ** -0.5, window)
        bo, bl = attention_bounds(dtype, d, d ** -0.5, *ref)
        close("lse", lse, ref[1], bl)
        got = f64(out)
        assert not np.isfinite(got[sees][:, :, 3]).any() and (j != edge or 0 < sees.sum() < n)
        for rows, chans in ((~sees, slice(None)), (sees, np.arange(d) != 3)):
            assert np.all(np.abs(got[rows][..., chans] - ref[0][rows][..., chans]) <= bo[rows][..., chans])


@pytest.mark.parametrize("dtype,n,Hk,d", [("bf16", 4, 1, 64), ("bf16", 4, 2, 128), ("bf16", 90, 1, 64),
                                          ("bf16", 90, 2, 128), ("bf16", 90, 130, 128), ("f32", 4, 1, 64)])
def test_infinite_scores(torch, dtype, n, Hk, d):
    """A key whose score is -inf counts for nothing, as one that does not exist (the same bits); a row whose keys all
    are such sees nothing; a score of +inf makes the rows that see it NaN."""
    from chunk_gated_delta_carve_amd import paged_attention
    kv, page = 300, 4
    cu, lens, table, pages = ragged(torch, 14, 1, [n], [kv], page)
    kc, vc = cache(torch, "plain", pages, page, Hk, d, dtype, 118)
    q = rand(torch, 120, (n, Hk, d), dtype)
    q[..., 5] = 1.0
    args = (ints(torch, lens), ints(torch, cu))
    j = kv - n // 2 - 1                          # the first row does not see this key's page
    holes = table.copy()
    holes[0, [2, j // page]] = -1
    want = paged_attention(q, kc, vc, ints(torch, holes), *args, return_lse=True)
    low = kc.clone()
    low[table[0, [2, j // page]], ..., 5] = float("-inf")
    got = paged_attention(q, low, vc, ints(torch, table), *args, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.isfinite(got[0]).all()
    low[..., 5] = float("-inf")
    out, lse = paged_attention(q, low, vc, ints(torch, table), *args, return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    high = kc.clone()
    high[table[0, j // page], j % page, :, 5] = float("inf")
    out, lse = paged_attention(q, high, vc, ints(torch, table), *args, return_lse=True)
    sees = torch.arange(kv - n, kv, device="cuda") >= j
    assert out[sees].isnan().all() and lse[sees].isnan().all()
    plain = paged_attention(q, kc, vc, ints(torch, table), *args)
    ref = orc.paged_attention(f64(q), f64(kc), f64(vc), table, lens, cu, d ** -0.5, 0)
    bo, _ = attention_bounds(dtype, d, d ** -0.5, *ref)
    rows = ~sees.cpu().numpy()
    close("rows before it", out[~sees], ref[0][rows], bo[rows])
    close("without it", plain, ref[0], bo)


def test_rows_behind_the_last_sequence_are_left(torch):
    from chunk_gated_delta_carve_amd import paged_attention
    for n, extra in ((3, 5), (140, 9)):
        cu, lens, table, pages = ragged(torch, 12, 1, [n], [n], 16)
        kc, vc = cache(torch, "plain", pages, 16, 2, 64, "bf16", 110)
        q = rand(torch, 112, (n + extra, 4, 64), "bf16")
        out = torch.full_like(q, 5.0)
        paged_attention(q, kc, vc, ints(torch, table), ints(torch, lens), ints(torch, cu), out=out)
        assert (out[n:] == 5.0).all() and not (out[:n] == 5.0).all()


@pytest.mark.parametrize("case", [
    # dtype, Hq, Hk, d, page, sequences, window, step: more sequences than a wave has lanes
    ("bf16", 4, 2, 64, 16, 150, 0, True),
    ("bf16", 4, 2, 128, 16, 70, 20, False),
    ("bf16", 8, 1, 64, 32, 90, 0, False),
    ("f32", 2, 2, 64, 16, 129, 0, False),
    ("bf16", 2, 2, 64, 16, 1500, 0, True),
], ids=["step", "ragged", "tiles", "f32", "more"])
def test_many_sequences(torch, case):
    from chunk_gated_delta_carve_amd import paged_append, paged_attention
    dtype, Hq, Hk, d, page, S, window, step = case
    rng = np.random.default_rng(18)
    top = 14 if Hq // Hk < 8 else 60
    n = [1] * S if step else list(rng.integers(0, top, S))
    kv = [int(x + rng.integers(0, 90)) if x else 0 for x in n]
    cu, lens, table, pages = ragged(torch, 19, S, n, kv, page)
    kc, vc = cache(torch, "plain", pages, page, Hk, d, dtype, 190)
    N = sum(n)
    q, k, v = (rand(torch, 192 + i, (N, h, d), dtype) for i, h in enumerate((Hq, Hk, Hk)))
    args = (ints(torch, table), ints(torch, lens), None if step else ints(torch, cu))
    before = f64(kc), f64(vc)
    paged_append(k, v, kc, vc, *args)
    ref = orc.paged_append(f64(k), f64(v), *before, table, lens, cu, page)
    assert np.array_equal(f64(kc), ref[0]) and np.array_equal(f64(vc), ref[1])
    out, lse = paged_attention(q, kc, vc, *args, window=window, return_lse=True)
    check_attention(torch, out, lse, q, kc, vc, table, lens, cu, d ** -0.5, window, dtype)


@pytest.mark.parametrize("dtype,d,n,growth,Hk", [
    ("bf16", 64, 1, 3.0, 1), ("bf16", 128, 3, 12.0, 1), ("f32", 64, 2, 3.0, 1), ("bf16", 64, 100, 3.0, 1),
    ("bf16", 128, 100, 0.5, 1), ("bf16", 128, 100, 12.0, 1), ("bf16", 64, 100, -3.0, 1), ("bf16", 128, 100, 0.5, 66),
    ("bf16", 128, 100, 12.0, 66), ("bf16", 128, 100, -3.0, 66)])
def test_scores_that_grow_along_the_context(torch, dtype, d, n, growth, Hk):
    """Scores that rise (or fall) by `growth` every 64 keys: the reference of the running softmax follows in small
    steps, in large ones, or stays."""
    from chunk_gated_delta_carve_amd import paged_attention
    kv = 700
    cu, lens, table, pages = ragged(torch, 20, 1, [n], [kv], 16)
    kc, vc = cache(torch, "plain", pages, 16, Hk, d, dtype, 200)
    q = rand(torch, 202, (n, 4 * Hk, d), dtype, 0.3)
    q[..., 0] = 4.0
    j = torch.arange(len(table[0]) * 16, device="cuda").view(-1, 16)
    kc[ints(torch, table[0]).long(), :, :, 0] = (j * (growth / 64 / 4)).to(kc.dtype)[..., None]
    out, lse = paged_attention(q, kc, vc, ints(torch, table), ints(torch, lens), ints(torch, cu), scale=1.0,
                               return_lse=True)
    check_attention(torch, out, lse, q, kc, vc, table, lens, cu, 1.0, 0, dtype)


def test_extreme_scores(torch):
    """One weight of 1 and the rest 0; scores far beyond what fp32 exponentials reach, at the largest scale."""
    from chunk_gated_delta_carve_amd import paged_attention
    for dtype, n in (("bf16", 2), ("bf16", 90), ("f32", 2)):
        cu, lens, table, pages = ragged(torch, 21, 1, [n], [200], 16)
        kc, vc = cache(torch, "plain", pages, 16, 1, 64, dtype, 210)
        q = rand(torch, 212, (n, 2, 64), dtype, 3.0)
        out, lse = paged_attention(q, kc * 3, vc, ints(torch, table), ints(torch, lens), ints(torch, cu), scale=16.0,
                                   return_lse=True)
        ref = orc.paged_attention(f64(q), f64(kc * 3), f64(vc), table, lens, cu, 16.0, 0)
        # the score error e moves weight between values that differ by up to 2 max|v|, where the mean of |v| that
        # the bound counts can be small
        bo, bl = attention_bounds(dtype, 64, 16.0, *ref)
        close("lse", lse, ref[1], bl)
        close("o", out, ref[0], bo + 2 * np.abs(bl)[..., None] * np.max(np.abs(f64(vc))))


def test_offsets_past_32_bits(torch):
    """Pages whose elements lie past 2^31 (and bytes past 2^32) of a cache of 2.3 * 10^9 elements."""
    from chunk_gated_delta_carve_amd import paged_append, paged_attention
    page, Hk, d = 64, 4, 128
    pages = 71000
    kc = torch.empty(pages, page, Hk, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    assert kc.numel() > 2 ** 31
    small = list(range(pages - 6, pages))
    for c, seed in ((kc, 220), (vc, 221)):
        c[small] = rand(torch, seed, (6, page, Hk, d), "bf16")
    for n, kv in ((1, 300), (70, 300)):
        table = np.array([[pages - 1, pages - 5, pages - 3, pages - 2, pages - 6]])
        lens, cu = ints(torch, [kv]), ints(torch, [0, n])
        q, k, v = (rand(torch, 222 + i, (n, h, d), "bf16") for i, h in enumerate((8, Hk, Hk)))
        paged_append(k, v, kc, vc, ints(torch, table), lens, cu)
        out, lse = paged_attention(q, kc, vc, ints(torch, table), lens, cu, return_lse=True)
        lo = table - (pages - 6)                 # the same six pages as a cache of their own
        assert torch.equal(kc[int(table[0, (kv - 1) // page]), (kv - 1) % page], k[-1])
        check_attention(torch, out, lse, q, kc[small], vc[small], lo, [kv], [0, n], d ** -0.5, 0, "bf16")


def test_calls_on_two_streams(torch):
    """Two calls under way at once, each with a workspace of its own, have the bits of calls one by one."""
    from chunk_gated_delta_carve_amd import paged_attention
    calls = []
    for seed, (n, kv, d) in enumerate(((1, 9000, 128), (200, 4000, 64))):
        cu, lens, table, pages = ragged(torch, 23 + seed, 2, [n, n], [kv, kv - 7], 16)
        kc, vc = cache(torch, "plain", pages, 16, 2, d, "bf16", 230 + 2 * seed)
        calls.append((rand(torch, 235 + seed, (2 * n, 8, d), "bf16"), kc, vc, ints(torch, table), ints(torch, lens),
                      ints(torch, cu)))
    want = [paged_attention(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = [paged_attention(*c, stream=s) for c, s in zip(calls, streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_strided_queries_and_outputs(torch):
    """q as a part of one projection's output, o into a part of a wider tensor, a table that is a slice."""
    from chunk_gated_delta_carve_amd import paged_attention
    n, kv = 37, 61
    cu, lens, table, pages = ragged(torch, 13, 1, [n], [kv], 16)
    kc, vc = cache(torch, "plain", pages, 16, 2, 64, "bf16", 120)
    wide = rand(torch, 122, (n, 9, 64), "bf16")
    room = torch.zeros(n, 10, 64, dtype=torch.bfloat16, device="cuda")
    big = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
    big[0, :table.shape[1]] = ints(torch, table[0])
    args = (ints(torch, lens), ints(torch, cu))
    a = paged_attention(wide[:, 3:7], kc, vc, big[:1, :table.shape[1]], *args, out=room[:, 2:6])
    b = paged_attention(wide[:, 3:7].contiguous(), kc, vc, ints(torch, table), *args)
    assert torch.equal(a, b) and not room[:, :2].any() and not room[:, 6:].any()


def test_refusals(torch):
    from chunk_gated_delta_carve_amd import paged_append, paged_attention, qk_norm_rope_fwd, rope_tables
    from chunk_gated_delta_carve_amd._lib import CarveError
    kc, vc = cache(torch, "plain", 4, 16, 2, 64, "bf16", 130)
    q, table, lens, cu = rand(torch, 131, (3, 4, 64), "bf16"), ints(torch, [[0, 1]]), ints(torch, [20]), ints(torch, [0, 3])
    k = q[:, :2]
    for err, call in [
        (ValueError, lambda: paged_attention(q.cpu(), kc, vc, table, lens, cu)),
        (ValueError, lambda: paged_attention(q.half(), kc, vc, table, lens, cu)),
        (ValueError, lambda: paged_attention(q.float(), kc, vc, table, lens, cu)),
        (ValueError, lambda: paged_attention(q, kc, vc, table, lens)),                      # 3 tokens, 1 sequence
        (ValueError, lambda: paged_attention(q, kc, vc, table.long(), lens, cu)),
        (ValueError, lambda: paged_attention(q, kc, vc, table, lens, cu[:1])),
        (ValueError, lambda: paged_attention(q, kc, vc[:3], table, lens, cu)),
        (ValueError, lambda: paged_attention(q, kc, vc, table, lens, cu, out=q[:2])),
        (ValueError, lambda: paged_attention(q.transpose(0, 1).contiguous().transpose(0, 1), kc, vc, table, lens, cu)),
        (CarveError, lambda: paged_attention(q, kc, vc, table, lens, cu, out=q)),
        (CarveError, lambda: paged_attention(q, kc, vc, table, lens, cu, scale=0.0)),
        (CarveError, lambda: paged_attention(q, kc, vc, table, lens, cu, window=-1)),
        (CarveError, lambda: paged_attention(q[:, :3], kc, vc, table, lens, cu)),           # 3 heads over 2
        (CarveError, lambda: paged_attention(q[..., :32].contiguous(), kc[..., :32], vc[..., :32], table, lens, cu)),
        (CarveError, lambda: paged_append(k, k, kc[:, :12], vc[:, :12], table, lens, cu)),  # 12 tokens a page
        (ValueError, lambda: paged_append(k, k, kc, vc, table, lens, cu, k_weight=kc[0, 0, 0])),
        (CarveError, lambda: paged_append(k, k, kc, kc, table, lens, cu)),
        (ValueError, lambda: qk_norm_rope_fwd(q, k[:2])),
        (ValueError, lambda: qk_norm_rope_fwd(q, k, torch.ones(4, 32, device="cuda"))),
        (ValueError, lambda: qk_norm_rope_fwd(q, k, *rope_tables(8, 64), positions=torch.arange(3, device="cuda"))),
        (CarveError, lambda: qk_norm_rope_fwd(q, k, *(t[:, :12].contiguous() for t in rope_tables(8, 64)))),
    ]:
        with pytest.raises(err):
            call()


# as they are used

def test_prompt_chunks_then_single_tokens(torch):
    """A prompt appended and attended in ragged chunks, then token by token, against the whole sequence at once."""
    from chunk_gated_delta_carve_amd import paged_append, paged_attention, rope_tables
    Hq, Hk, d, page, T = 12, 4, 64, 16, 150
    cuts = [[0, 70, 71, 140, 150], [0, 33, 100, 149, 150]]         # two sequences, four calls; then nothing but steps
    steps = 5
    q, k, v = (rand(torch, 140 + i, (2, T + steps, h, d), "bf16", 1.5) for i, h in enumerate((Hq, Hk, Hk)))
    wq, wk = (rand(torch, 143 + i, (d,), "bf16", 0.2, 1.0) for i in range(2))
    cos, sin = rope_tables(T + steps, d)
    _, _, table, pages = ragged(torch, 14, 2, [1, 1], [T + steps] * 2, page)
    kc, vc = cache(torch, "joint", pages, page, Hk, d, "bf16", 145)
    tab = ints(torch, table)
    kw = dict(cos=cos, sin=sin, q_weight=wq, k_weight=wk, norm=True)
    o = torch.zeros_like(q)
    qs = torch.zeros_like(q)
    for i in range(4 + steps):
        span = [(c[i], c[i + 1]) if i < 4 else (T + i - 4, T + i - 3) for c in cuts]
        pick = lambda t: torch.cat([t[s, a:b] for s, (a, b) in enumerate(span)])  # noqa: E731
        lens = ints(torch, [b for _, b in span])
        cu = None if i >= 4 else ints(torch, np.concatenate([[0], np.cumsum([b - a for a, b in span])]))
        qr = paged_append(pick(k), pick(v), kc, vc, tab, lens, cu, q=pick(q), **kw)
        out = paged_attention(qr, kc, vc, tab, lens, cu)
        at = 0
        for s, (a, b) in enumerate(span):
            o[s, a:b], qs[s, a:b] = out[at:at + b - a], qr[at:at + b - a]
            at += b - a
    from chunk_gated_delta_carve_amd import qk_norm_rope_fwd
    q2, k2 = qk_norm_rope_fwd(q, k, cos, sin, q_weight=wq, k_weight=wk)
    assert torch.equal(q2, qs)                                       # the same arithmetic in both entry points
    for s in range(2):
        rows = kc[tab[s].long()].flatten(0, 1)[:T + steps]
        assert torch.equal(rows, k2[s])
    lens = np.full(2, T + steps)
    check = orc.paged_attention(f64(qs.flatten(0, 1)), f64(kc), f64(vc), table, lens, [0, T + steps, 2 * (T + steps)],
                                d ** -0.5, 0)
    bo, _ = attention_bounds("bf16", d, d ** -0.5, *check)
    close("o", o.flatten(0, 1), check[0], bo)


def test_hybrid_block_prompt_and_decode(torch):
    """A mixer layer feeding a sliding-window attention layer: the prompt as one chunk through chunk_fwd and
    paged_attention, then tokens through recurrent_step and the same attention call, against the whole run at once."""
    from chunk_gated_delta_carve_amd import chunk_fwd, paged_append, paged_attention, recurrent_step, rope_tables
    B, H, d, T, steps, window, L = 2, 4, 64, 128, 6, 48, 64
    x = {n: rand(torch, 150 + i, (B, T + steps, H, d), "bf16") for i, n in enumerate(("q", "k", "v", "g", "bx"))}
    for n in "qk":
        x[n] = (x[n].float() / x[n].float().norm(dim=-1, keepdim=True)).bfloat16()
    x["g"] = -torch.nn.functional.softplus(x["g"].float()).bfloat16()
    w = torch.sigmoid(rand(torch, 156, (B, T + steps, H), "f32")).bfloat16()
    cos, sin = rope_tables(T + steps, d)
    _, _, table, pages = ragged(torch, 15, B, [1, 1], [T + steps] * B, 16)
    kc, vc = cache(torch, "plain", pages, 16, H, d, "bf16", 157)
    tab = ints(torch, table)

    def attend(y, t0):                           # y [B, n, H, d] at positions t0 ..
        n = y.shape[1]
        lens, cu = ints(torch, [t0 + n] * B), None if n == 1 else ints(torch, np.arange(B + 1) * n)
        y = y.reshape(B * n, H, d)
        qr = paged_append(y, y, kc, vc, tab, lens, cu, cos, sin, q=y, norm=True)
        return paged_attention(qr, kc, vc, tab, lens, cu, window=window).view(B, n, H, d), qr

    part = lambda a, b: [x[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "bx")] + [w[:, a:b].contiguous()]  # noqa: E731
    y, S, m = chunk_fwd(*part(0, T), L=L, return_state=True)
    ys, outs, qrs = [y], [], []
    o, qr = attend(y, 0)
    outs.append(o)
    qrs.append(qr.view(B, T, H, d))
    acc = torch.zeros_like(m)
    for t in range(T, T + steps):
        y = recurrent_step(*(a[:, 0].contiguous() for a in part(t, t + 1)), S, m, acc, (t - T) % L, L)[:, None]
        ys.append(y)
        o, qr = attend(y.contiguous(), t)
        outs.append(o)
        qrs.append(qr.view(B, 1, H, d))
    o, qr = torch.cat(outs, 1), torch.cat(qrs, 1)
    ref = orc.paged_attention(f64(qr.flatten(0, 1)), f64(kc), f64(vc), table, [T + steps] * B,
                              np.arange(B + 1) * (T + steps), d ** -0.5, window)
    bo, _ = attention_bounds("bf16", d, d ** -0.5, *ref)
    close("o", o.flatten(0, 1), ref[0], bo)
    rows = vc[tab[0].long()].flatten(0, 1)[:T + steps]
    assert torch.equal(rows, torch.cat(ys, 1)[0])


def test_captured_step_follows_the_lengths(torch):
    """A decode step captured once and replayed as the sequences grow, with eager work in between; two captured
    graphs that share one workspace run one after the other."""
    from chunk_gated_delta_carve_amd import paged_append, paged_attention, paged_workspace_bytes, rope_tables
    S, Hq, Hk, d, page, width = 3, 16, 2, 128, 16, 64
    kc, vc = cache(torch, "plain", S * width, page, Hk, d, "bf16", 160)
    tab = torch.arange(S * width, dtype=torch.int32, device="cuda").view(S, width)
    lens = ints(torch, [100, 700, 5])
    cos, sin = rope_tables(1024, d)
    q, k, v = (rand(torch, 161 + i, (S, h, d), "bf16") for i, h in enumerate((Hq, Hk, Hk)))
    ws = torch.empty(paged_workspace_bytes(S, S, Hq, Hk, d, page, width, step=True), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    outs = [torch.empty_like(q) for _ in range(2)]

    def step(out, window):
        qr = paged_append(k, v, kc, vc, tab, lens, cos=cos, sin=sin, q=q, norm=True)
        return paged_attention(qr, kc, vc, tab, lens, out=out, window=window, workspace=ws)

    step(outs[0], 0)
    step(outs[1], 200)
    torch.cuda.synchronize()
    graphs = []
    for i, window in enumerate((0, 200)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(outs[i], window)
        graphs.append(g)
    for turn in range(4):
        lens.add_(turn)
        q.copy_(rand(torch, 170 + turn, (S, Hq, d), "bf16"))
        for g in graphs:
            g.replay()
        got = [o.clone() for o in outs]
        want = [step(torch.empty_like(q), window) for window in (0, 200)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), turn


def test_another_stream(torch):
    """Calls on a stream that is not the current one: temporaries are that stream's, results are ordered with it."""
    from chunk_gated_delta_carve_amd import paged_attention
    cu, lens, table, pages = ragged(torch, 17, 1, [1], [5000], 16)
    kc, vc = cache(torch, "plain", pages, 16, 2, 64, "bf16", 180)
    q = rand(torch, 182, (1, 4, 64), "bf16")
    args = (q, kc, vc, ints(torch, table), ints(torch, lens))
    want = paged_attention(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for handle in (s, s.cuda_stream):
        out = torch.empty_like(q)
        got = [paged_attention(*args, stream=handle) for _ in range(3)]
        paged_attention(*args, stream=handle, out=out)
        s.synchronize()
        for g in (*got, out):
            assert torch.equal(g, want)
    with torch.cuda.stream(s):                   # 0 is the default stream, whichever is current
        got = paged_attention(*args, stream=0)
        assert torch.cuda.current_stream() == s
    torch.cuda.default_stream().synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("dtype,n,kv,Hq,Hk,d", [("f32", [700, 3, 150], [700, 900, 400], 4, 2, 64),
                                                ("f32", [333], [333], 4, 1, 128),
                                                ("bf16", [150] + [1] * 30, [400] + [90] * 30, 2, 2, 64)])
def test_prompts_of_the_row_kernel(torch, dtype, n, kv, Hq, Hk, d, window):
    """Many items to a sequence, whose rows see very different parts of it."""
    from chunk_gated_delta_carve_amd import paged_attention
    cu, lens, table, pages = ragged(torch, 30, len(n), n, kv, 16)
    kc, vc = cache(torch, "plain", pages, 16, Hk, d, dtype, 290)
    q = rand(torch, 292, (sum(n), Hq, d), dtype)
    out, lse = paged_attention(q, kc, vc, ints(torch, table), ints(torch, lens), ints(torch, cu), window=window,
                               return_lse=True)
    check_attention(torch, out, lse, q, kc, vc, table, lens, cu, d ** -0.5, window, dtype)


def test_a_windowed_prompt_of_half_a_million_tokens(torch):
    """2^31 blocks of 128 keys if every 16 rows had their sequence's; with the window they have four each."""
    from chunk_gated_delta_carve_amd import paged_attention
    N, Hq, Hk, d, page, window = 524288, 16, 4, 64, 64, 256
    g = torch.Generator(device="cuda").manual_seed(300)
    q = torch.randn(N, Hq, d, generator=g, device="cuda")
    kc, vc = (torch.randn(N // page, page, Hk, d, generator=g, device="cuda") for _ in range(2))
    table = torch.randperm(N // page, generator=g, device="cuda").to(torch.int32)[None]
    out = torch.full_like(q, float("nan"))
    _, lse = paged_attention(q, kc, vc, table, ints(torch, [N]), ints(torch, [0, N]), window=window, out=out,
                             return_lse=True)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    for r in (0, 200, 255, 256, 70001, N // 2, N - 1):
        t0 = max(0, r - window + 1) // page
        part = table[0, t0:r // page + 1].long()
        o, l, A, reach, keys = orc.paged_attention(f64(q[r:r + 1]), f64(kc[part]), f64(vc[part]),
                                                   np.arange(len(part))[None], [r - t0 * page + 1], [0, 1], d ** -0.5,
                                                   window)
        bo, bl = attention_bounds("f32", d, d ** -0.5, o, l, A, reach, keys)
        close(f"row {r}", out[r:r + 1], o, bo)
        assert np.all(np.abs(f64(lse[r:r + 1]) - l) <= bl)


@pytest.mark.parametrize("n,Hq,Hk,d,stride", [(1, 4, 2, 64, 310_000_000), (100, 4, 2, 64, 310_000_000),
                                              (100, 4, 2, 128, 720_000_000), (40, 130, 130, 128, 720_000_000)])
def test_tokens_far_apart(torch, n, Hq, Hk, d, stride):
    """A token-major pool [page_size, pages, Hk, d] whose token stride is so wide that the eight tokens of a page span
    more than 2^32 bytes: the bits of the same call on a cache of its own."""
    from chunk_gated_delta_carve_amd import paged_append, paged_attention
    kv, page = 120, 8
    cu, lens, table, pages = ragged(torch, 24, 1, [n], [kv], page)
    entry = pages * Hk * d
    pool = torch.empty((page - 1) * stride + 2 * entry, dtype=torch.bfloat16, device="cuda")
    far = [pool.as_strided((pages, page, Hk, d), (Hk * d, stride, d, 1), i * entry) for i in range(2)]
    near = cache(torch, "plain", pages, page, Hk, d, "bf16", 240)
    for a, b in zip(far, near):
        a.copy_(b)
    q, k, v = (rand(torch, 242 + i, (n, h, d), "bf16") for i, h in enumerate((Hq, Hk, Hk)))
    args = (ints(torch, table), ints(torch, lens), ints(torch, cu))
    for c in (far, near):
        paged_append(k, v, *c, *args)
    assert all(torch.equal(a, b) for a, b in zip(far, near))
    got = paged_attention(q, *far, *args, return_lse=True)
    want = paged_attention(q, *near, *args, return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_attention(torch, *got, q, *near, table, lens, cu, d ** -0.5, 0, "bf16")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,n,kv,Hk,d", [
    ("bf16", 4, 300, 1, 64), ("bf16", 4, 300, 2, 128), ("bf16", 90, 300, 1, 64), ("bf16", 90, 300, 2, 128),
    ("bf16", 90, 300, 130, 128), ("f32", 4, 300, 1, 64), ("f32", 40, 300, 1, 128),
    ("bf16", 4, 4000, 1, 128), ("bf16", 100, 4000, 1, 64), ("f32", 4, 4000, 1, 64)])
def test_values_of_keys_that_count_for_nothing(torch, bad, dtype, n, kv, Hk, d):
    """A key whose score is -inf is not seen, so its value does not matter, infinities and NaN included; contexts in
    one piece and split ones."""
    from chunk_gated_delta_carve_amd import paged_attention
    page = 4
    cu, lens, table, pages = ragged(torch, 25, 1, [n], [kv], page)
    kc, vc = cache(torch, "plain", pages, page, Hk, d, dtype, 250)
    q = rand(torch, 252, (n, Hk, d), dtype)
    q[..., 5] = 1.0
    slots = [2, kv // 2 // page, (kv - n // 2) // page]
    gone = table[0, slots]
    kc[gone, ..., 5] = float("-inf")
    vc[gone] = bad
    out, lse = paged_attention(q, kc, vc, ints(torch, table), ints(torch, lens), ints(torch, cu), return_lse=True)
    holes = table.copy()
    holes[0, slots] = -1
    check_attention(torch, out, lse, q, kc, vc, holes, lens, cu, d ** -0.5, 0, dtype)


@pytest.mark.parametrize("dtype,n,kv,Hk,d", [
    ("bf16", 4, 300, 1, 64), ("bf16", 4, 300, 2, 128), ("bf16", 90, 300, 1, 64), ("bf16", 90, 300, 2, 128),
    ("bf16", 90, 300, 130, 128), ("f32", 4, 300, 1, 64), ("f32", 40, 300, 1, 128),
    ("bf16", 4, 4000, 1, 128), ("bf16", 100, 4000, 1, 64), ("f32", 4, 4000, 1, 64)])
@pytest.mark.parametrize("size,sign", [(2.0 ** e, sign) for e in (18, 30, 50, 63) for sign in (1, -1)])
def test_scores_of_any_finite_size(torch, size, sign, dtype, n, kv, Hk, d):
    """Scores q k of one channel between 2^36 and 2^128, all of one sign: neighbours differ by more than any weight
    survives, so a row is the value of its highest key and lse is that key's scaled score. The products of two 8-bit
    factors are exact in fp32. o: half a step for a weight that is not exactly 1 (bf16, tiles) and half a step for the
    output, 2^-22 for the division. lse: a scale of 24 bits, the weight's own error of at most 2^-24 of the score, a
    logarithm and a sum make less than 2^-22 of it."""
    from chunk_gated_delta_carve_amd import paged_attention
    cu, lens, table, pages = ragged(torch, 26, 1, [n], [kv], 16)
    kc, vc = cache(torch, "plain", pages, 16, Hk, d, dtype, 260)
    vc = vc.bfloat16().to(vc.dtype)
    rng = np.random.default_rng(27)
    steps = rng.integers(0, 120, kv)             # the highest key stands out by at least 2^-8 of itself
    q = torch.zeros(n, Hk, d, dtype=dt(torch, dtype), device="cuda")
    q[..., 3] = size * torch.tensor(1 + rng.integers(0, 64, n) / 128, dtype=torch.float32).to(q)[:, None]
    best = int(rng.integers(0, kv - n))           # every row sees it
    steps[best] = 127 if sign > 0 else -1
    cells = np.zeros(len(table[0]) * 16, np.float32)
    cells[:kv] = sign * size * (1 + (steps if sign > 0 else steps + 1) / 128.0)
    kc.zero_()
    kc[ints(torch, table[0]).long(), :, :, 3] = torch.tensor(cells, device="cuda").view(-1, 16)[..., None].to(kc.dtype)
    out, lse = paged_attention(q, kc, vc, ints(torch, table), ints(torch, lens), ints(torch, cu), return_lse=True)
    row = vc[table[0, best // 16], best % 16].double()            # [Hk, d]
    assert torch.all((out.double() - row).abs() <= (2.1 * HALF[dtype] + 2.0 ** -22) * row.abs())
    want = q[..., 3].double() * kc[table[0, best // 16], best % 16, :, 3].double() * d ** -0.5
    assert torch.all((lse.double() - want).abs() <= 2.0 ** -22 * want.abs())


@pytest.mark.parametrize("dtype,n,d", [("bf16", 1, 64), ("bf16", 100, 64), ("bf16", 100, 128), ("f32", 3, 128)])
def test_a_window_wider_than_any_table(torch, dtype, n, d):
    """Lengths far past the table with windows above 2^30: the keys in the table that the windows reach are seen."""
    from chunk_gated_delta_carve_amd import paged_attention
    width, page, pages = 8, 16, 8
    kc, vc = cache(torch, "plain", pages, page, 2, d, dtype, 270)
    q = rand(torch, 272, (n, 4, d), dtype)
    table, cu = np.random.default_rng(28).permutation(pages)[None], [0, n]
    for kv, window in ((2 ** 30 + 200, 2 ** 30 + 50), (2 ** 30 + 100, 2 ** 30 + 50), (2 ** 31 - 1, 2 ** 31 - 1),
                       (2 ** 31 - 1, 2 ** 31 - 60), (50, 2 ** 31 - 1), (5, 2 ** 31 - 1)):
        out, lse = paged_attention(q, kc, vc, ints(torch, table), ints(torch, [kv]), ints(torch, cu), window=window,
                                   return_lse=True)
        # the same rows one by one over the part of the table that each sees
        want, wl = np.zeros((n, 4, d)), np.full((n, 4), -np.inf)
        bo, bl = np.zeros((n, 4, d)), np.zeros((n, 4))
        for i in range(n):
            p = kv - n + i
            seen = [j for j in range(max(0, p - window + 1), min(p + 1, width * page))]
            if not seen:
                continue
            o, l, A, reach, keys = orc.paged_attention(
                f64(q[i:i + 1]), *(f64(c[table[0]]).reshape(1, width * page, 2, d)[:, seen] for c in (kc, vc)),
                np.array([[0]]), [len(seen)], [0, 1], d ** -0.5, 0)
            want[i], wl[i] = o[0], l[0]
            b = attention_bounds(dtype, d, d ** -0.5, o, l, A, reach, keys)
            bo[i], bl[i] = b[0][0], b[1][0]
        close("o", out, want, bo)
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(f64(lse)), empty) and (kv == 2 ** 30 + 200 or not empty.all())
        assert np.all(np.abs(f64(lse)[~empty] - wl[~empty]) <= bl[~empty])


# the forms that large calls take: several pieces to a lane, several trips of the gradient's loop

MANY = [
    # as ROPE; waves take 2, 3, 3 (two waves to a token), 4, 4, 3 and 3 pieces a lane
    ("bf16", (20, 150), 12, 4, 64, 64, False, True, True, False),
    ("bf16", (1500,), 16, 4, 64, 32, True, True, True, True),
    ("bf16", (901,), 16, 2, 128, 128, False, True, True, True),
    ("bf16", (7, 160), 17, 13, 64, 48, False, True, False, False),
    ("f32", (11, 100), 12, 4, 64, 64, False, True, True, False),
    ("f32", (1401,), 5, 1, 128, 128, True, True, True, True),
    ("f32", (1399,), 3, 2, 128, 64, False, False, False, True),
]
MANY_IDS = ["-".join(str(x).replace(" ", "") for x in c) for c in MANY]


@pytest.mark.parametrize("case", MANY, ids=MANY_IDS)
def test_norm_rope_of_many_tokens(torch, case):
    test_norm_rope(torch, case)


# 1024 blocks take 32, 16 or 8 rows a trip (16 and 32 lanes a row): two trips and more here
MANY_ROWS = [("bf16", (20, 150), 12, 12, 64, 64, False, True, True, False),
             ("bf16", (1401,), 16, 4, 128, 128, False, True, True, True),
             ("bf16", (9, 199), 20, 1, 64, 32, True, True, True, False),
             ("f32", (1201,), 12, 4, 64, 64, True, True, True, True),
             ("f32", (13, 100), 12, 4, 128, 96, False, True, True, False),
             ("f32", (1300,), 8, 2, 128, 128, False, False, False, True)]


@pytest.mark.parametrize("case", MANY_ROWS, ids=["-".join(str(x).replace(" ", "") for x in c) for c in MANY_ROWS])
def test_norm_rope_gradient_of_many_rows(torch, case):
    test_norm_rope_gradient(torch, case)


MANY_NEW = [
    # as APPEND; 2, 3, 3 (two waves) and 4 pieces a lane
    ("bf16", 8, 4, 64, 16, [1200, 1, 900], [1300, 50, 900], 64, False, True, "plain", False),
    ("bf16", 0, 10, 64, 32, [1500], [1500], 32, True, False, "heads", False),
    ("bf16", 12, 3, 128, 64, [500, 420], [700, 420], 128, False, True, "joint", False),
    ("f32", 8, 4, 64, 16, [700, 411], [700, 600], 64, True, True, "plain", False),
    ("f32", 2, 2, 128, 16, [900, 500], [900, 700], 128, False, False, "heads", False),
]


@pytest.mark.parametrize("case", MANY_NEW, ids=[str(i) for i in range(len(MANY_NEW))])
def test_append_of_many_tokens(torch, case):
    test_append(torch, case)


@pytest.mark.parametrize("d,G,n,kv,page,window", [(64, 1, 1, 40, 16, 0), (64, 4, 3, 50, 4, 0), (128, 4, 1, 33, 16, 0),
                                                  (128, 2, 6, 90, 64, 40)])
def test_few_rows_keep_sixteen_bits_of_the_weights(torch, d, G, n, kv, page, window):
    """With few rows the weights enter the second product as two bf16 parts: what is left of a weight is at most half a
    step of half a step, 2^-16 of it. Small queries keep the scores' own error below that. Against outputs near 0, where
    the output's rounding is small, one part would show: 2^-9 of |v| over the root of the number of keys."""
    from chunk_gated_delta_carve_amd import paged_attention
    cu, lens, table, pages = ragged(torch, 33, 1, [n], [kv], page)
    kc, vc = cache(torch, "plain", pages, page, 2, d, "bf16", 330)
    q = rand(torch, 332, (n, 2 * G, d), "bf16", 0.05)
    out, lse = paged_attention(q, kc, vc, ints(torch, table), ints(torch, lens), ints(torch, cu), window=window,
                               return_lse=True)
    o, l, A, reach, keys = orc.paged_attention(f64(q), f64(kc), f64(vc), table, lens, cu, d ** -0.5, window)
    e = d ** -0.5 * (d + 4) * 2.0 ** -24 * reach + 2.0 ** -20
    slack = 2 * e + (keys[:, None] + 64) * 2.0 ** -24 + 2.0 ** -16
    close("o", out, o, HALF["bf16"] * np.abs(o) + slack[..., None] * A)
    assert np.all(np.abs(f64(lse) - l) <= e + (keys[:, None] + 64) * 2.0 ** -24 + 2.0 ** -22 * np.abs(l))
    # the bound tells the two apart: weights rounded to one part fail it
    s0 = f64(kc)[table[0]].reshape(-1, 2, d)[:kv], f64(vc)[table[0]].reshape(-1, 2, d)[:kv]
    p = kv - 1
    seen = slice(max(0, p - window + 1) if window else 0, kv)
    w = np.exp(d ** -0.5 * s0[0][seen, 0] @ f64(q)[-1, 0])
    one = f64(torch.tensor(w / w.max(), dtype=torch.float32).bfloat16())
    rough = one @ s0[1][seen, 0] / (w / w.max()).sum()
    assert np.any(np.abs(rough - o[-1, 0]) > HALF["bf16"] * np.abs(o[-1, 0]) + slack[-1, 0] * A[-1, 0])


@pytest.mark.parametrize("dtype,n,Hq,Hk,d,window", [("bf16", 100, 8, 2, 64, 0), ("bf16", 100, 8, 2, 128, 900),
                                                    ("bf16", 90, 130, 130, 128, 0), ("f32", 20, 4, 2, 64, 0)])
def test_captured_chunk_follows_the_lengths(torch, dtype, n, Hq, Hk, d, window):
    """A prompt chunk's append and attention, and the gradient of its rotation, captured once and replayed over longer
    and shorter contexts (in one piece, split, cut by the table), with eager work between the replays."""
    from chunk_gated_delta_carve_amd import paged_append, paged_attention, qk_norm_rope_bwd, rope_tables
    page, width = 16, 256
    kc, vc = cache(torch, "joint", width, page, Hk, d, dtype, 340)
    tab = torch.randperm(width, generator=torch.Generator().manual_seed(341)).to(torch.int32).cuda()[None]
    lens, cu = ints(torch, [n]), ints(torch, [0, n])
    cos, sin = rope_tables(width * page, d)
    q, k, v, dq, dk = (rand(torch, 342 + i, (n, h, d), dtype) for i, h in enumerate((Hq, Hk, Hk, Hq, Hk)))
    w = rand(torch, 347, (d,), dtype, 0.1, 1.0)

    def work():
        qr = paged_append(k, v, kc, vc, tab, lens, cu, cos, sin, q=q, q_weight=w, k_weight=w, norm=True)
        out, lse = paged_attention(qr, kc, vc, tab, lens, cu, window=window, return_lse=True)
        return [qr, out, lse, *qk_norm_rope_bwd(q, k, dq, dk, cos, sin, q_weight=w, k_weight=w).values()]

    work()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = work()
    for turn, kv in enumerate((n, 4000, n // 2, 700, width * page)):
        lens.fill_(kv)
        q.copy_(rand(torch, 350 + turn, (n, Hq, d), dtype))
        g.replay()
        got = [t.clone() for t in held]
        want = work()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)), (turn, kv, i)
        assert torch.isfinite(got[1]).all()
