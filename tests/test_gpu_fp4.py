"""The 4-bit paged cache and the room in a paged cache on the GPU, against oracle/fp4_oracle.py and, for attention over
the values that the codes stand for, oracle/attention_oracle.py.

Codes, scales, pages, slots and values read back are exact: equality. Attention has the bounds of test_gpu_attention.py
(its head says how they come about): codes are exact in bf16, so products and sums are those of the bf16 and fp32 caches.
"""
import numpy as np
import pytest

from oracle import attention_oracle as att
from oracle import fp4_oracle as orc
from test_gpu_attention import (ATTENTION, HALF, attention_bounds, check_attention, close, dt, f64, ints, ragged, rand,  # noqa: F401
                                row_max, say, torch)

pytestmark = pytest.mark.gpu


def u8(t):
    return t.cpu().numpy()


def tensor(torch, x):  # noqa: F811
    return torch.tensor(np.asarray(x), device="cuda")


def cache4(torch, layout, pages, page, Hk, d, seed, lo=122, hi=126):  # noqa: F811
    """A cache of random codes with scales 2^(lo - 127) .. 2^(hi - 128), in one of the layouts a program may keep."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def fill(t, a, b):
        t.copy_(torch.randint(a, b, t.shape, generator=g, device="cuda", dtype=torch.uint8))

    parts = []
    if layout == "plain":                        # tokens before heads
        parts = [torch.empty(pages, page, Hk, n, dtype=torch.uint8, device="cuda") for n in (d // 2, d // 32) * 2]
    elif layout == "joint":                      # a page's four parts in one allocation, page after page
        sizes = [Hk * page * n for n in (d // 2, d // 32) * 2]
        sizes = [-(-n // 16) * 16 for n in sizes]
        whole = torch.zeros(pages, sum(sizes), dtype=torch.uint8, device="cuda")
        at = 0
        for i, n in enumerate((d // 2, d // 32) * 2):
            parts.append(whole[:, at:at + Hk * page * n].view(pages, page, Hk, n))
            at += sizes[i]
    else:
        from chunk_gated_delta_carve_amd import paged_fp4_cache
        parts = list(paged_fp4_cache(pages, page, Hk, d))
    for i, t in enumerate(parts):
        fill(t, *((lo, hi) if i % 2 else (0, 256)))
    return tuple(parts)


def values(parts):
    """(k, v) of a whole cache in 64 bits."""
    kc, ks, vc, vs = (u8(t) for t in parts)
    return orc.decode(kc, ks), orc.decode(vc, vs)


# append

def inputs(torch, seed, N, H, d, dtype):  # noqa: F811
    """Rows whose blocks differ in size by powers of two."""
    x = rand(torch, seed, (N, H, d), dtype, 1.0)
    g = torch.Generator().manual_seed(seed + 1)
    size = torch.randint(-20, 20, (N, H, d // 32), generator=g).float().exp2().cuda().repeat_interleave(32, -1)
    return (x.float() * size).to(dt(torch, dtype))


def stored(before, table, lens, cu, page, k, v):
    """The four parts after the rows of k and v were stored."""
    after = [u8(t).copy() for t in before]
    count = 0
    for n, at in enumerate(att.token_places(cu, lens, len(k))):
        cell = None if at is None else att.place(table, at[0], at[1], page, len(after[0]))
        if cell is None:
            continue
        count += 1
        for i, x in ((0, k), (2, v)):
            after[i][cell], after[i + 1][cell] = orc.encode(x[n])
    return after, count


APPEND = [
    # dtype, Hk, d, page, n, kv, layout, step
    ("bf16", 4, 64, 16, [5, 0, 33, 1], [5, 7, 40, 100], "plain", False),
    ("bf16", 2, 128, 64, [100, 1], [163, 64], "joint", False),
    ("bf16", 4, 128, 16, [1] * 9, [1, 16, 17, 31, 32, 33, 200, 2, 48], "heads", True),
    ("bf16", 3, 64, 1, [3, 2], [4, 2], "plain", False),
    ("bf16", 1, 64, 256, [77], [300], "heads", False),
    ("f32", 4, 64, 16, [9, 14], [20, 14], "heads", False),
    ("f32", 3, 128, 32, [1, 1], [33, 1], "joint", True),
    ("f32", 1, 64, 8, [17], [17], "plain", False),
]


@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
def test_append(torch, case):  # noqa: F811
    from chunk_gated_delta_carve_amd import paged_append_fp4
    dtype, Hk, d, page, n, kv, layout, step = case
    say("case", case)
    cu, lens, table, pages = ragged(torch, 5, len(n), n, kv, page)
    parts = cache4(torch, layout, pages, page, Hk, d, 50)
    kv_new = inputs(torch, 51, sum(n), 2 * Hk, d, dtype)          # parts of one projection: strided tokens
    k, v = kv_new[:, :Hk], kv_new[:, Hk:]
    want, _ = stored(parts, table, lens, cu, page, f64(k), f64(v))
    assert paged_append_fp4(k, v, *parts, ints(torch, table), ints(torch, lens), None if step else ints(torch, cu)) is None
    for got, ref in zip(parts, want):
        assert np.array_equal(u8(got), ref)


@pytest.mark.parametrize("dtype,Hq,Hk,d,rot,inter,norm,weights", [
    ("bf16", 12, 4, 64, 64, False, True, True), ("bf16", 4, 2, 128, 32, True, True, False),
    ("f32", 6, 3, 128, 128, False, True, True), ("f32", 0, 2, 64, 16, True, False, False)])
def test_append_with_norm_and_rotation(torch, dtype, Hq, Hk, d, rot, inter, norm, weights):  # noqa: F811
    """The keys stored are those of qk_norm_rope_fwd, and so are the queries."""
    from chunk_gated_delta_carve_amd import paged_append_fp4, qk_norm_rope_fwd, rope_tables
    n, kv, page = [7, 1, 30], [90, 1, 30], 16
    cu, lens, table, pages = ragged(torch, 6, 3, n, kv, page)
    parts = cache4(torch, "heads", pages, page, Hk, d, 60)
    N = sum(n)
    q = rand(torch, 61, (N, max(Hq, 1), d), dtype, 1.5)
    k, v = rand(torch, 62, (N, Hk, d), dtype, 1.5), rand(torch, 63, (N, Hk, d), dtype)
    cos, sin = rope_tables(128, rot)
    kw = dict(norm=norm, interleaved=inter)
    wq, wk = (rand(torch, 64 + i, (d,), dtype, 0.3, 1.0) for i in range(2)) if weights else (None, None)
    pos = ints(torch, [p for _, p in att.token_places(cu, lens, N)])
    q2, k2 = qk_norm_rope_fwd(q, k, cos, sin, pos, wq, wk, **kw)
    want, _ = stored(parts, table, lens, cu, page, f64(k2), f64(v))
    out = paged_append_fp4(k, v, *parts, ints(torch, table), ints(torch, lens), ints(torch, cu), cos, sin,
                           q=q if Hq else None, q_weight=wq if Hq else None, k_weight=wk, **kw)
    for got, ref in zip(parts, want):
        assert np.array_equal(u8(got), ref)
    assert torch.equal(out, q2) if Hq else out is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_of_special_values(torch, dtype):  # noqa: F811
    """Ties, zeros of either sign, denormals, the ends of the range, infinities and NaN."""
    from chunk_gated_delta_carve_amd import paged_append_fp4, paged_read_fp4
    big = float(torch.finfo(dt(torch, dtype)).max)
    tiny = float(torch.finfo(dt(torch, dtype)).smallest_normal)
    rows = [[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], [0.0, -0.0], [tiny, -tiny / 4, tiny / 2, tiny * 0.75],
            [tiny * 0.25], [big, -big, big / 2, 1.0], [float("inf"), 1.0], [float("-inf")], [float("nan"), 2.0],
            [7.0625, 1.0, -1.0], [14.0, 0.5], [2.0 ** -125 * 7, 2.0 ** -126], [2.0 ** 127, 2.0 ** 125 * 1.75],
            [-7.0, -0.25, -0.75, -5.0], [6.5, -6.5, 0.125]]
    for scale in (1.0, 2.0 ** -40, 2.0 ** 33):
        x = torch.zeros(len(rows), 2, 64)
        for i, r in enumerate(rows):
            x[i, i % 2, 32 * (i % 2):32 * (i % 2) + len(r)] = torch.tensor(r) * (scale if i < 2 else 1.0)
        x = x.to(dt(torch, dtype)).cuda()
        N = len(rows)
        parts = cache4(torch, "plain", 2, 16, 2, 64, 70)
        args = (ints(torch, [[1]]), ints(torch, [N]), ints(torch, [0, N]))
        paged_append_fp4(x, x, *parts, *args)
        codes, scales = orc.encode(f64(x))
        for i in (0, 2):
            assert np.array_equal(u8(parts[i])[1, :N], codes) and np.array_equal(u8(parts[i + 1])[1, :N], scales)
        k, v = paged_read_fp4(*parts, tensor(torch, np.arange(16, 16 + N)), dtype=torch.float32)
        assert np.array_equal(f64(k), orc.decode(codes, scales), equal_nan=True) and np.isfinite(f64(k)).sum() > 0


def test_append_drops_what_has_no_place(torch):  # noqa: F811
    """Negative positions, positions past the table, page numbers outside the cache and tokens behind the last
    sequence leave the cache (and q_out of the latter) as they were."""
    from chunk_gated_delta_carve_amd import paged_append_fp4
    page, Hk, d, pages = 16, 2, 64, 5
    n, kv = [4, 4, 20, 3], [2, 64, 20, 3]        # two negative positions; past the table; through bad pages; good
    cu = np.concatenate([[0], np.cumsum(n)])
    table = np.array([[0, -1], [1, 2], [-5, 99], [3, 4]])
    N = sum(n) + 6
    parts = cache4(torch, "plain", pages, page, Hk, d, 80)
    k, v, q = (rand(torch, 81 + i, (N, Hk, d), "bf16") for i in range(3))
    want, count = stored(parts, table, kv, cu, page, f64(k), f64(v))
    assert count == 2 + 3
    out = torch.full_like(q, 7.0)
    paged_append_fp4(k, v, *parts, ints(torch, table), ints(torch, kv), ints(torch, cu), q=q, q_out=out)
    for got, ref in zip(parts, want):
        assert np.array_equal(u8(got), ref)
    assert torch.equal(out[:31], q[:31]) and (out[31:] == 7.0).all()


@pytest.mark.parametrize("dtype,Hk,d,N", [("bf16", 16, 128, 3001), ("bf16", 1, 64, 9003), ("f32", 5, 64, 9003),
                                          ("bf16", 3, 128, 9003), ("f32", 1, 128, 5003), ("bf16", 3, 128, 3001)])
def test_append_and_read_many_tokens(torch, dtype, Hk, d, N):  # noqa: F811
    """Enough tokens for several pieces to a lane and several tokens to a wave, sequences that end inside of one's:
    what is read back is what one token at a time stores."""
    from chunk_gated_delta_carve_amd import paged_append_fp4, paged_read_fp4
    page = 16
    n = [1999, 1, 0, 2, N - 2002]
    cu, lens, table, pages = ragged(torch, 8, 5, n, [2100, 1, 0, 33, N - 2002], page)
    parts = cache4(torch, "heads", pages, page, Hk, d, 90)
    k, v = inputs(torch, 91, N, Hk, d, dtype), inputs(torch, 93, N, Hk, d, dtype)
    paged_append_fp4(k, v, *parts, ints(torch, table), ints(torch, lens), ints(torch, cu))
    at = [(s, int(lens[s]) - n[s] + i) for s in range(5) for i in range(n[s])]
    slots = np.array([table[s, p // page] * page + p % page for s, p in at])
    got = paged_read_fp4(*parts, tensor(torch, slots), dtype=dt(torch, dtype))
    rows = np.r_[0:40, 1990:2010, N - 20:N]
    for a, x in zip(got, (k, v)):
        y = orc.decode(*orc.encode(f64(x[rows])))
        assert np.array_equal(f64(a[rows]), y)
        # every row: a scale s has max > 3.5 s, and a value is off by at most s
        top = x.float().abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True)
        off = (a.float() - x.float()).abs().unflatten(-1, (-1, 32))
        assert (off <= top * (2 / 7)).all()


@pytest.mark.parametrize("S,N,behind", [(64, 4500, 5), (65, 4500, 0), (300, 6000, 3), (1, 4200, 9), (63, 4301, 1)])
def test_append_of_many_tokens_of_many_sequences(torch, S, N, behind):  # noqa: F811
    """Waves whose tokens belong to several sequences, empty ones among them: as many as a wave has lanes, and more."""
    from chunk_gated_delta_carve_amd import paged_append_fp4, paged_read_fp4
    page, Hk, d = 8, 1, 64
    rng = np.random.default_rng(S)
    share = rng.random(S) ** 4 * (rng.random(S) < 0.6)
    share[S // 2] = 0.2
    n = np.floor(share / share.sum() * N).astype(int)
    n[np.argmax(n)] += N - n.sum()
    kv = [int(x + rng.integers(0, 30)) for x in n]
    cu, lens, table, pages = ragged(torch, 16, S, list(n), kv, page)
    parts = cache4(torch, "heads", pages, page, Hk, d, 99)
    before = [u8(t).copy() for t in parts]
    k, v = (rand(torch, 105 + i, (N + behind, Hk, d), "bf16", 1.5) for i in range(2))
    paged_append_fp4(k, v, *parts, ints(torch, table), ints(torch, lens), ints(torch, cu))
    at = [(s, int(lens[s]) - n[s] + i) for s in range(S) for i in range(n[s])]
    page_no, off = np.array([table[s, p // page] for s, p in at]), np.array([p % page for _, p in at])
    for (codes, scale), x, (c0, s0) in zip((parts[:2], parts[2:]), (k, v), (before[:2], before[2:])):
        c0[page_no, off], s0[page_no, off] = orc.encode(f64(x[:N]))
        assert np.array_equal(u8(codes), c0) and np.array_equal(u8(scale), s0)
    got = paged_read_fp4(*parts, tensor(torch, page_no * page + off))
    assert all(np.array_equal(f64(a), orc.decode(*orc.encode(f64(x[:N])))) for a, x in zip(got, (k, v)))


@pytest.mark.parametrize("dtype,Hq,Hk,d,N", [("bf16", 4, 2, 64, 9001), ("f32", 12, 4, 64, 2501), ("bf16", 16, 16, 128, 3001)])
def test_append_in_one_call_or_two(torch, dtype, Hq, Hk, d, N):  # noqa: F811
    """Norm and rotation on the way of many tokens, some of them behind the last sequence."""
    from chunk_gated_delta_carve_amd import paged_append_fp4, qk_norm_rope_fwd, rope_tables
    live, page = N - 7, 32
    n = [5, live - 5]
    cu, lens, table, pages = ragged(torch, 15, 2, n, [70, live - 5], page)
    q, k, v = (rand(torch, 95 + i, (N, h, d), dtype, 1.5) for i, h in enumerate((Hq, Hk, Hk)))
    pos = np.r_[65:70, 0:live - 5, [0] * 7]
    cos, sin = rope_tables(int(pos.max()) + 1, d)
    q2, k2 = qk_norm_rope_fwd(q, k, cos, sin, ints(torch, pos))
    args = ints(torch, table), ints(torch, lens), ints(torch, cu)
    one, two = (cache4(torch, "heads", pages, page, Hk, d, 98) for _ in range(2))
    out = torch.full_like(q, 3.0)
    paged_append_fp4(k, v, *one, *args, cos, sin, q=q, q_out=out, norm=True)
    paged_append_fp4(k2, v, *two, *args)
    for a, b in zip(one, two):
        assert torch.equal(a, b)
    assert torch.equal(out[:live], q2[:live]) and (out[live:] == 3.0).all()


# read

@pytest.mark.parametrize("dtype,Hk,d,layout", [("bf16", 2, 64, "plain"), ("f32", 3, 128, "joint"), ("bf16", 7, 128, "heads"),
                                               ("f32", 1, 64, "heads")])
def test_read(torch, dtype, Hk, d, layout):  # noqa: F811
    """All codes and scales, twice the same slot, slots outside the cache (zeros), outputs inside wider tensors."""
    from chunk_gated_delta_carve_amd import paged_read_fp4
    pages, page = 9, 8
    parts = cache4(torch, layout, pages, page, Hk, d, 100, 2, 253)
    parts[1][3, 2, 0, 1] = 255
    rng = np.random.default_rng(3)
    slots = rng.integers(0, pages * page, 50)
    slots[:8] = [3 * page + 2, -1, pages * page, 0, pages * page - 1, -2 ** 60, 2 ** 60, 3 * page + 2]
    there = (slots >= 0) & (slots < pages * page)
    room = torch.full((50, 2 * Hk + 1, d), 7.0, dtype=dt(torch, dtype), device="cuda")
    k, v = paged_read_fp4(*parts, tensor(torch, slots), dtype=dt(torch, dtype), k_out=room[:, :Hk], v_out=room[:, Hk:2 * Hk])
    at = np.where(there, slots, 0)
    for got, ref in zip((k, v), values(parts)):
        want = np.where(there[:, None, None], ref[at // page, at % page], 0.0)
        assert np.array_equal(f64(got), want, equal_nan=True)
    assert np.isnan(f64(k[0, 0, 32:64])).all() and (room[:, 2 * Hk] == 7.0).all()
    two = paged_read_fp4(*parts, tensor(torch, slots.reshape(5, 10)), dtype=dt(torch, dtype))
    assert two[0].shape == (5, 10, Hk, d) and np.array_equal(f64(two[1]).reshape(50, Hk, d), f64(v))
    none = paged_read_fp4(*parts, tensor(torch, np.zeros(0, np.int64)))
    assert none[0].shape == (0, Hk, d)


# attention

@pytest.mark.parametrize("case", ATTENTION, ids=[str(i) for i in range(len(ATTENTION))])
def test_attention(torch, case):  # noqa: F811
    """Every cache entry that no row sees is NaN: other pages, the rest of the last page, keys before every window;
    block-table entries past a sequence's pages are -1."""
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    dtype, Hq, Hk, d, page, n, kv, window, layout, step = case
    say("case", case)
    S, N = len(n), sum(n)
    cu, lens, table, pages = ragged(torch, 7, S, n, kv, page)
    parts = cache4(torch, layout, pages, page, Hk, d, 110)
    q = rand(torch, 112, (N, Hq, d), dtype)
    seen = np.zeros((pages, page), bool)
    for s, p in att.token_places(cu, lens, N):
        for j in range(max(0, p - window + 1) if window else 0, p + 1):
            seen[att.place(table, s, j, page, pages)] = True
    hide = tensor(torch, ~seen)[..., None, None]
    for i in (1, 3):
        parts[i].masked_fill_(hide, 255)
    out, lse = paged_attention_fp4(q, *parts, ints(torch, table), ints(torch, lens), None if step else ints(torch, cu),
                                   window=window, return_lse=True)
    torch.cuda.synchronize()
    k, v = (tensor(torch, np.where(seen[..., None, None], x, 0.0)) for x in values(parts))
    check_attention(torch, out, lse, q, k, v, table, lens, cu, d ** -0.5, window, dtype)


LONG = [
    # dtype, Hq, Hk, d, page, n, kv, window, step: contexts that several workgroups share
    ("bf16", 12, 12, 64, 16, [1], [9000], 0, True), ("bf16", 16, 2, 128, 64, [1, 1], [20011, 300], 0, True),
    ("bf16", 4, 1, 128, 16, [300], [5001], 0, False), ("f32", 4, 2, 64, 16, [2], [3001], 0, False),
    ("bf16", 12, 4, 64, 16, [1999], [2000], 0, False), ("bf16", 16, 8, 128, 32, [1030], [2300], 0, False),
    ("bf16", 8, 2, 128, 16, [1, 1, 1], [7000, 3, 4096], 1000, True), ("f32", 4, 4, 128, 64, [1, 1], [2500, 2499], 0, True),
    ("bf16", 4, 2, 64, 16, [20, 1, 9], [4000, 50, 2222], 700, False),
]


@pytest.mark.parametrize("case", LONG, ids=[str(i) for i in range(len(LONG))])
def test_attention_over_long_contexts(torch, case):  # noqa: F811
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    dtype, Hq, Hk, d, page, n, kv, window, step = case
    say("case", case)
    cu, lens, table, pages = ragged(torch, 9, len(n), n, kv, page)
    parts = cache4(torch, "heads", pages, page, Hk, d, 120)
    q = rand(torch, 121, (sum(n), Hq, d), dtype)
    args = (ints(torch, table), ints(torch, lens), None if step else ints(torch, cu))
    out, lse = paged_attention_fp4(q, *parts, *args, window=window, return_lse=True)
    again = paged_attention_fp4(q, *parts, *args, window=window)
    assert torch.equal(out, again)
    rows = np.unique(np.r_[0:min(40, sum(n)), max(0, sum(n) - 40):sum(n)])    # the oracle is slow
    keep = [r for r in rows]
    k, v = values(parts)
    places = att.token_places(cu, lens, sum(n))
    for r in keep[::max(1, len(keep) // 24)]:
        s, p = places[r]
        ref = att.paged_attention(f64(q[r:r + 1]), k, v, table[s:s + 1], [p + 1], [0, 1], d ** -0.5, window)
        bo, bl = attention_bounds(dtype, d, d ** -0.5, *ref)
        close(f"o {r}", out[r:r + 1], ref[0], bo)
        close(f"lse {r}", lse[r:r + 1], ref[1], bl)


RAGGED = [
    # dtype, Hq, Hk, d, page, sequences, most new tokens, longest context, window
    ("bf16", 4, 2, 128, 16, 150, 1, 4000, 0), ("bf16", 3, 3, 64, 64, 90, 1, 3000, 0), ("f32", 4, 2, 64, 16, 70, 1, 3000, 0),
    ("bf16", 4, 1, 128, 4, 40, 1, 3000, 0), ("bf16", 4, 2, 64, 32, 60, 4, 3000, 0), ("bf16", 2, 2, 64, 16, 100, 1, 4000, 1500),
    ("f32", 2, 1, 128, 2, 30, 9, 2500, 900),
]


@pytest.mark.parametrize("case", RAGGED, ids=[str(i) for i in range(len(RAGGED))])
def test_ragged_contexts_dealt_to_workgroups(torch, case):  # noqa: F811
    """Many sequences from one key on, under a table that is far wider: several items to a workgroup, and items that
    several share."""
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    dtype, Hq, Hk, d, page, S, most, top, window = case
    say("case", case)
    rng = np.random.default_rng(31)
    n = rng.integers(1, most + 1, S)
    kv = [int(max(x, round(np.exp(rng.uniform(0, np.log(top)))))) for x in n]
    cu, lens, table, pages = ragged(torch, 32, S, list(n), kv, page, width=20000 // page)
    parts = cache4(torch, "heads", pages, page, Hk, d, 135)
    N = int(n.sum())
    q = rand(torch, 136, (N, Hq, d), dtype)
    step = most == 1
    out, lse = paged_attention_fp4(q, *parts, ints(torch, table), ints(torch, lens), None if step else ints(torch, cu),
                                   window=window, return_lse=True)
    kf, vf = (tensor(torch, x) for x in values(parts))
    check_attention(torch, out, lse, q, kf, vf, table, lens, cu, d ** -0.5, window, dtype)


CHUNKS = [
    # dtype, Hq, Hk, d, page, n, kv, window: several 16-row tiles to a sequence, and batches of single tokens with a chunk
    ("bf16", 8, 2, 128, 16, [32, 1, 17, 9], [3000, 2, 17, 800], 0), ("bf16", 4, 4, 128, 64, [100, 128], [100, 2222], 150),
    ("bf16", 16, 2, 128, 8, [15, 16], [2500, 90], 0), ("bf16", 4, 4, 64, 16, [48, 30, 33], [48, 1900, 333], 0),
    ("bf16", 4, 4, 64, 16, [79], [5000], 1111), ("bf16", 3, 1, 64, 32, [1] * 30 + [200], [700, 1, 33] * 10 + [900], 0),
    ("bf16", 4, 1, 128, 16, [300] + [1] * 20, [300] + [2100] * 20, 0), ("f32", 4, 2, 128, 16, [70, 2], [1300, 2], 0),
    ("f32", 3, 3, 64, 4, [99, 1, 17], [99, 400, 1700], 64),
]


CHUNKS += [  # and of many rows, in pages of few tokens and of many
    ("bf16", 16, 16, 128, 2, [700, 1400], [900, 1400], 0), ("bf16", 16, 16, 128, 16, [1400, 3, 800], [1500, 3000, 800], 300),
    ("bf16", 4, 2, 128, 4, [200, 255], [1333, 255], 0), ("bf16", 4, 2, 64, 2, [300, 77], [500, 77], 0),
    ("bf16", 12, 4, 64, 1, [222], [300], 100), ("bf16", 2, 2, 64, 128, [600, 129, 1], [600, 2500, 64], 0),
]


@pytest.mark.parametrize("case", CHUNKS, ids=[str(i) for i in range(len(CHUNKS))])
def test_chunks(torch, case):  # noqa: F811
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    dtype, Hq, Hk, d, page, n, kv, window = case
    say("case", case)
    cu, lens, table, pages = ragged(torch, 37, len(n), n, kv, page)
    parts = cache4(torch, "heads", pages, page, Hk, d, 137)
    q = rand(torch, 138, (sum(n), Hq, d), dtype)
    args = ints(torch, table), ints(torch, lens), ints(torch, cu)
    out, lse = paged_attention_fp4(q, *parts, *args, window=window, return_lse=True)
    kf, vf = (tensor(torch, x) for x in values(parts))
    check_attention(torch, out, lse, q, kf, vf, table, lens, cu, d ** -0.5, window, dtype)
    assert torch.equal(out, paged_attention_fp4(q, *parts, *args, window=window))


@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 16), ("bf16", 64, 64), ("f32", 64, 16)])
def test_long_stretches(torch, dtype, d, page):  # noqa: F811
    """More blocks to a workgroup than a lane's pages last for: each sequence has the bits of its first keys alone only
    if all are seen, so a few are checked against the definition."""
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    S, Hk, kv = 48, 16, 6000
    cu, lens, table, pages = ragged(torch, 33, S, [1] * S, [kv - 7 * s for s in range(S)], page)
    parts = cache4(torch, "heads", pages, page, Hk, d, 137)
    q = rand(torch, 138, (S, Hk, d), dtype)
    out, lse = paged_attention_fp4(q, *parts, ints(torch, table), ints(torch, lens), return_lse=True)
    for s in (0, 23, 47):
        need = -(-int(lens[s]) // page)
        own = [t[torch.tensor(table[s, :need], device="cuda")] for t in parts]
        k, v = values(own)
        ref = att.paged_attention(f64(q[s:s + 1]), k, v, np.arange(need)[None], [lens[s]], [0, 1], d ** -0.5, 0)
        bo, bl = attention_bounds(dtype, d, d ** -0.5, *ref)
        close(f"o {s}", out[s:s + 1], ref[0], bo)
        close(f"lse {s}", lse[s:s + 1], ref[1], bl)


@pytest.mark.parametrize("dtype,n,kv,d", [("bf16", 1, 40, 64), ("bf16", 100, 100, 128), ("f32", 9, 20, 64),
                                          ("bf16", 3, 5000, 128)])
def test_pages_that_are_not_there(torch, dtype, n, kv, d):  # noqa: F811
    """Holes in the table (-1, or past the cache) are keys that nobody sees; page 0, which is loaded in their place,
    is NaN."""
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    cu, lens, table, pages = ragged(torch, 10, 1, [n], [kv], 16)
    table = np.where(table == 0, pages, table)                  # page 0 belongs to nobody
    pages += 1
    parts = cache4(torch, "plain", pages, 16, 2, d, 130)
    for i in (1, 3):
        parts[i][0] = 255
    table[0, 0], table[0, table.shape[1] // 2] = -1, pages + 7
    q = rand(torch, 131, (n, 4, d), dtype)
    out, lse = paged_attention_fp4(q, *parts, ints(torch, table), ints(torch, lens), ints(torch, cu), return_lse=True)
    k, v = values(parts)
    check_attention(torch, out, lse, q, tensor(torch, k), tensor(torch, v), table, lens, cu, d ** -0.5, 0, dtype)


def test_nothing_to_see(torch):  # noqa: F811
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    parts = cache4(torch, "plain", 2, 16, 2, 64, 140)
    for dtype in ("bf16", "f32"):
        for n in (2, 100):
            q = rand(torch, 141, (n, 4, 64), dtype)
            for table, kv in (([[-1, -1]], n), ([[0, 1]], 0), ([[0, 1]], -5)):
                out, lse = paged_attention_fp4(q, *parts, ints(torch, table), ints(torch, [kv]), ints(torch, [0, n]),
                                               return_lse=True)
                assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("dtype,n,Hk,d,kv", [("bf16", 6, 2, 64, 26), ("bf16", 150, 2, 64, 170), ("f32", 6, 2, 64, 26),
                                             ("bf16", 150, 2, 128, 170), ("bf16", 150, 66, 128, 170),
                                             ("bf16", 5, 2, 128, 4000), ("bf16", 90, 1, 64, 4000)])
def test_a_bad_block_reaches_only_the_rows_that_see_it(torch, dtype, n, Hk, d, kv):  # noqa: F811
    """A token's block of NaN, inside what other rows of the same tile share, leaves the rows that do not see it."""
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    window, Hq = 10 if kv < 1000 else 0, 2 * Hk
    cu, lens, table, pages = ragged(torch, 11, 1, [n], [kv], 16)
    for which in (0, 1):
        parts = cache4(torch, "plain", pages, 16, Hk, d, 150)
        q = rand(torch, 152, (n, Hq, d), dtype)
        j = kv - n // 2                          # that position's page entry
        parts[1 + 2 * which][table[0, j // 16], j % 16, :, 1] = 255
        out, lse = paged_attention_fp4(q, *parts, ints(torch, table), ints(torch, lens), ints(torch, cu), window=window,
                                       return_lse=True)
        p = np.arange(kv - n, kv)
        sees = (j <= p) & ((j > p - window) if window else True)
        k, v = values(parts)
        rows = np.flatnonzero(~sees)[-6:]
        for r in rows:
            ref = att.paged_attention(f64(q[r:r + 1]), k, v, table, [p[r] + 1], [0, 1], d ** -0.5, window)
            bo, bl = attention_bounds(dtype, d, d ** -0.5, *ref)
            close(f"row {r}", out[r:r + 1], ref[0], bo)
            close(f"its lse {r}", lse[r:r + 1], ref[1], bl)
        seen = f64(out)[sees]
        assert np.isfinite(f64(out)[~sees]).all()
        if which:                                # a value shows in its channels alone
            assert np.isnan(seen[:, :, 32:64]).all() and np.isfinite(np.delete(seen, range(32, 64), 2)).all()
        else:
            assert np.isnan(seen).all()


@pytest.mark.parametrize("dtype,n,kv,d", [("bf16", 4, 300, 64), ("bf16", 4, 300, 128), ("bf16", 90, 3000, 64),
                                          ("bf16", 90, 3000, 128), ("f32", 4, 300, 64), ("bf16", 300, 300, 128)])
@pytest.mark.parametrize("size", [2.0 ** e for e in (18, 40, 63)])
def test_scores_of_any_finite_size(torch, size, dtype, n, kv, d):  # noqa: F811
    """Keys that grow along the context: the largest score takes the row."""
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    cu, lens, table, pages = ragged(torch, 12, 1, [n], [kv], 16)
    parts = cache4(torch, "plain", pages, 16, 1, d, 160)
    e = int(np.log2(size))
    parts[0].fill_(0x22)                         # ones
    for j in range(kv):
        parts[1][table[0, j // 16], j % 16] = 127 + e - (kv - j) % 7      # sizes that differ by factors of two
    q = torch.zeros(n, 2, d, dtype=dt(torch, dtype), device="cuda")
    q[:, 0, :], q[:, 1, 0] = 1.0, -1.0
    out, lse = paged_attention_fp4(q, *parts, ints(torch, table), ints(torch, lens), ints(torch, cu), return_lse=True)
    k, v = values(parts)
    for r in (0, n // 2, n - 1):
        p = kv - n + r
        ref = att.paged_attention(f64(q[r:r + 1]), k, v, table, [p + 1], [0, 1], d ** -0.5, 0)
        # the scores are exact (sums of powers of two), so only equal ones share a row
        h = HALF[dtype]
        assert np.all(np.abs(f64(out[r]) - ref[0][0]) <= 2 * h * np.abs(ref[0][0]) + (h + 2.0 ** -18) * ref[2][0] + 1e-30)
        assert np.allclose(f64(lse[r]), ref[1][0], rtol=2.0 ** -21)


def test_rows_behind_the_last_sequence_are_left(torch):  # noqa: F811
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    for dtype in ("bf16", "f32"):
        for n, extra in ((3, 5), (140, 9)):
            cu, lens, table, pages = ragged(torch, 12, 1, [n], [n], 16)
            parts = cache4(torch, "plain", pages, 16, 2, 64, 170)
            q = rand(torch, 172, (n + extra, 4, 64), dtype)
            out = torch.full_like(q, 5.0)
            paged_attention_fp4(q, *parts, ints(torch, table), ints(torch, lens), ints(torch, cu), out=out)
            assert (out[n:] == 5.0).all() and not (out[:n] == 5.0).all()


@pytest.mark.parametrize("case", [
    # dtype, Hq, Hk, d, page, sequences, window, step: more sequences than a wave has lanes
    ("bf16", 4, 2, 64, 16, 150, 0, True), ("bf16", 4, 2, 128, 16, 70, 20, False), ("bf16", 8, 1, 64, 32, 90, 0, False),
    ("f32", 2, 2, 64, 16, 129, 0, False), ("bf16", 2, 2, 128, 16, 1500, 0, True),
], ids=["step", "ragged", "tiles", "f32", "more"])
def test_many_sequences(torch, case):  # noqa: F811
    from chunk_gated_delta_carve_amd import paged_append_fp4, paged_attention_fp4
    dtype, Hq, Hk, d, page, S, window, step = case
    rng = np.random.default_rng(18)
    top = 14 if Hq // Hk < 8 else 60
    n = [1] * S if step else list(rng.integers(0, top, S))
    kv = [int(x + rng.integers(0, 90)) if x else 0 for x in n]
    cu, lens, table, pages = ragged(torch, 19, S, n, kv, page)
    parts = cache4(torch, "heads", pages, page, Hk, d, 180)
    N = sum(n)
    q, k, v = (rand(torch, 192 + i, (N, h, d), dtype) for i, h in enumerate((Hq, Hk, Hk)))
    args = (ints(torch, table), ints(torch, lens), None if step else ints(torch, cu))
    want, _ = stored(parts, table, lens, cu, page, f64(k), f64(v))
    paged_append_fp4(k, v, *parts, *args)
    for got, ref in zip(parts, want):
        assert np.array_equal(u8(got), ref)
    out, lse = paged_attention_fp4(q, *parts, *args, window=window, return_lse=True)
    kf, vf = (tensor(torch, x) for x in values(parts))
    check_attention(torch, out, lse, q, kf, vf, table, lens, cu, d ** -0.5, window, dtype)


def test_offsets_past_32_bits(torch):  # noqa: F811
    """Pages whose bytes lie past 2^32 of the codes and past 2^28 of the scales, for every call."""
    from chunk_gated_delta_carve_amd import paged_append_fp4, paged_attention_fp4, paged_fp4_cache, paged_read_fp4
    page, Hk, d, pages = 64, 4, 128, 290000
    parts = paged_fp4_cache(pages, page, Hk, d)
    assert parts[0].numel() > 2 ** 32
    small = list(range(pages - 6, pages))
    for t, s in zip(parts, cache4(torch, "plain", 6, page, Hk, d, 200)):
        t[small] = s
    for n, kv in ((1, 300), (70, 300)):
        table = np.array([[pages - 1, pages - 5, pages - 3, pages - 2, pages - 6]])
        lens, cu = ints(torch, [kv]), ints(torch, [0, n])
        q, k, v = (rand(torch, 202 + i, (n, h, d), "bf16") for i, h in enumerate((8, Hk, Hk)))
        paged_append_fp4(k, v, *parts, ints(torch, table), lens, cu)
        out, lse = paged_attention_fp4(q, *parts, ints(torch, table), lens, cu, return_lse=True)
        lo = table - (pages - 6)                 # the same six pages as a cache of their own
        kf, vf = (tensor(torch, x) for x in values([t[small] for t in parts]))
        check_attention(torch, out, lse, q, kf, vf, lo, [kv], [0, n], d ** -0.5, 0, "bf16")
        p = kv - 1
        got, _ = paged_read_fp4(*parts, tensor(torch, [int(table[0, p // page]) * page + p % page]))
        assert np.array_equal(f64(got[0]), orc.decode(*orc.encode(f64(k[-1]))))


def test_calls_on_two_streams(torch):  # noqa: F811
    """Two calls under way at once, each with a workspace of its own, have the bits of calls one by one."""
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    calls = []
    for seed, (n, kv, d) in enumerate(((1, 9000, 128), (200, 4000, 64))):
        cu, lens, table, pages = ragged(torch, 23 + seed, 2, [n, n], [kv, kv - 7], 16)
        parts = cache4(torch, "heads", pages, 16, 2, d, 210 + seed)
        calls.append((rand(torch, 235 + seed, (2 * n, 8, d), "bf16"), *parts, ints(torch, table), ints(torch, lens),
                      ints(torch, cu)))
    want = [paged_attention_fp4(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(3):
        got = [paged_attention_fp4(*c, stream=s) for c, s in zip(calls, streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_another_stream(torch):  # noqa: F811
    """Calls on a stream that is not the current one: temporaries are that stream's, results are ordered with it."""
    from chunk_gated_delta_carve_amd import paged_append_fp4, paged_assign, paged_attention_fp4, paged_read_fp4
    cu, lens, table, pages = ragged(torch, 17, 1, [1], [5000], 16)
    parts = cache4(torch, "heads", pages, 16, 2, 64, 220)
    q, k = rand(torch, 222, (1, 4, 64), "bf16"), rand(torch, 223, (1, 2, 64), "bf16")
    tab, kv = ints(torch, table), ints(torch, lens)
    new, stack, count = ints(torch, [1]), ints(torch, [3, 4]), ints(torch, [2, 0])

    def calls(**kw):
        room = paged_assign(tab.clone(), kv - 1, new, stack, count, 16, 1, **kw)
        paged_append_fp4(k, k, *parts, tab, kv, **kw)
        got = paged_read_fp4(*parts, room[3], **kw)
        return [*room, *got, paged_attention_fp4(q, *parts, tab, kv, **kw)]

    want = calls()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):                   # clone() and kv - 1 belong to it too
        for handle in (s, s.cuda_stream):
            got = calls(stream=handle)
            s.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)
    with torch.cuda.stream(s):                   # 0 is the default stream, whichever is current
        got = paged_attention_fp4(q, *parts, tab, kv, stream=0)
    torch.cuda.default_stream().synchronize()
    assert torch.equal(got, want[-1])


def test_strided_queries_and_outputs(torch):  # noqa: F811
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    n, kv = 37, 61
    cu, lens, table, pages = ragged(torch, 13, 1, [n], [kv], 16)
    parts = cache4(torch, "plain", pages, 16, 2, 64, 230)
    wide = rand(torch, 232, (n, 9, 64), "bf16")
    room = torch.zeros(n, 10, 64, dtype=torch.bfloat16, device="cuda")
    big = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
    big[0, :table.shape[1]] = ints(torch, table[0])
    args = (ints(torch, lens), ints(torch, cu))
    a = paged_attention_fp4(wide[:, 3:7], *parts, big[:1, :table.shape[1]], *args, out=room[:, 2:6])
    b = paged_attention_fp4(wide[:, 3:7].contiguous(), *parts, ints(torch, table), *args)
    assert torch.equal(a, b) and not room[:, :2].any() and not room[:, 6:].any()


@pytest.mark.parametrize("n,d,layout", [(1, 64, "plain"), (1, 128, "heads"), (100, 64, "heads"), (300, 128, "plain")])
def test_layouts_and_pages_have_the_same_bits(torch, n, d, layout):  # noqa: F811
    """The same tokens in pages of 1, 4, 16 and 256 and in any layout."""
    from chunk_gated_delta_carve_amd import paged_append_fp4, paged_attention_fp4
    kv, Hk = 333, 2
    k, v, q = (rand(torch, 240 + i, (kv, h, d), "bf16") for i, h in enumerate((Hk, Hk, 4)))
    outs = []
    for page, lay in ((1, "plain"), (4, "heads"), (16, layout), (256, "joint"), (8, "heads")):
        cu, lens, table, pages = ragged(torch, 14, 1, [kv], [kv], page)
        parts = cache4(torch, lay, pages, page, Hk, d, 245)
        tab, full = ints(torch, table), ints(torch, [0, kv])
        paged_append_fp4(k, v, *parts, tab, ints(torch, lens), full)
        # tables of one width, so that the same kernel is taken
        wide = torch.full((1, 512), -1, dtype=torch.int32, device="cuda")
        wide[:, :tab.shape[1]] = tab
        outs.append(paged_attention_fp4(q[-n:], *parts, wide, ints(torch, lens), ints(torch, [0, n])))
    kf, vf = (orc.decode(*orc.encode(f64(x))) for x in (k, v))
    ref = att.paged_attention(f64(q[-n:]), kf[None], vf[None], np.zeros((1, 1), int), [kv], [0, n], d ** -0.5, 0)
    for o in outs:
        close("o", o, ref[0], attention_bounds("bf16", d, d ** -0.5, *ref)[0])


# room in the cache

def stack_of(pages, free, capacity):
    return np.concatenate([free, np.full(capacity - len(free), -7)])


def check_assign(torch, table, kv, new, stack, count, page, tokens, done, **kw):  # noqa: F811
    from chunk_gated_delta_carve_amd import paged_assign
    tab, free = ints(torch, table), ints(torch, stack)
    got = paged_assign(tab, ints(torch, kv), ints(torch, new), free, ints(torch, count), page, tokens,
                       done=None if done is None else ints(torch, done), **kw)
    want = orc.assign(table, kv, new, stack, count, page, tokens, done)
    for name, g, w in zip(("cu", "lens", "positions", "slots", "count", "table", "free"), (*got, tab, free), want):
        assert np.array_equal(g.cpu().numpy(), np.asarray(w).reshape(g.shape)), name
    return got


ASSIGN = [
    # requests, longest context, most new tokens, page, part that ended, pages to spare, padding
    (1, 40, 1, 16, 0.0, 3, 0), (5, 100, 30, 16, 0.4, 3, 7), (64, 500, 1, 16, 0.0, 9, 0), (200, 300, 50, 4, 0.3, -90, 11),
    (1024, 60, 5, 8, 0.2, 0, 100), (1025, 60, 3, 8, 0.2, 5, 1), (2500, 30, 2, 1, 0.5, -300, 0), (3, 20000, 9000, 16, 0.0, 0, 5),
    (30, 2000, 700, 256, 0.1, 2, 0), (7, 0, 20, 16, 0.0, 4, 0), (4000, 10, 0, 16, 0.9, 0, 3),
    (5000, 20, 3, 4, 0.25, -100, 9), (4096, 9, 4, 2, 0.0, 0, 1), (2, 100, 60000, 64, 0.0, 0, 0),
]


@pytest.mark.parametrize("case", ASSIGN, ids=[str(i) for i in range(len(ASSIGN))])
def test_assign(torch, case):  # noqa: F811
    S, top, most, page, ended, spare, pad = case
    say("case", case)
    rng = np.random.default_rng(S + page)
    kv, new = rng.integers(0, top + 1, S), rng.integers(0, most + 1, S)
    done = (rng.random(S) < ended).astype(int)
    held = -(-kv // page)
    need = int(np.sum(-(-np.where(done, new, kv + new) // page) - np.where(done, 0, held)))
    free = max(0, need - int(np.sum(held * done)) + spare)
    capacity = int(held.sum()) + free
    order = rng.permutation(capacity)
    width = -(-(top + most) // page) + 1
    table = np.full((S, width), -1)
    at = 0
    for s in range(S):
        table[s, :held[s]] = order[at:at + held[s]]
        at += held[s]
    stack = stack_of(capacity, order[at:], capacity)
    for d in ((None, done) if ended < 0.3 else (done,)):
        check_assign(torch, table, kv, new, stack, [free, 4], page, int(new.sum()) + pad, d)


@pytest.mark.parametrize("S,top,page,holes,fit", [(40, 9000, 4, 0.0, 1.0), (40, 9000, 4, 0.3, 1.0), (3, 30000, 1, 0.1, 0.6),
                                                  (1500, 40, 2, 0.2, 1.0), (1500, 40, 2, 0.0, 0.3), (2, 8192, 1, 0.0, 1.0)])
def test_assign_gives_back_what_others_take(torch, S, top, page, holes, fit):  # noqa: F811
    """Most requests end, tables with entries that are no pages, stacks that do not hold all that comes back, and new
    tokens that take pages given back just now and ones that were free before."""
    rng = np.random.default_rng(S + page)
    kv = rng.integers(top // 2, top + 1, S)
    done = (rng.random(S) < 0.7).astype(int)
    done[0] = 1
    held = -(-kv // page)
    new = np.where(rng.random(S) < 0.8, rng.integers(0, int(1.5 * top) + 1, S), 0)
    free = 50
    pages = int(held.sum()) + free
    order = rng.permutation(pages)
    table = np.full((S, -(-3 * top // page)), -1)
    at = 0
    for s in range(S):
        table[s, :held[s]] = order[at:at + held[s]]
        at += held[s]
    table[rng.random(table.shape) < holes] = -1
    capacity = max(free, int(pages * fit))
    stack = stack_of(pages, order[at:], capacity)
    check_assign(torch, table, kv, new, stack, [free, 1], page, int(new.sum()), done)


def test_assign_at_its_edges(torch):  # noqa: F811
    """Negative lengths, holes in the table of an ended request, tokens past the table, too few rows for the tokens, a
    stack that overflows, counts outside of it, no requests, no tokens, no pages."""
    table = np.array([[4, -1, 6, -1], [7, 8, 9, 10], [11, -1, -1, -1]])
    stack = [0, 1, 2, 3, -7, -7]
    check_assign(torch, table, [40, -3, 5], [-2, 30, 4], stack, [4, 0], 16, 40, [1, 0, 0])
    check_assign(torch, table, [48, 64, 5], [0, 0, 100], stack, [4, 2], 16, 100, [1, 1, 0])       # 6 of 6 entries held
    check_assign(torch, table, [60, 60, 60], [10, 70, 1], stack, [4, 0], 16, 81, None)           # past 64 tokens
    check_assign(torch, table, [0, 0, 0], [10, 10, 10], stack, [99, 0], 16, 25, None)            # 25 rows for 30 tokens
    check_assign(torch, table, [0, 0, 0], [10, 10, 10], stack, [-5, 7], 16, 30, None)
    check_assign(torch, table, [20, 0, 0], [0, 0, 0], stack, [4, 0], 16, 0, None)
    check_assign(torch, np.zeros((0, 4), int), [], [], stack, [4, 0], 16, 3, None)
    check_assign(torch, np.zeros((2, 0), int), [3, 4], [1, 2], stack, [4, 0], 16, 3, [0, 1])
    check_assign(torch, table, [20, 1, 1], [30, 5, 0], [], [0, 0], 16, 35, [0, 1, 0])


def test_assign_in_place_and_in_a_graph(torch):  # noqa: F811
    """A captured step goes on from the last one's lengths, table and free pages; requests that end are replaced."""
    from chunk_gated_delta_carve_amd import paged_assign
    S, page, width, pages = 6, 4, 16, 40
    rng = np.random.default_rng(8)
    table, kv = np.full((S, width), -1), np.zeros(S, int)
    stack, count = np.arange(pages), [pages, 0]
    dev = [ints(torch, x) for x in (table, kv, stack, count)]
    new, done = ints(torch, np.zeros(S)), ints(torch, np.zeros(S))
    N = 32

    def step(tab, lens, free, cnt):
        return paged_assign(tab, lens, new, free, cnt, page, N, done=done, kv_lens_out=lens, free_count_out=cnt)

    step(*[t.clone() for t in dev])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(*dev)
    for turn in range(12):
        n = rng.integers(0, 6, S)
        over = ((rng.random(S) < 0.25) & (kv > 0)).astype(int) if turn else np.zeros(S, int)
        new.copy_(ints(torch, n))
        done.copy_(ints(torch, over))
        g.replay()
        torch.cuda.synchronize()
        cu, lens, pos, slots, count, table, stack = orc.assign(table, kv, n, stack, count, page, N, over)
        kv = np.array(lens)
        for got, want in zip((*out, dev[0], dev[2]), (cu, lens, pos, slots, count, table, stack)):
            assert np.array_equal(got.cpu().numpy(), np.asarray(want)), turn
        assert len(set(slots[slots >= 0])) == (slots >= 0).sum()


# together

@pytest.mark.parametrize("dtype,Hq,Hk,d", [("bf16", 12, 4, 64), ("bf16", 16, 2, 128), ("f32", 4, 2, 128)])
def test_prompts_then_single_tokens(torch, dtype, Hq, Hk, d):  # noqa: F811
    """As a serving loop uses them: room for ragged prompts, stored in two chunks, then single tokens with a request that
    ends and one that takes its place; every output against attention over what the oracle says was stored."""
    from chunk_gated_delta_carve_amd import (paged_append_fp4, paged_assign, paged_attention_fp4, paged_fp4_cache,
                                             paged_read_fp4, qk_norm_rope_fwd, rope_tables)
    S, page, pages, width = 4, 16, 60, 16
    cos, sin = rope_tables(256, d)
    parts = paged_fp4_cache(pages, page, Hk, d)
    tab = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    lens, free, count = ints(torch, [0] * S), ints(torch, np.arange(pages)), ints(torch, [pages, 0])
    history = [([], []) for _ in range(S)]        # keys and values of every request as the cache has them
    steps = [([70, 33, 0, 9], None), ([31, 40, 120, 1], None), ([1] * S, None), ([1, 1, 0, 1], None),
             ([1, 50, 1, 1], [0, 1, 0, 0]), ([1] * S, None), ([1] * S, [0, 0, 0, 1])]
    for turn, (n, over) in enumerate(steps):
        N = sum(n) + (3 if turn == 1 else 0)      # one padded batch
        q, k, v = (rand(torch, 300 + 3 * turn + i, (N, h, d), dtype, 1.5) for i, h in enumerate((Hq, Hk, Hk)))
        cu, lens, pos, slots, count = paged_assign(tab, lens, ints(torch, n), free, count, page, N,
                                                   done=None if over is None else ints(torch, over), kv_lens_out=lens)
        single = all(x == 1 for x in n)
        qr = paged_append_fp4(k, v, *parts, tab, lens, None if single else cu, cos, sin, q=q, norm=True)
        out, lse = paged_attention_fp4(qr, *parts, tab, lens, None if single else cu, window=100, return_lse=True)
        q2, k2 = qk_norm_rope_fwd(q, k, cos, sin, pos)
        got_k, got_v = paged_read_fp4(*parts, slots, dtype=torch.float32)
        k2, v2 = (orc.decode(*orc.encode(f64(x))) for x in (k2, v))
        offs = cu.cpu().numpy()
        assert np.array_equal(f64(got_k)[:sum(n)], k2[:sum(n)]) and np.array_equal(f64(got_v)[:sum(n)], v2[:sum(n)])
        assert torch.equal(qr[:sum(n)], q2[:sum(n)]) and not got_k[sum(n):].any()
        for s in range(S):
            if over is not None and over[s]:
                history[s] = ([], [])
            history[s][0].extend(k2[offs[s]:offs[s + 1]])
            history[s][1].extend(v2[offs[s]:offs[s + 1]])
            if not n[s]:
                continue
            kf, vf = (np.array(x)[None] for x in history[s])
            rows = slice(int(offs[s]), int(offs[s + 1]))
            ref = att.paged_attention(f64(qr[rows]), kf, vf, np.zeros((1, 1), int), [kf.shape[1]], [0, n[s]], d ** -0.5, 100)
            bo, bl = attention_bounds(dtype, d, d ** -0.5, *ref)
            close(f"turn {turn} request {s}", out[rows], ref[0], bo)
            close(f"turn {turn} request {s} lse", lse[rows], ref[1], bl)
    held = tab[:, 0].cpu().numpy()
    assert int(count[1]) == 0 and int(count[0]) == pages - sum(-(-int(x) // page) for x in lens.cpu()) and len(set(held)) == S


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 128)])
def test_room_in_a_cache_that_is_not_in_4_bits(torch, dtype, d):  # noqa: F811
    """paged_assign's results as paged_append, paged_attention and qk_norm_rope_fwd take them."""
    from chunk_gated_delta_carve_amd import paged_append, paged_assign, paged_attention, qk_norm_rope_fwd, rope_tables
    S, Hq, Hk, page, pages, width = 3, 4, 2, 16, 40, 12
    cos, sin = rope_tables(256, d)
    kc, vc = (torch.zeros(pages, page, Hk, d, dtype=dt(torch, dtype), device="cuda") for _ in range(2))
    tab = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    lens, free, count = ints(torch, [0] * S), ints(torch, np.arange(pages)), ints(torch, [pages, 0])
    history = [([], []) for _ in range(S)]
    for turn, (n, over) in enumerate([([40, 7, 65], None), ([1, 1, 1], None), ([1, 20, 1], [0, 1, 0]), ([1, 1, 1], None)]):
        N = sum(n)
        q, k, v = (rand(torch, 400 + 3 * turn + i, (N, h, d), dtype) for i, h in enumerate((Hq, Hk, Hk)))
        cu, lens, pos, slots, count = paged_assign(tab, lens, ints(torch, n), free, count, page, N,
                                                   done=None if over is None else ints(torch, over), kv_lens_out=lens)
        qr = paged_append(k, v, kc, vc, tab, lens, cu, cos, sin, q=q)
        q2, k2 = qk_norm_rope_fwd(q, k, cos, sin, pos, norm=False)
        assert torch.equal(qr, q2)
        assert torch.equal(kc.flatten(0, 1)[slots], k2) and torch.equal(vc.flatten(0, 1)[slots], v)
        out = paged_attention(qr, kc, vc, tab, lens, cu)
        offs = cu.cpu().numpy()
        for s in range(S):
            if over is not None and over[s]:
                history[s] = ([], [])
            history[s][0].extend(f64(k2)[offs[s]:offs[s + 1]])
            history[s][1].extend(f64(v)[offs[s]:offs[s + 1]])
            kf, vf = (np.array(x)[None] for x in history[s])
            rows = slice(int(offs[s]), int(offs[s + 1]))
            ref = att.paged_attention(f64(qr[rows]), kf, vf, np.zeros((1, 1), int), [kf.shape[1]], [0, n[s]], d ** -0.5, 0)
            close(f"turn {turn} request {s}", out[rows], ref[0], attention_bounds(dtype, d, d ** -0.5, *ref)[0])


def test_captured_decode_steps(torch):  # noqa: F811
    """A whole decode step (room, append, attention) captured once: every replay has the bits of an eager run of the same
    step on a copy of the state, with eager work in between. Two graphs share one workspace."""
    from chunk_gated_delta_carve_amd import (paged_append_fp4, paged_assign, paged_attention_fp4, paged_fp4_cache,
                                             paged_fp4_workspace_bytes, rope_tables)
    S, Hq, Hk, d, page, width = 3, 16, 2, 128, 16, 64
    pages = S * width
    cos, sin = rope_tables(1024, d)
    q, k, v = (rand(torch, 251 + i, (S, h, d), "bf16") for i, h in enumerate((Hq, Hk, Hk)))
    new = ints(torch, [1] * S)
    ws = torch.empty(paged_fp4_workspace_bytes(S, S, Hq, Hk, d, page, width, step=True), dtype=torch.uint8, device="cuda")

    def state():
        kv = [100, 700, 5]
        held = [-(-x // page) for x in kv]
        table, at = np.full((S, width), -1), 0
        for s in range(S):
            table[s, :held[s]] = np.arange(at, at + held[s])
            at += held[s]
        stack = np.concatenate([np.arange(at, pages), np.zeros(at)])
        return [ints(torch, x) for x in (table, kv, stack, [pages - at, 0])] + list(cache4(torch, "heads", pages, page, Hk, d, 255))

    def step(st, window):
        tab, lens, free, count, *parts = st
        paged_assign(tab, lens, new, free, count, page, S, kv_lens_out=lens, free_count_out=count)
        qr = paged_append_fp4(k, v, *parts, tab, lens, cos=cos, sin=sin, q=q, norm=True)
        return paged_attention_fp4(qr, *parts, tab, lens, window=window, workspace=ws if ws.numel() else None)

    live = [state(), state()]
    copy = [state(), state()]
    step(state(), 0)
    torch.cuda.synchronize()
    graphs = []
    for st, window in zip(live, (0, 200)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(st, window)
        graphs.append((g, out))
    for turn in range(20):
        q.copy_(rand(torch, 270 + turn, (S, Hq, d), "bf16"))
        for g, _ in graphs:
            g.replay()
        got = [o.clone() for _, o in graphs]
        want = [step(st, window) for st, window in zip(copy, (0, 200))]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), turn
        for a, b in zip(live[0][:4] + live[1][:4], copy[0][:4] + copy[1][:4]):
            assert torch.equal(a, b), turn


def test_refusals(torch):  # noqa: F811
    from chunk_gated_delta_carve_amd import paged_append_fp4, paged_assign, paged_attention_fp4, paged_read_fp4
    from chunk_gated_delta_carve_amd._lib import CarveError
    kc, ks, vc, vs = parts = cache4(torch, "plain", 4, 16, 2, 64, 280)
    q, table, lens, cu = rand(torch, 281, (3, 4, 64), "bf16"), ints(torch, [[0, 1]]), ints(torch, [20]), ints(torch, [0, 3])
    k = q[:, :2]
    att_, app = paged_attention_fp4, paged_append_fp4
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    stack, count = ints(torch, [2, 3]), ints(torch, [2, 0])
    asg = lambda *a, **kw: paged_assign(*a, **kw)  # noqa: E731
    for i, (err, call) in enumerate([
        (ValueError, lambda: att_(q.cpu(), *parts, table, lens, cu)),
        (ValueError, lambda: att_(q.half(), *parts, table, lens, cu)),
        (ValueError, lambda: att_(q, *parts, table, lens)),                         # 3 tokens, 1 sequence
        (ValueError, lambda: att_(q, *parts, table.long(), lens, cu)),
        (ValueError, lambda: att_(q, kc.to(torch.int8), ks, vc, vs, table, lens, cu)),
        (ValueError, lambda: att_(q, kc, ks[..., :1], vc, vs, table, lens, cu)),
        (ValueError, lambda: att_(q, kc, ks, vc[:3], vs, table, lens, cu)),
        (ValueError, lambda: att_(q, kc, ks, vc, vs.cpu(), table, lens, cu)),
        (ValueError, lambda: att_(rand(torch, 1, (3, 4, 128), "bf16"), *parts, table, lens, cu)),
        (ValueError, lambda: att_(q, kc.transpose(2, 3).contiguous().transpose(2, 3), ks, vc, vs, table, lens, cu)),
        (ValueError, lambda: att_(q, *parts, table, lens, cu, out=q[:2])),
        (CarveError, lambda: att_(q, *parts, table, lens, cu, out=q)),
        (CarveError, lambda: att_(q, *parts, table, lens, cu, scale=0.0)),
        (CarveError, lambda: att_(q, *parts, table, lens, cu, scale=1e39)),
        (CarveError, lambda: att_(q, *parts, table, lens, cu, scale=float("inf"))),
        (CarveError, lambda: att_(q, *parts, table, lens, cu, window=-1)),
        (CarveError, lambda: att_(q[:, :3], *parts, table, lens, cu)),              # 3 heads over 2
        (CarveError, lambda: att_(q, *(t[:, :12] for t in parts), table, lens, cu)),     # 12 tokens a page
        (CarveError, lambda: app(k, k, kc, ks, kc, vs, table, lens, cu)),
        (CarveError, lambda: app(k, k, kc, ks, vc, ks, table, lens, cu)),
        (ValueError, lambda: app(k, k, *parts, table, lens, cu, k_weight=q[0, 0])),
        (ValueError, lambda: app(k, k, *parts, table, lens, cu, q_weight=q[0, 0], norm=True)),
        (ValueError, lambda: app(k, k[:2], *parts, table, lens, cu)),
        (ValueError, lambda: paged_read_fp4(*parts, slots.int())),
        (ValueError, lambda: paged_read_fp4(*parts, slots, dtype=torch.float16)),
        (ValueError, lambda: paged_read_fp4(*parts, slots, k_out=q)),
        (ValueError, lambda: paged_read_fp4(*(t.cpu() for t in parts), slots)),
        (ValueError, lambda: asg(table.long(), lens, lens, stack, count, 16, 3)),
        (ValueError, lambda: asg(table, lens, lens.long(), stack, count, 16, 3)),
        (ValueError, lambda: asg(table, lens, lens, stack, count[:1], 16, 3)),
        (ValueError, lambda: asg(table, lens, lens, stack, count, 16, -1)),
        (ValueError, lambda: asg(table, lens, lens, stack, count, 16, 3, done=cu)),
        (ValueError, lambda: asg(table.cpu(), lens, lens, stack, count, 16, 3)),
        (CarveError, lambda: asg(table, lens, lens.clone(), stack, count, 12, 3)),
        (CarveError, lambda: asg(table, lens, lens.clone(), stack, count, 16, 3, free_count_out=stack)),
    ]):
        with pytest.raises(err):
            call()
            say("not refused:", i)


@pytest.mark.parametrize("dtype,d,Hk,n", [
    ("bf16", 64, 2, [1] * 4), ("bf16", 128, 1, [1] * 70), ("f32", 64, 3, [1]), ("f32", 128, 2, [1] * 5),
    ("bf16", 64, 2, [3, 1, 0, 2]), ("f32", 64, 2, [40, 1]), ("bf16", 64, 2, [150, 60]), ("bf16", 128, 2, [150, 60]),
    ("bf16", 128, 66, [150, 200])])
def test_a_table_without_pages(torch, dtype, d, Hk, n):  # noqa: F811
    """Width 0, in the row kernel and in the tile kernels of four and of eight waves: nothing is stored, no key is seen."""
    from chunk_gated_delta_carve_amd import paged_append_fp4, paged_attention_fp4
    S, N, step = len(n), sum(n), all(x == 1 for x in n)
    table = torch.empty(S, 0, dtype=torch.int32, device="cuda")
    lens, cu = ints(torch, [x + 9 for x in n]), None if step else ints(torch, np.concatenate([[0], np.cumsum(n)]))
    parts = cache4(torch, "plain", 2, 16, Hk, d, 310)
    q, k, v = (rand(torch, 312 + i, (N, h, d), dtype) for i, h in enumerate((2 * Hk, Hk, Hk)))
    was = [t.clone() for t in parts]
    assert torch.equal(paged_append_fp4(k, v, *parts, table, lens, cu, q=q), q)
    assert all(torch.equal(a, b) for a, b in zip(parts, was))
    out = torch.full_like(q, 3.0)
    o, lse = paged_attention_fp4(q, *parts, table, lens, cu, out=out, return_lse=True)
    assert o is out and not out.any() and torch.isneginf(lse).all()


def test_assign_after_a_length_was_set_back(torch):  # noqa: F811
    """A request of 40 tokens in pages 3, 4 and 5, set back to 10: what its table holds past them is written over, and is
    kept where the caller gave it back."""
    for stack, count, page in (([0, 1, 2, -7, -7, -7], 3, 2), ([0, 1, 2, 5, 4, -7], 5, 4)):
        tab, free = ints(torch, [[3, 4, 5, -1]]), ints(torch, stack)
        check_assign(torch, [[3, 4, 5, -1]], [10], [20], stack, [count, 0], 16, 20, None)
        from chunk_gated_delta_carve_amd import paged_assign
        cu, lens, pos, slots, left = paged_assign(tab, ints(torch, [10]), ints(torch, [20]), free, ints(torch, [count, 0]),
                                                  16, 20)
        assert tab[0].tolist() == [3, page, 5, -1] and lens.tolist() == [30] and left.tolist() == [count - 1, 0]
        assert slots.tolist() == [3 * 16 + i for i in range(10, 16)] + [page * 16 + i for i in range(14)]
        kept = set(free[:count - 1].tolist()) | set(tab[0, :2].tolist())
        assert (kept == {0, 1, 2, 3, 4, 5}) == (count == 5)


from test_gpu_attention import SIDE_BY_SIDE  # noqa: E402


@pytest.mark.parametrize("kv", SIDE_BY_SIDE, ids=[str(i) for i in range(len(SIDE_BY_SIDE))])
@pytest.mark.parametrize("dtype,Hq,Hk,d", [("bf16", 16, 2, 128), ("f32", 4, 2, 64)])
def test_short_and_long_contexts_joined_in_one_call(torch, dtype, Hq, Hk, d, kv):  # noqa: F811
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    S = len(kv)
    cu, lens, table, pages = ragged(torch, 41, S, [1] * S, kv, 64)
    parts = cache4(torch, "heads", pages, 64, Hk, d, 320)
    q = rand(torch, 322, (S, Hq, d), dtype)
    args = q, *parts, ints(torch, table), ints(torch, lens)
    out, lse = paged_attention_fp4(*args, return_lse=True)
    kf, vf = (tensor(torch, x) for x in values(parts))
    check_attention(torch, out, lse, q, kf, vf, table, lens, cu, d ** -0.5, 0, dtype)
    assert torch.equal(out, paged_attention_fp4(*args))
