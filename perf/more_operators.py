"""Measured cases of the 4-bit paged cache for the attention layer beside the CARVE mixer: pages and slots worked out
on the GPU from request lengths, keys and values stored in 4 bits, read back, and attended to.

The cache holds blocks of 32 channels: 4-bit numbers (sign, two bits of exponent, one of mantissa: 0, 0.5, 1, 1.5, 2, 3,
4, 6), two to a byte with the even channel low, and one byte for the block's scale 2^(byte - 127), 255 for NaN. A block
takes the smallest scale s with max |x| <= 7 s; its numbers are the nearest ones, ties to the even code.

`run` computes an operator in its plain form (elementary torch operations in 32 bits) or, with `own`, through this
package's entry points. `exact` computes it in 64 bits from its definition.
"""
import math

import numpy as np
import torch

own = False

# (query heads, key/value heads, head width): the mixer's own head counts and widths, alone and grouped
HEADS = {"12x64": (12, 12, 64), "12/4x64": (12, 4, 64), "16/4x128": (16, 4, 128), "16/2x128": (16, 2, 128),
         "16x128": (16, 16, 128)}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32
_GOLD = 0.6180339887498949


def listed():
    return [
        # a decode step's bookkeeping: 64 running requests get room for one token each
        dict(name="assign step", op="assign", S=64, n=1, n_min=1, kv=8192, kv_min=17, page=16, done=0, pad=0, short=False),
        # a step that admits prompts while others end: ragged, padded to a fixed number of tokens
        dict(name="assign prompts", op="assign", S=333, n=1021, n_min=0, kv=4096, kv_min=0, page=16, done=57, pad=999,
             short=False),
        # one decode step's append for 64 short chats, and their cache's values
        dict(name="append step", op="append", heads="16/4x128", S=64, n=1, n_min=1, kv=512, kv_min=17, page=16,
             dtype="bf16"),
        # ragged prompts stored at once, fp32, odd lengths, and the cache's values
        dict(name="append prompts f32", op="append", heads="12/4x64", S=7, n=4093, n_min=301, kv=6001, kv_min=4097,
             page=64, dtype="f32"),
        # one short sequence's values in fp32: the smallest call
        dict(name="read short f32", op="read", heads="12x64", S=1, kv=777, kv_min=777, page=16, dtype="f32"),
        # long contexts moved out of the 4-bit cache (the mixer's 65536-token shape)
        dict(name="read long", op="read", heads="16/2x128", S=4, kv=65536, kv_min=50001, page=64, dtype="bf16"),
        # one sequence, one token, short context: latency
        dict(name="decode one", op="attn", heads="12x64", S=1, n=1, n_min=1, kv=1000, kv_min=1000, page=16, window=0,
             lse=False, dtype="bf16"),
        # a serving batch: 64 sequences of ragged length up to 8192
        dict(name="decode batch", op="attn", heads="16/4x128", S=64, n=1, n_min=1, kv=8192, kv_min=200, page=16,
             window=0, lse=False, dtype="bf16"),
        # few sequences with long contexts, few key/value heads
        dict(name="decode long", op="attn", heads="16/2x128", S=4, n=1, n_min=1, kv=65536, kv_min=50001, page=64,
             window=0, lse=True, dtype="bf16"),
        # a prompt chunk over a long cached prefix
        dict(name="chunk over prefix", op="attn", heads="16/4x128", S=1, n=4096, n_min=4096, kv=16384, kv_min=16384,
             page=64, window=0, lse=False, dtype="bf16"),
        # ragged whole prompts of a hybrid's sliding-window layer
        dict(name="prompts window", op="attn", heads="12/4x64", S=8, n=4001, n_min=333, kv=4001, kv_min=333, page=16,
             window=1024, lse=False, dtype="bf16"),
        # fp32, odd sizes, a few new tokens each
        dict(name="attention f32", op="attn", heads="12/4x64", S=5, n=37, n_min=3, kv=2047, kv_min=65, page=16,
             window=0, lse=True, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["assign", "append", "read", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 256])
    if op == "assign":
        S = _log_int(rng, 1, 1024)
        n = _log_int(rng, 1, max(1, min(4096, 300000 // S))) if rng.random() < 0.6 else 1
        kv = _log_int(rng, 1, max(2, min(16384, 4000000 // S)))
        return dict(op=op, S=S, n=n, n_min=rng.randint(0, n), kv=kv, kv_min=rng.randint(0, kv), page=page,
                    done=rng.choice([0, rng.randint(0, S // 2)]), pad=rng.choice([0, _log_int(rng, 1, 1000)]),
                    short=rng.random() < 0.2)
    heads = rng.choice(sorted(HEADS))
    Hq, Hk, d = HEADS[heads]
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    S = _log_int(rng, 1, 64)
    if op == "read":
        kv = _log_int(rng, 1, max(1, min(65536, (1 << 26) // (S * Hk * d))))
        return dict(op=op, heads=heads, S=S, kv=kv, kv_min=rng.randint(1, kv), page=page, dtype=dtype)
    if op == "append":
        n = _log_int(rng, 1, max(1, min(4096, 24000 // S)))
        kv = _log_int(rng, n, max(n, min(8192, 40000 // S)))
        return dict(op=op, heads=heads, S=S, n=n, n_min=rng.randint(1, n), kv=kv, kv_min=rng.randint(n, kv), page=page,
                    dtype=dtype)
    kv = _log_int(rng, 16, 65536)
    while S * kv * Hk * d > 1 << 28:
        S = max(1, S // 2)
        kv = kv if S > 1 else (1 << 28) // (Hk * d)
    cap = (1 << 30) // (16 * S * kv)
    if dtype == "f32":
        cap //= 16
    n = _log_int(rng, 1, max(1, min(4096, kv, cap))) if rng.random() < 0.6 else 1
    return dict(op=op, heads=heads, S=S, n=n, n_min=rng.randint(1, n), kv=kv, kv_min=rng.randint(n, kv), page=page,
                window=rng.choice([0, 0, _log_int(rng, 1, kv)]), lse=rng.choice([False, True]), dtype=dtype)


def _spread(hi, lo, S):
    """S lengths between lo and hi, the first of them hi."""
    return [hi - int((hi - lo) * ((s * _GOLD) % 1.0)) for s in range(S)]


def _up(a, b):
    return -(-a // b)


def _assign_lens(case):
    """(lengths, new tokens, ended or not) of the requests."""
    S = case["S"]
    kv, n = _spread(case["kv"], case["kv_min"], S), _spread(case["n"], case["n_min"], S)
    over = {(s * S) // max(case["done"], 1) for s in range(case["done"])}
    return kv, [0 if s in over else x for s, x in enumerate(n)], [int(s in over) for s in range(S)]


def _seq_lens(case):
    n = _spread(case.get("n", 0), case.get("n_min", 0), case["S"])
    return n, [max(a, b) for a, b in zip(_spread(case["kv"], case["kv_min"], case["S"]), n)]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    S, page = case["S"], case["page"]
    if case["op"] == "assign":
        kv, n, over = _assign_lens(case)
        held = [_up(x, page) for x in kv]
        more = sum(max(0, _up(a + b, page) - _up(a, page)) for a, b, x in zip(kv, n, over) if not x)
        back = sum(h for h, x in zip(held, over) if x)
        free = max(0, (more - back) // 2) if case["short"] else more + 7
        total, width = sum(held) + free, _up(case["kv"] + case["n"], page) + 1
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for s in range(S):
            table[s, :held[s]] = order[at:at + held[s]]
            at += held[s]
        stack = torch.full((total,), -1, dtype=torch.int32, device="cuda")   # the top of the free pages is its end
        stack[:free] = order[at:]
        return dict(case=case, table=table, kv_lens=_i32(kv), new_lens=_i32(n), done=_i32(over) if case["done"] else None,
                    free=stack, count=_i32([free, 0]), N=sum(n) + case["pad"])
    dt = DTYPES[case["dtype"]]
    Hq, Hk, d = HEADS[case["heads"]]

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    n, kv = _seq_lens(case)
    N = sum(n)
    pages = [_up(x, page) for x in kv]
    total = sum(pages) + 3  # a few pages belong to nobody
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((S, max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s in range(S):
        table[s, :pages[s]] = order[at:at + pages[s]]
        at += pages[s]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    st = dict(case=case, Hq=Hq, Hk=Hk, d=d, table=table, kv_lens=_i32(kv), cu=_i32(cu), maxn=max(n), maxkv=max(kv), N=N)
    # the pages hold what earlier tokens left there; a head's tokens are neighbours in memory
    for name in "kv":
        codes, scale = (torch.empty(total, Hk, page, x, dtype=torch.uint8, device="cuda").transpose(1, 2)
                        for x in (d // 2, d // BLOCK))
        for p in range(0, total, 1024):
            codes[p:p + 1024], scale[p:p + 1024] = _to_4bit(randn(min(1024, total - p), page, Hk, d))
        st[name + "_cache"], st[name + "_scale"] = codes, scale
    if case["op"] == "attn":
        st["q"] = randn(N, Hq, d).to(dt)
        return st
    if case["op"] == "append":
        kv_new = randn(N, 2 * Hk, d).mul_(1.5).to(dt)      # keys and values as the two parts of one projection
        st["k"], st["v"] = kv_new[:, :Hk], kv_new[:, Hk:]
    # every token of every sequence, to read it back
    j = torch.arange(st["maxkv"], device="cuda")
    slots = table.long()[:, j // page] * page + j % page
    st["slots"] = slots[j < st["kv_lens"][:, None]].contiguous()
    return st


# the plain forms

def _to_4bit(x):
    """(codes [..., d / 2], scales [..., d / 32]) of x [..., d] in 32 bits."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1)
    m, e = torch.frexp(top)                               # top = m 2^e with m in [1/2, 1)
    byte = (e + 124 + (m > 0.875)).clamp(2, 252)
    byte = torch.where(top == 0, 2, byte)
    bad = ~torch.isfinite(top)
    a = torch.ldexp(b, 127 - byte[..., None])
    z = a.abs()
    code = ((z > 0.25).byte() + (z >= 0.75).byte() + (z > 1.25).byte() + (z >= 1.75).byte() + (z > 2.5).byte()
            + (z >= 3.5).byte() + (z > 5).byte() + 8 * torch.signbit(a).byte())
    code = code.masked_fill(bad[..., None], 0).flatten(-2)
    return code[..., ::2] | code[..., 1::2] << 4, torch.where(bad, 255, byte).byte()


def _from_4bit(codes, scale):
    """The values [..., d] in 32 bits."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    x = table[torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).int()].unflatten(-1, (-1, BLOCK))
    s = torch.ldexp(torch.ones((), device=codes.device), scale.int() - 127).masked_fill(scale == 255, math.nan)
    return (x * s[..., None]).flatten(-2)


def _plain_assign(st):
    c, table, free = st["case"], st["table"], st["free"]
    page, (S, width), F, dev = c["page"], table.shape, free.numel(), table.device
    kv, n = st["kv_lens"].long().clamp(min=0), st["new_lens"].long().clamp(min=0)
    over = torch.zeros_like(kv, dtype=torch.bool) if st["done"] is None else st["done"] != 0
    i = torch.arange(width, device=dev)
    # pages of ended requests go on top of the free ones
    back = over[:, None] & (i < ((kv + page - 1) // page)[:, None]) & (table >= 0)
    rank = back.flatten().long().cumsum(0) - 1
    count = st["count"].long()
    top = count[0].clamp(0, F)
    place = torch.where(back.flatten() & (top + rank < F), top + rank, F)
    free.copy_(torch.cat((free, free[:1])).scatter_(0, place, table.flatten())[:F])
    top = (top + back.sum()).clamp(max=F)
    # and the others take theirs from the top
    old = torch.where(over, 0, kv)
    have, need = ((old + page - 1) // page).clamp(max=width), ((old + n + page - 1) // page).clamp(max=width)
    first = (need - have).cumsum(0) - (need - have)
    at = top - 1 - (first[:, None] + i - have[:, None])
    new = (i >= have[:, None]) & (i < need[:, None])
    table.copy_(torch.where(new, torch.where(at >= 0, free[at.clamp(0, F - 1)], -1), table))
    want = (need - have).sum()
    count = torch.stack(((top - want).clamp(min=0), count[1] + (want - top).clamp(min=0)))
    cu = torch.cat((n.new_zeros(1), n.cumsum(0)))
    t = torch.arange(st["N"], device=dev)
    s = torch.searchsorted(cu[1:], t, right=True)
    real, s = s < S, s.clamp(max=S - 1)
    pos = torch.where(real, old[s] + t - cu[s], 0)
    id = table[s, (pos // page).clamp(max=width - 1)].long()
    slots = torch.where(real & (pos // page < width) & (id >= 0), id * page + pos % page, -1)
    return {"cu_seqlens": cu.int(), "kv_lens": (old + n).int(), "positions": pos.int(), "slots": slots,
            "free_count": count.int(), "block_table": table, "free_pages": free}


def _values(st, name, slots):
    c, page = st["case"], st["case"]["page"]
    p, o = slots // page, slots % page
    return _from_4bit(st[name + "_cache"][p, o], st[name + "_scale"][p, o]).to(DTYPES[c["dtype"]])


def _plain_read(st):
    return {"k": _values(st, "k", st["slots"]), "v": _values(st, "v", st["slots"])}


def _plain_append(st):
    cu, page = st["cu"].long(), st["case"]["page"]
    i = torch.arange(st["N"], device=cu.device)
    s = torch.searchsorted(cu[1:], i, right=True)
    pos = st["kv_lens"].long()[s] - cu[s + 1] + i
    p, o = st["table"].long()[s, pos // page], pos % page
    for name in "kv":
        st[name + "_cache"][p, o], st[name + "_scale"][p, o] = _to_4bit(st[name])
    return _plain_read(st)


def _plain_attn(st):
    c, page, Hq, Hk = st["case"], st["case"]["page"], st["Hq"], st["Hk"]
    G, n, m, d = Hq // Hk, st["maxn"], st["maxkv"], st["d"]
    cu, kv = st["cu"].long(), st["kv_lens"].long()
    j = torch.arange(m, device=cu.device)
    pg, off = st["table"].long()[:, j // page].clamp(min=0), j % page                             # [S, m], [m]
    here = (j < kv[:, None])[:, :, None, None]

    def values(name):
        return _from_4bit(st[name + "_cache"][pg, off], st[name + "_scale"][pg, off]).masked_fill_(~here, 0)

    i = torch.arange(n, device=cu.device)
    rows = (cu[:-1, None] + i).clamp(max=st["N"] - 1)                                             # [S, n]
    q = st["q"][rows].float().unflatten(2, (Hk, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)          # [S, Hk, n G, d]
    k = values("k").permute(0, 2, 3, 1).contiguous()                                              # [S, Hk, d, m]
    x = torch.matmul(q, k).mul_(d ** -0.5).unflatten(2, (n, G))                                   # [S, Hk, n, G, m]
    p = (kv - cu[1:] + cu[:-1])[:, None] + i                                                      # [S, n]
    seen = j <= p[:, :, None]
    if c["window"]:
        seen &= j > p[:, :, None] - c["window"]
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    v = values("v").transpose(1, 2).contiguous()                                                  # [S, Hk, m, d]
    o = torch.matmul(x.flatten(2, 3), v).unflatten(2, (n, G)) / total
    t = torch.arange(st["N"], device=cu.device)
    s = torch.searchsorted(cu[1:], t, right=True)
    o = o.permute(0, 2, 1, 3, 4)[s, t - cu[s]].flatten(1, 2).to(st["q"].dtype)                    # [N, Hq, d]
    if not c["lse"]:
        return o
    lse = (top + total.log())[..., 0].permute(0, 2, 1, 3)[s, t - cu[s]].flatten(1, 2)
    return {"o": o, "lse": lse}


# the framework's calls

def _cache(st):
    return st["k_cache"], st["k_scale"], st["v_cache"], st["v_scale"]


def _own_assign(st):
    from chunk_gated_delta_carve_amd import paged_assign
    cu, lens, positions, slots, count = paged_assign(st["table"], st["kv_lens"], st["new_lens"], st["free"], st["count"],
                                                     st["case"]["page"], st["N"], done=st["done"])
    return {"cu_seqlens": cu, "kv_lens": lens, "positions": positions, "slots": slots, "free_count": count,
            "block_table": st["table"], "free_pages": st["free"]}


def _own_read(st):
    from chunk_gated_delta_carve_amd import paged_read_fp4
    k, v = paged_read_fp4(*_cache(st), st["slots"], dtype=DTYPES[st["case"]["dtype"]])
    return {"k": k, "v": v}


def _own_append(st):
    from chunk_gated_delta_carve_amd import paged_append_fp4
    paged_append_fp4(st["k"], st["v"], *_cache(st), st["table"], st["kv_lens"],
                     None if st["case"]["n"] == 1 else st["cu"])
    return _own_read(st)


def _own_attn(st):
    from chunk_gated_delta_carve_amd import paged_attention_fp4
    c = st["case"]
    r = paged_attention_fp4(st["q"], *_cache(st), st["table"], st["kv_lens"], None if c["n"] == 1 else st["cu"],
                            window=c["window"], return_lse=c["lse"])
    return {"o": r[0], "lse": r[1]} if c["lse"] else r


_PLAIN = {"assign": _plain_assign, "append": _plain_append, "read": _plain_read, "attn": _plain_attn}
_OWN = {"assign": _own_assign, "append": _own_append, "read": _own_read, "attn": _own_attn}


def run(st):
    return (_OWN if own else _PLAIN)[st["case"]["op"]](st)


def work(case):
    S, page = case["S"], case["page"]
    if case["op"] == "assign":
        kv, n, over = _assign_lens(case)
        new = sum(max(0, _up(a + b, page) - _up(a, page)) for a, b, x in zip(kv, n, over) if not x)
        back = sum(_up(a, page) for a, x in zip(kv, over) if x)
        N = sum(n) + case["pad"]
        return {"bytes": S * (4 * 4 + (4 if case["done"] else 0)) + 8 * (new + back) + 12 * N, "flops": S + N}
    Hq, Hk, d = HEADS[case["heads"]]
    es = 4 if case["dtype"] == "f32" else 2
    entry = d // 2 + d // BLOCK                           # bytes of a head's key or value in the cache
    n, kv = _seq_lens(case)
    if case["op"] == "read":
        return {"bytes": sum(kv) * (2 * Hk * (entry + d * es) + 8), "flops": sum(kv) * 2 * Hk * d}
    if case["op"] == "append":
        return {"bytes": sum(n) * 2 * Hk * (d * es + entry) + sum(kv) * (2 * Hk * (entry + d * es) + 8),
                "flops": sum(n) * 2 * Hk * d * 3 + sum(kv) * 2 * Hk * d}
    cells = keys = 0
    for a, b in zip(n, kv):
        w = case["window"] or b
        first = b - a
        keys += b - max(0, first - w + 1)
        # sum over p = first .. b-1 of min(p + 1, w)
        full = max(0, b - max(first, w))
        part = a - full
        cells += full * w + part * (first + 1 + first + part) // 2
    return {"bytes": 2 * sum(n) * Hq * d * es + 2 * keys * Hk * entry + (4 * sum(n) * Hq if case["lse"] else 0),
            "flops": 4 * cells * Hq * d}


# 64 bits, from the definitions

def _exact_codes(x):
    """(sign bit, index into the grid, scale's exponent) of x [..., 32] in 64 bits: the nearest grid point by distance."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    top = x.abs().amax(-1, keepdim=True)
    e = torch.full_like(top, -125.0)
    e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / 7)), e).clamp(-125, 125)
    e = torch.where((top > 7 * 2.0 ** e) & (e < 125), e + 1, e)          # log2 may have landed next to a whole number
    e = torch.where((top <= 7 * 2.0 ** (e - 1)) & (e > -125), e - 1, e)
    far = (x.abs() * 2.0 ** -e).unsqueeze(-1).sub(grid).abs()
    near = far == far.amin(-1, keepdim=True)
    # the nearest, the even one of two
    score = near * (2 - torch.arange(8, device=x.device) % 2)
    return torch.signbit(x), score.argmax(-1), e, grid


def _exact_values(x):
    sign, idx, e, grid = _exact_codes(x.double().unflatten(-1, (-1, BLOCK)))
    return (torch.where(sign, -grid[idx], grid[idx]) * 2.0 ** e).flatten(-2)


def _exact_open(codes, scale):
    c = torch.stack((codes % 16, codes // 16), dim=-1).flatten(-2).double().unflatten(-1, (-1, BLOCK))
    sign, c = 1 - 2 * torch.floor(c / 8), torch.remainder(c, 8)
    ex, man = torch.floor(c / 2), torch.remainder(c, 2)
    size = torch.where(ex == 0, man / 2, (1 + man / 2) * 2.0 ** (ex - 1))
    return (sign * size * 2.0 ** (scale.double() - 127)[..., None]).flatten(-2)


def _exact_assign(st):
    c, page = st["case"], st["case"]["page"]
    table, free = st["table"].cpu().numpy().copy(), st["free"].cpu().numpy().copy()
    kv, n = st["kv_lens"].tolist(), st["new_lens"].tolist()
    over = [0] * c["S"] if st["done"] is None else st["done"].tolist()
    top, lacking = st["count"].tolist()
    lens, cu, positions, slots = [], [0], [], []
    for s in range(c["S"]):
        if over[s]:
            for p in table[s, :_up(kv[s], page)]:
                free[top] = p
                top += 1
    for s in range(c["S"]):
        old = 0 if over[s] else kv[s]
        for i in range(_up(old, page), _up(old + n[s], page)):
            if top > 0:
                top -= 1
                table[s, i] = free[top]
            else:
                lacking += 1
                table[s, i] = -1
        pos = np.arange(old, old + n[s])
        pg = table[s, pos // page].astype(np.int64)
        positions.append(pos)
        slots.append(np.where(pg >= 0, pg * page + pos % page, -1))
        lens.append(old + n[s])
        cu.append(cu[-1] + n[s])
    positions, slots = np.concatenate(positions), np.concatenate(slots)
    pad = st["N"] - len(positions)
    positions, slots = np.pad(positions, (0, pad)), np.pad(slots, (0, pad), constant_values=-1)
    t = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device="cuda")  # noqa: E731
    return {"cu_seqlens": t(cu), "kv_lens": t(lens), "positions": t(positions), "slots": t(slots, torch.int64),
            "free_count": t([top, lacking]), "block_table": t(table), "free_pages": t(free)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "assign":
        return _exact_assign(st)
    page, Hq, Hk, d = case["page"], st["Hq"], st["Hk"], st["d"]
    cu, kv = st["cu"].tolist(), st["kv_lens"].tolist()

    def sequence(name, s):
        pg = st["table"][s, :_up(kv[s], page)].long()
        return _exact_open(st[name + "_cache"][pg].flatten(0, 1)[:kv[s]], st[name + "_scale"][pg].flatten(0, 1)[:kv[s]])

    if case["op"] in ("read", "append"):
        out = {"k": [], "v": []}
        for s in range(case["S"]):
            for name in "kv":
                x = sequence(name, s)
                if case["op"] == "append":
                    x[kv[s] - (cu[s + 1] - cu[s]):] = _exact_values(st[name][cu[s]:cu[s + 1]])
                out[name].append(x)
        return {name: torch.cat(x) for name, x in out.items()}
    if work(case)["flops"] > 1e13:
        return None
    G = Hq // Hk
    o = torch.empty(st["N"], Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["N"], Hq, dtype=torch.float64, device="cuda")
    for s in range(case["S"]):
        k, v = sequence("k", s), sequence("v", s)
        j = torch.arange(kv[s], device="cuda")
        p = torch.arange(kv[s] - (cu[s + 1] - cu[s]), kv[s], device="cuda")[:, None]
        hide = j > p
        if case["window"]:
            hide |= j <= p - case["window"]
        for h in range(Hq):
            x = st["q"][cu[s]:cu[s + 1], h].double() @ k[:, h // G].T / math.sqrt(d)
            x = x.masked_fill(hide, -math.inf)
            o[cu[s]:cu[s + 1], h] = torch.softmax(x, -1) @ v[:, h // G]
            lse[cu[s]:cu[s + 1], h] = torch.logsumexp(x, -1)
    return {"o": o, "lse": lse} if case["lse"] else o
