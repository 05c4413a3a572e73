"""Measured cases of the attention-layer operators that stand beside the CARVE mixer in a hybrid model:
per-head norm and rotation of queries and keys (forward and backward), appending to a paged cache,
and attention of new tokens over that cache.

`run` computes an operator in its plain form (elementary torch operations in 32 bits) or, with `own`,
through this package's entry points. `exact` computes it in 64 bits from its definition.
"""
import math

import torch

own = False

# (query heads, key/value heads, head width): the mixer's own head counts and widths, alone and grouped
HEADS = {"12x64": (12, 12, 64), "12/4x64": (12, 4, 64), "16/4x128": (16, 4, 128), "16/2x128": (16, 2, 128),
         "16x128": (16, 16, 128)}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
_GOLD = 0.6180339887498949


def listed():
    return [
        # one decode step's queries and keys, 64 sequences: the smallest call, where latency counts
        dict(name="rope step", op="rope", heads="16/2x128", B=64, T=1, rot=128, inter=False, dtype="bf16"),
        # a training step's projections at the mixer's default shape (B4 T2048, 12 heads of 64)
        dict(name="rope train", op="rope", heads="12x64", B=4, T=2048, rot=64, inter=False, dtype="bf16"),
        # the gradient at the long training shape (B4 T8192, 16 query heads of 128)
        dict(name="rope grad", op="rope_bwd", heads="16/4x128", B=4, T=8192, rot=128, inter=False, dtype="bf16"),
        # fp32 gradient, odd length, partial rotation of adjacent pairs
        dict(name="rope grad f32 odd", op="rope_bwd", heads="12/4x64", B=3, T=1001, rot=32, inter=True, dtype="f32"),
        # one decode step's append for 64 sequences of different lengths
        dict(name="append step", op="append", heads="16/4x128", S=64, n=1, n_min=1, kv=8192, kv_min=17, page=16,
             rot=128, inter=False, norm=True, dtype="bf16"),
        # ragged prompts appended at once, queries prepared in the same call
        dict(name="append prompts", op="append", heads="16/4x128", S=7, n=4096, n_min=301, kv=6000, kv_min=4096,
             page=64, rot=128, inter=False, norm=True, dtype="bf16"),
        # one sequence, one token, short context: latency
        dict(name="decode one", op="attn", heads="12x64", S=1, n=1, n_min=1, kv=1000, kv_min=1000, page=16,
             window=0, lse=False, dtype="bf16"),
        # a serving batch: 64 sequences of ragged length up to 8192
        dict(name="decode batch", op="attn", heads="16/4x128", S=64, n=1, n_min=1, kv=8192, kv_min=200, page=16,
             window=0, lse=False, dtype="bf16"),
        # few sequences with long contexts (the mixer's 65536-token shape), few key/value heads
        dict(name="decode long", op="attn", heads="16/2x128", S=4, n=1, n_min=1, kv=65536, kv_min=50001, page=64,
             window=0, lse=False, dtype="bf16"),
        # a prompt chunk over a long cached prefix
        dict(name="chunk over prefix", op="attn", heads="16/4x128", S=1, n=4096, n_min=4096, kv=16384, kv_min=16384,
             page=64, window=0, lse=True, dtype="bf16"),
        # ragged whole prompts of a hybrid's sliding-window layer
        dict(name="prompts window", op="attn", heads="12/4x64", S=8, n=4096, n_min=333, kv=4096, kv_min=333, page=16,
             window=1024, lse=False, dtype="bf16"),
        # fp32, odd sizes, a few new tokens each
        dict(name="attention f32", op="attn", heads="12/4x64", S=5, n=37, n_min=3, kv=2047, kv_min=65, page=16,
             window=0, lse=True, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "attn", "attn", "attn"])
    heads = rng.choice(sorted(HEADS))
    Hq, Hk, d = HEADS[heads]
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    rot = rng.choice([d, d, d // 2])
    inter = rng.choice([False, True])
    if op in ("rope", "rope_bwd"):
        T = _log_int(rng, 1, 8192)
        B = _log_int(rng, 1, max(1, min(64, 32768 * 24 * 128 // (T * (Hq + Hk) * d * (2 if dtype == "f32" else 1)))))
        return dict(op=op, heads=heads, B=B, T=T, rot=rot, inter=inter, dtype=dtype)
    S, page = _log_int(rng, 1, 64), rng.choice([16, 32, 64, 256])
    if op == "append":
        n = _log_int(rng, 1, max(1, min(4096, 24000 // S)))
        kv = _log_int(rng, n, max(n, min(16384, 65536 // S)))
        return dict(op=op, heads=heads, S=S, n=n, n_min=rng.randint(1, n), kv=kv, kv_min=rng.randint(n, kv), page=page,
                    rot=rot, inter=inter, norm=rng.choice([False, True]), dtype=dtype)
    kv = _log_int(rng, 16, 65536)
    while S * kv * Hk * d > 1 << 29:
        S = max(1, S // 2)
        kv = kv if S > 1 else (1 << 29) // (Hk * d)
    cap = (1 << 30) // (16 * S * kv)
    if dtype == "f32":
        cap //= 16
    n = _log_int(rng, 1, max(1, min(4096, kv, cap))) if rng.random() < 0.6 else 1
    return dict(op=op, heads=heads, S=S, n=n, n_min=rng.randint(1, n), kv=kv, kv_min=rng.randint(n, kv), page=page,
                window=rng.choice([0, 0, _log_int(rng, 1, kv)]), lse=rng.choice([False, True]), dtype=dtype)


def _spread(hi, lo, S):
    """S lengths between lo and hi, the first of them hi."""
    return [hi - int((hi - lo) * ((s * _GOLD) % 1.0)) for s in range(S)]


def _tables(length, rot, device):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(length, dtype=torch.float64, device=device)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    Hq, Hk, d = HEADS[case["heads"]]

    def randn(*shape, scale=1.0, add=0.0):
        return torch.randn(shape, generator=g, device=dev).mul_(scale).add_(add).to(dt)

    st = dict(case=case, Hq=Hq, Hk=Hk, d=d)
    if case["op"] in ("rope", "rope_bwd"):
        B, T = case["B"], case["T"]
        # queries and keys as the two parts of one projection's output
        qk = randn(B, T, Hq + Hk, d, scale=1.5)
        st["q"], st["k"] = qk[:, :, :Hq], qk[:, :, Hq:]
        st["q_weight"], st["k_weight"] = randn(d, scale=0.1, add=1.0), randn(d, scale=0.1, add=1.0)
        if T == 1:  # decode: every sequence at a place of its own
            st["cos"], st["sin"] = _tables(8192, case["rot"], dev)
            st["positions"] = torch.randint(0, 8192, (B, T), generator=g, device=dev, dtype=torch.int32)
        else:
            st["cos"], st["sin"] = _tables(T, case["rot"], dev)
            st["positions"] = None
        if case["op"] == "rope_bwd":
            st["dq"], st["dk"] = randn(B, T, Hq, d), randn(B, T, Hk, d)
        return st
    S, page = case["S"], case["page"]
    n = _spread(case["n"], case["n_min"], S)
    kv = [max(a, b) for a, b in zip(_spread(case["kv"], case["kv_min"], S), n)]
    N, width = sum(n), -(-max(kv) // page)
    pages = [-(-x // page) for x in kv]
    total = sum(pages) + 3  # a few pages belong to nobody
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for s in range(S):
        table[s, :pages[s]] = order[at:at + pages[s]]
        at += pages[s]
    st["table"] = table
    st["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=dev)
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    st["maxn"], st["maxkv"], st["N"] = max(n), max(kv), N
    # pages hold what earlier sequences left there
    st["k_cache"], st["v_cache"] = randn(total, page, Hk, d), randn(total, page, Hk, d)
    st["q"] = randn(N, Hq, d)
    if case["op"] == "append":
        st["k"], st["v"] = randn(N, Hk, d, scale=1.5), randn(N, Hk, d)
        st["cos"], st["sin"] = _tables(max(kv), case["rot"], dev)
        w = case["norm"]
        st["q_weight"] = randn(d, scale=0.1, add=1.0) if w else None
        st["k_weight"] = randn(d, scale=0.1, add=1.0) if w else None
    return st


# the plain forms

def _turn(x, cos, sin, rot, inter, back=False):
    """Rotate the first `rot` channels of x [..., H, d] by tables [..., 1, rot/2]; `back` turns the other way."""
    if back:
        sin = -sin
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _norm_rope(x, w, cos, sin, rot, inter, norm):
    z = x.float()
    if norm:
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS)
        if w is not None:
            z = z * w.float()
    return _turn(z, cos, sin, rot, inter).to(x.dtype)


def _norm_rope_bwd(x, w, dy, cos, sin, rot, inter):
    z, dz = x.float(), _turn(dy.float(), cos, sin, rot, inter, back=True)
    r = torch.rsqrt(z.square().mean(-1, keepdim=True) + EPS)
    n = z * r
    dw = (dz * n).sum(dim=(0, 1, 2))
    dn = dz * w.float()
    return (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(x.dtype), dw


def _rope_tables(st):
    p = st["positions"]
    if p is None:
        return st["cos"][None, :, None], st["sin"][None, :, None]
    return st["cos"][p.long()][:, :, None], st["sin"][p.long()][:, :, None]


def _plain_rope(st):
    c = st["case"]
    cos, sin = _rope_tables(st)
    return {n: _norm_rope(st[n], st[n + "_weight"], cos, sin, c["rot"], c["inter"], True) for n in ("q", "k")}


def _plain_rope_bwd(st):
    c = st["case"]
    cos, sin = _rope_tables(st)
    dq, dqw = _norm_rope_bwd(st["q"], st["q_weight"], st["dq"], cos, sin, c["rot"], c["inter"])
    dk, dkw = _norm_rope_bwd(st["k"], st["k_weight"], st["dk"], cos, sin, c["rot"], c["inter"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _plain_append(st):
    c, cu, page = st["case"], st["cu"].long(), st["case"]["page"]
    i = torch.arange(st["N"], device=cu.device)
    s = torch.searchsorted(cu[1:], i, right=True)
    p = st["kv_lens"].long()[s] - cu[s + 1] + i
    slot = st["table"].long()[s, p // page] * page + p % page
    cos, sin = st["cos"][p][:, None], st["sin"][p][:, None]
    rope = lambda x, w: _norm_rope(x, w, cos, sin, c["rot"], c["inter"], c["norm"])  # noqa: E731
    st["k_cache"].flatten(0, 1).index_copy_(0, slot, rope(st["k"], st["k_weight"]))
    st["v_cache"].flatten(0, 1).index_copy_(0, slot, st["v"])
    return {"q": rope(st["q"], st["q_weight"]), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_attn(st):
    c, page, Hq, Hk, d = st["case"], st["case"]["page"], st["Hq"], st["Hk"], st["d"]
    G, S, n, m = Hq // Hk, c["S"], st["maxn"], st["maxkv"]
    cu, kv = st["cu"].long(), st["kv_lens"].long()
    j = torch.arange(m, device=cu.device)
    slot = st["table"].long()[:, j // page].clamp(min=0) * page + j % page                        # [S, m]
    here = (j < kv[:, None])[:, :, None, None]
    k = st["k_cache"].flatten(0, 1)[slot].float().masked_fill(~here, 0).permute(0, 2, 3, 1)       # [S, Hk, d, m]
    v = st["v_cache"].flatten(0, 1)[slot].float().masked_fill(~here, 0).transpose(1, 2)           # [S, Hk, m, d]
    i = torch.arange(n, device=cu.device)
    rows = (cu[:-1, None] + i).clamp(max=st["N"] - 1)                                             # [S, n]
    q = st["q"][rows].float().unflatten(2, (Hk, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)          # [S, Hk, n G, d]
    x = torch.matmul(q, k.contiguous()).mul_(d ** -0.5).unflatten(2, (n, G))                      # [S, Hk, n, G, m]
    p = (kv - cu[1:] + cu[:-1])[:, None] + i                                                      # [S, n]
    seen = j <= p[:, :, None]
    if c["window"]:
        seen &= j > p[:, :, None] - c["window"]
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), v.contiguous()).unflatten(2, (n, G)) / total
    t = torch.arange(st["N"], device=cu.device)
    s = torch.searchsorted(cu[1:], t, right=True)
    o = o.permute(0, 2, 1, 3, 4)[s, t - cu[s]].flatten(1, 2).to(st["q"].dtype)                    # [N, Hq, d]
    if not c["lse"]:
        return o
    lse = (top + total.log())[..., 0].permute(0, 2, 1, 3)[s, t - cu[s]].flatten(1, 2)
    return {"o": o, "lse": lse}


# the framework's calls

def _own_rope(st):
    from chunk_gated_delta_carve_amd import qk_norm_rope_fwd
    q, k = qk_norm_rope_fwd(st["q"], st["k"], st["cos"], st["sin"], st["positions"], st["q_weight"], st["k_weight"],
                            eps=EPS, interleaved=st["case"]["inter"])
    return {"q": q, "k": k}


def _own_rope_bwd(st):
    from chunk_gated_delta_carve_amd import qk_norm_rope_bwd
    return qk_norm_rope_bwd(st["q"], st["k"], st["dq"], st["dk"], st["cos"], st["sin"], st["positions"],
                            st["q_weight"], st["k_weight"], eps=EPS, interleaved=st["case"]["inter"])


def _own_append(st):
    from chunk_gated_delta_carve_amd import paged_append
    c = st["case"]
    q = paged_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["kv_lens"],
                     None if c["n"] == 1 else st["cu"], st["cos"], st["sin"], q=st["q"], q_weight=st["q_weight"],
                     k_weight=st["k_weight"], norm=c["norm"], eps=EPS, interleaved=c["inter"])
    return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _own_attn(st):
    from chunk_gated_delta_carve_amd import paged_attention
    c = st["case"]
    r = paged_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["kv_lens"],
                        None if c["n"] == 1 else st["cu"], window=c["window"], return_lse=c["lse"])
    return {"o": r[0], "lse": r[1]} if c["lse"] else r


_PLAIN = {"rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "append": _plain_append, "attn": _plain_attn}
_OWN = {"rope": _own_rope, "rope_bwd": _own_rope_bwd, "append": _own_append, "attn": _own_attn}


def run(st):
    return (_OWN if own else _PLAIN)[st["case"]["op"]](st)


def work(case):
    Hq, Hk, d = HEADS[case["heads"]]
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("rope", "rope_bwd"):
        tokens = case["B"] * case["T"]
        table = min(case["T"] if case["T"] > 1 else case["B"], 8192) * case["rot"] * 4
        back = case["op"] == "rope_bwd"
        return {"bytes": tokens * (Hq + Hk) * d * es * (3 if back else 2) + table,
                "flops": tokens * (Hq + Hk) * d * (14 if back else 8)}
    n = _spread(case["n"], case["n_min"], case["S"])
    kv = [max(a, b) for a, b in zip(_spread(case["kv"], case["kv_min"], case["S"]), n)]
    if case["op"] == "append":
        N = sum(n)
        return {"bytes": 2 * N * (Hq + 2 * Hk) * d * es + N * case["rot"] * 4, "flops": N * (Hq + Hk) * d * 8}
    cells = keys = 0
    for a, b in zip(n, kv):
        w = case["window"] or b
        first = b - a
        keys += b - max(0, first - w + 1)
        # sum over p = first .. b-1 of min(p + 1, w)
        full = max(0, b - max(first, w))
        part = (a - full)
        cells += full * w + part * (first + 1 + first + part) // 2
    return {"bytes": (2 * sum(n) * Hq * d + 2 * keys * Hk * d) * es + (4 * sum(n) * Hq if case["lse"] else 0),
            "flops": 4 * cells * Hq * d}


# 64 bits, from the definitions

def _exact_matrix(cos, sin, rot, d, inter):
    """Rotation of one position as the pair of gather indices and coefficients: y = x * a + x[idx] * b."""
    h = rot // 2
    a = torch.ones(cos.shape[:-1] + (d,), dtype=torch.float64, device=cos.device)
    b = torch.zeros_like(a)
    idx = torch.arange(d, device=cos.device)
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, h), slice(h, rot))
    first, second = idx[lo].clone(), idx[hi].clone()
    a[..., lo], a[..., hi] = cos.double(), cos.double()
    b[..., lo], b[..., hi] = -sin.double(), sin.double()
    idx[lo], idx[hi] = second, first
    return a, b, idx


def _exact_rows(x, w, cos, sin, case, norm):
    a, b, idx = _exact_matrix(cos, sin, case["rot"], x.shape[-1], case["inter"])
    z = x.double()
    if norm:
        z = z / (z.pow(2).sum(-1, keepdim=True) / z.shape[-1] + EPS).sqrt()
    if w is not None:
        z = z * w.double()
    return z * a + z[..., idx] * b


def _exact_grad(x, w, dy, cos, sin, case):
    x, w = x.double().clone().requires_grad_(True), w.double().clone().requires_grad_(True)
    with torch.enable_grad():
        y = _exact_rows(x, w, cos, sin, case, True)
        dx, dw = torch.autograd.grad(y, (x, w), dy.double())
    return dx, dw


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("rope", "rope_bwd"):
        B, T = case["B"], case["T"]
        p = st["positions"].long() if st["positions"] is not None else torch.arange(T, device="cuda").expand(B, T)
        cos, sin = st["cos"][p].unsqueeze(2), st["sin"][p].unsqueeze(2)
        if case["op"] == "rope":
            return {n: _exact_rows(st[n], st[n + "_weight"], cos, sin, case, True) for n in ("q", "k")}
        dq, dqw = _exact_grad(st["q"], st["q_weight"], st["dq"], cos, sin, case)
        dk, dkw = _exact_grad(st["k"], st["k_weight"], st["dk"], cos, sin, case)
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    page, Hq, Hk, d = case["page"], st["Hq"], st["Hk"], st["d"]
    cu, kv = st["cu"].tolist(), st["kv_lens"].tolist()
    if case["op"] == "append":
        kc, vc, q = st["k_cache"].double(), st["v_cache"].double(), torch.empty_like(st["q"], dtype=torch.float64)
        for s in range(case["S"]):
            new = slice(cu[s], cu[s + 1])
            p = torch.arange(kv[s] - (cu[s + 1] - cu[s]), kv[s], device="cuda")
            pg, off = st["table"][s].long()[p // page], p % page
            cos, sin = st["cos"][p].unsqueeze(1), st["sin"][p].unsqueeze(1)
            kc[pg, off] = _exact_rows(st["k"][new], st["k_weight"], cos, sin, case, case["norm"])
            vc[pg, off] = st["v"][new].double()
            q[new] = _exact_rows(st["q"][new], st["q_weight"], cos, sin, case, case["norm"])
        return {"q": q, "k_cache": kc, "v_cache": vc}
    if work(case)["flops"] > 1e13:
        return None
    G = Hq // Hk
    o = torch.empty(st["N"], Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["N"], Hq, dtype=torch.float64, device="cuda")
    for s in range(case["S"]):
        pg = st["table"][s, :-(-kv[s] // page)].long()
        k = st["k_cache"][pg].flatten(0, 1)[:kv[s]].double()
        v = st["v_cache"][pg].flatten(0, 1)[:kv[s]].double()
        j = torch.arange(kv[s], device="cuda")
        p = torch.arange(kv[s] - (cu[s + 1] - cu[s]), kv[s], device="cuda")[:, None]
        hide = (j > p) | ((j <= p - case["window"]) if case["window"] else torch.zeros((), dtype=torch.bool, device="cuda"))
        for h in range(Hq):
            x = st["q"][cu[s]:cu[s + 1], h].double() @ k[:, h // G].T / math.sqrt(d)
            x = x.masked_fill(hide, -math.inf)
            o[cu[s]:cu[s + 1], h] = torch.softmax(x, -1) @ v[:, h // G]
            lse[cu[s]:cu[s + 1], h] = torch.logsumexp(x, -1)
    return {"o": o, "lse": lse} if case["lse"] else o
