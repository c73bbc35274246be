"""The attention operators and the paged 4-bit KV cache, as cases to time and compare.

Every case is one pass through one operator:

  plan     kv_plan_pages     block tables and slot maps from request lengths
  cache    kv_append_i4, kv_read_i4   new K and V rows go into the 4-bit cache and are read back
  decode   attention_kv_i4   attention of the last tokens over the paged 4-bit cache
  prompt   attention_prompt  causal attention over packed prompts

``run`` computes them either from elementary torch operations in 32 bits (64 where values sit next to a
rounding border) or, with ``own``, through the package.  ``exact`` gives the definition in 64 bits.

The cache is uint8 [pages, kv heads, page size / 16, 16 (D + 8)]: each block of 16 tokens holds the K codes
[16, D / 2] (channel 2i in the low half of byte i), the V codes [16, D / 2], then (s, lo) fp16 of the 16
K rows and of the 16 V rows; a value is code * s + lo.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


def _gen(seed, salt=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


# ---------------------------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a small batch: a token per request, some of them starting a new page
        {"name": "plan_decode", "op": "plan", "B": 8, "ps": 16, "max_ctx": 4096, "max_new": 1},
        # a large batch with prompts being admitted next to running requests
        {"name": "plan_prompts", "op": "plan", "B": 256, "ps": 64, "max_ctx": 8192, "max_new": 1500},
        # the new tokens of a decode step with grouped heads
        {"name": "cache_decode", "op": "cache", "T": 16, "Hkv": 8, "D": 128, "ps": 16, "fused": True},
        # the prompts of a Llama-7B-shaped layer (32 heads of 128), K and V views of a fused QKV output
        {"name": "cache_prompt", "op": "cache", "T": 8190, "Hkv": 32, "D": 128, "ps": 64, "fused": True},
        # heads of 64, an odd count of tokens
        {"name": "cache_d64", "op": "cache", "T": 4099, "Hkv": 8, "D": 64, "ps": 32, "fused": False},
        # one user, a short context, as many K/V heads as query heads (Llama-7B)
        {"name": "decode_one", "op": "decode", "lens": "one:700", "B": 1, "Lq": 1, "Hq": 32, "Hkv": 32, "D": 128,
         "ps": 16},
        # a serving batch of ragged contexts, grouped heads
        {"name": "decode_batch", "op": "decode", "lens": "ragged:8192", "B": 64, "Lq": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "ps": 64},
        # one user, a long document
        {"name": "decode_long", "op": "decode", "lens": "one:120001", "B": 1, "Lq": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "ps": 64},
        # four drafted tokens to verify per request, a padded batch (some entries empty), heads of 64
        {"name": "decode_verify", "op": "decode", "lens": "padded:6000", "B": 32, "Lq": 4, "Hq": 32, "Hkv": 8, "D": 64,
         "ps": 32},
        # a handful of short chat turns
        {"name": "prompt_short", "op": "prompt", "lens": "ragged:220", "B": 6, "Hq": 32, "Hkv": 32, "D": 128},
        # a prefill batch of packed prompts of very different lengths
        {"name": "prompt_packed", "op": "prompt", "lens": "padded:3700", "B": 9, "Hq": 32, "Hkv": 8, "D": 128},
        # one long document
        {"name": "prompt_long", "op": "prompt", "lens": "one:16384", "B": 1, "Hq": 32, "Hkv": 8, "D": 128},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "cache", "decode", "decode", "prompt", "prompt"])
    ps = rng.choice([16, 32, 64, 128])
    if op == "plan":
        return {"op": op, "B": _log_int(rng, 1, 512), "ps": ps, "max_ctx": _log_int(rng, 16, 16384),
                "max_new": rng.choice([1, _log_int(rng, 1, 700)])}
    D = rng.choice([64, 128, 128])
    if op == "cache":
        Hkv = rng.choice([1, 2, 4, 8, 8, 32])
        return {"op": op, "T": _log_int(rng, 1, 262144 // Hkv), "Hkv": Hkv, "D": D, "ps": ps,
                "fused": rng.random() < 0.5}
    Hkv, G = rng.choice([(1, 8), (2, 4), (2, 7), (4, 1), (8, 4), (8, 4), (8, 8), (8, 1), (32, 1), (4, 16)])
    kind = rng.choice(["one", "ragged", "padded"])
    if op == "decode":
        B = 1 if kind == "one" else _log_int(rng, 2, 96)
        most = 2200000 // (B * Hkv)  # tokens x heads of the largest listed case
        n = _log_int(rng, 1, min(most, 131072))
        return {"op": op, "lens": f"{kind}:{n}", "B": B, "Lq": rng.choice([1, 1, 1, 2, 5]), "Hq": Hkv * G, "Hkv": Hkv,
                "D": D, "ps": ps}
    B = 1 if kind == "one" else _log_int(rng, 2, 24)
    most = int(16384 * math.sqrt(32.0 / (Hkv * G) / B))
    n = _log_int(rng, 1, min(most, 16384))
    return {"op": op, "lens": f"{kind}:{n}", "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D}


def _lens(case, seed):
    """Lengths of the case: one length as stated, or 'ragged' up to it, or the same with empty entries.  The
    shape of the work does not hang on the seed's luck: the longest is always there."""
    kind, n = case["lens"].split(":")
    n, B = int(n), case["B"]
    if kind == "one":
        return [n] * B
    g = torch.Generator().manual_seed(int(seed) + 17)
    order = torch.randperm(B, generator=g).tolist()
    out = [0] * B
    for rank, i in enumerate(order):
        if kind == "padded" and rank % 5 == 4:
            continue
        out[i] = max(1, n - (n * rank) // B - (rank % 7 if n > 64 else 0))
    return out


# ---------------------------------------------------------------------------------------------
# The cache's format, in plain operations
# ---------------------------------------------------------------------------------------------

def _quantise(x, wide):
    """x [..., D] fp16 -> codes, s, lo (s and lo fp16), in `wide` arithmetic."""
    v = x.to(wide)
    lo = v.amin(-1, keepdim=True)
    s = ((v.amax(-1, keepdim=True) - lo) / 15).to(torch.float16)
    s = torch.where(s == 0, torch.ones_like(s), s)
    codes = torch.round((v - lo) / s.to(wide)).clamp_(0, 15).to(torch.uint8)
    return codes, s[..., 0], lo[..., 0].to(torch.float16)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _blocks(cache, D):
    """The parts of the cache's blocks as views [pages, heads, blocks, 16, ...]: K codes, V codes, K (s, lo), V (s, lo)."""
    h = D // 2
    cut = [16 * h, 16 * h, 64, 64]
    kc, vc, kp, vp = torch.split(cache, cut, dim=-1)
    shape = cache.shape[:-1]
    return (kc.unflatten(-1, (16, h)), vc.unflatten(-1, (16, h)),
            kp.view(torch.float16).view(*shape, 16, 2), vp.view(torch.float16).view(*shape, 16, 2))


def _write_rows(cache, D, slots, ps, k, v, wide):
    """Rows k, v [T, heads, D] fp16 into the cache at `slots` (int64, none negative)."""
    page, blk, row = slots // ps, (slots % ps) // 16, slots % 16
    parts = _blocks(cache, D)
    for x, codes_part, par_part in ((k, parts[0], parts[2]), (v, parts[1], parts[3])):
        codes, s, lo = _quantise(x, wide)
        codes_part[page, :, blk, row] = _pack(codes)
        par_part[page, :, blk, row] = torch.stack([s, lo], -1)


def _rows(cache, D, slots, ps, wide):
    """The K and V values at `slots`: [T, heads, D] in `wide`."""
    page, blk, row = slots // ps, (slots % ps) // 16, slots % 16
    parts = _blocks(cache, D)
    out = []
    for codes_part, par_part in ((parts[0], parts[2]), (parts[1], parts[3])):
        c, p = codes_part[page, :, blk, row], par_part[page, :, blk, row].to(wide)
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2).to(wide)
        out.append(c * p[..., 0:1] + p[..., 1:2])
    return out


def _kv_like(T, H, D, g):
    """K with a few channels of large offset, as rotary keys have, and V without; both fp16."""
    k = torch.randn((T, H, D), generator=g, device=DEV)
    off = torch.randn((1, H, D), generator=g, device=DEV)
    k += torch.where(off.abs() > 2.2, 4.0 * off, 0.3 * off)
    v = torch.randn((T, H, D), generator=g, device=DEV)
    v *= torch.rand((T, 1, 1), generator=g, device=DEV) + 0.25
    return k.to(torch.float16), v.to(torch.float16)


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def prepare(case, seed):
    return {"plan": _prepare_plan, "cache": _prepare_cache, "decode": _prepare_decode,
            "prompt": _prepare_prompt}[case["op"]](case, seed)


def _prompt_len(rank, B, most):
    return most - (most - 1) * rank // max(1, (B + 1) // 2)


def _plan_tokens(case):
    B, most = case["B"], case["max_new"]
    return B if most == 1 else B // 2 + sum(_prompt_len(r, B, most) for r in range((B + 1) // 2))


def _prepare_plan(case, seed):
    B, ps = case["B"], case["ps"]
    g = _gen(seed)
    ctx = torch.randint(0, case["max_ctx"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    if case["max_new"] == 1:
        new = torch.ones((B,), device=DEV, dtype=torch.int32)
        new[torch.rand((B,), generator=g, device=DEV) < 0.1] = 0  # finished requests that keep their place
    else:
        rank = torch.randperm(B, generator=g, device=DEV).to(torch.int32)
        half = rank < (B + 1) // 2
        ctx = torch.where(half, torch.zeros_like(ctx), ctx)   # prompts of 1 .. max_new tokens start empty
        new = torch.where(half, _prompt_len(rank, B, case["max_new"]), torch.ones_like(rank))  # running requests: one
    width = (case["max_ctx"] + case["max_new"] + ps - 1) // ps
    held = (ctx + ps - 1) // ps
    most = int(B * width) + 8
    perm = torch.randperm(most, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    col = torch.arange(width, device=DEV)[None]
    first = torch.cumsum(held, 0) - held
    table = torch.where(col < held[:, None], perm[(first[:, None] + col).clamp_(max=most - 1)], -1).to(torch.int32)
    used = int(held.sum())
    free = perm[used:].contiguous()
    T = _plan_tokens(case) + 5 if case["max_new"] > 1 else B  # a padded step
    return {"case": case, "ctx": ctx, "new": new, "table": table, "free": free,
            "free_count": torch.tensor([free.numel()], device=DEV, dtype=torch.int32), "T": T}


def _prepare_cache(case, seed):
    T, H, D, ps = case["T"], case["Hkv"], case["D"], case["ps"]
    g = _gen(seed)
    k, v = _kv_like(T, H, D, g)
    if case["fused"]:  # views of [T, (Hq + 2 Hkv) D] with as many query heads again
        qkv = torch.zeros((T, 3 * H, D), device=DEV, dtype=torch.float16)
        qkv[:, H:2 * H], qkv[:, 2 * H:] = k, v
        k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    pages = (T + ps - 1) // ps + 3
    perm = torch.randperm(pages, generator=g, device=DEV)
    t = torch.arange(T, device=DEV)
    slots = (perm[t // ps] * ps + t % ps).to(torch.int32)
    cache = torch.zeros((pages, H, ps // 16, 16 * (D + 8)), device=DEV, dtype=torch.uint8)
    return {"case": case, "k": k, "v": v, "slots": slots, "cache": cache}


def _prepare_decode(case, seed):
    B, Lq, Hq, Hkv, D, ps = (case[n] for n in ("B", "Lq", "Hq", "Hkv", "D", "ps"))
    lens = _lens(case, seed)
    g = _gen(seed)
    width = max(1, max((n + ps - 1) // ps for n in lens))
    need = sum((n + ps - 1) // ps for n in lens)
    pages = need + 4
    perm = torch.randperm(pages, generator=g, device=DEV)
    table = torch.full((B, width), -1, device=DEV, dtype=torch.int32)
    # what earlier requests left behind: any bytes at all, behind the lengths and in unused pages
    cache = torch.randint(0, 256, (pages, Hkv, ps // 16, 16 * (D + 8)), generator=g, device=DEV, dtype=torch.uint8)
    at = 0
    for i, n in enumerate(lens):
        m = (n + ps - 1) // ps
        table[i, :m] = perm[at:at + m]
        at += m
        for a in range(0, n, 16384):
            t = torch.arange(a, min(n, a + 16384), device=DEV)
            k, v = _kv_like(t.numel(), Hkv, D, g)
            _write_rows(cache, D, table[i].long()[t // ps] * ps + t % ps, ps, k, v, torch.float32)
    q = torch.randn((B, Lq, Hq, D), generator=g, device=DEV)
    q *= 0.5 + torch.rand((B, 1, Hq, 1), generator=g, device=DEV)
    st = {"case": case, "q": q.to(torch.float16), "cache": cache, "table": table, "lens": lens,
          "kv_lens": torch.tensor(lens, device=DEV, dtype=torch.int32),
          "out": torch.empty((B, Lq, Hq, D), device=DEV, dtype=torch.float16)}
    if own:
        import weight_quantized_linear_gb300 as wql
        n = wql.attention_kv_i4_workspace_bytes(B, Lq, Hq, Hkv, D)
        st["workspace"] = torch.empty((n,), device=DEV, dtype=torch.uint8)
    return st


def _prepare_prompt(case, seed):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    lens = _lens(case, seed)
    T = sum(lens)
    g = _gen(seed)
    # views of the fused QKV projection's output
    qkv = torch.empty((T, Hq + 2 * Hkv, D), device=DEV, dtype=torch.float16)
    q = torch.randn((T, Hq, D), generator=g, device=DEV)
    q *= 0.5 + torch.rand((1, Hq, 1), generator=g, device=DEV)
    qkv[:, :Hq] = q.to(torch.float16)
    qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:] = _kv_like(T, Hkv, D, g)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return {"case": case, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv], "v": qkv[:, Hq + Hkv:], "lens": lens,
            "cu": torch.tensor(cu, device=DEV, dtype=torch.int32),
            "out": torch.empty((T, Hq, D), device=DEV, dtype=torch.float16)}


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "cache": _own_cache, "decode": _own_decode, "prompt": _own_prompt}[op](state)
    return {"plan": _plain_plan, "cache": _plain_cache, "decode": _plain_decode, "prompt": _plain_prompt}[op](state)


def _own_plan(st):
    import weight_quantized_linear_gb300 as wql
    slots, cu, kv_lens, left = wql.kv_plan_pages(st["ctx"], st["new"], st["table"], st["free"], st["free_count"],
                                                 st["case"]["ps"], st["T"])
    return {"slots": slots, "cu": cu, "kv_lens": kv_lens, "free_count": left, "table": st["table"]}


def _plain_plan(st):
    ps, T = st["case"]["ps"], st["T"]
    ctx, new, table, free = st["ctx"].long(), st["new"].long(), st["table"], st["free"]
    n_free = st["free_count"].long()
    width = table.shape[1]
    cu = torch.zeros((ctx.numel() + 1,), device=DEV, dtype=torch.int64)
    cu[1:] = torch.cumsum(new, 0)
    held = (ctx + ps - 1) // ps
    total = (ctx + new + ps - 1) // ps
    fits = total <= width
    need = torch.where(fits, total - held, 0)
    off = torch.cumsum(need, 0) - need
    ok = fits & ((need == 0) | (off + need <= n_free))
    left = n_free - torch.where(ok, need, 0).sum()
    col = torch.arange(width, device=DEV)[None]
    fresh = ok[:, None] & (col >= held[:, None]) & (col < total[:, None])
    at = (n_free - 1 - off[:, None] - (col - held[:, None])).clamp_(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[at], table))
    t = torch.arange(T, device=DEV)
    req = (torch.searchsorted(cu, t, right=True) - 1).clamp_(max=ctx.numel() - 1)
    pos = ctx[req] + t - cu[req]
    page = table[req, (pos // ps).clamp_(max=width - 1)].long()
    slots = torch.where((t < cu[-1]) & ok[req], page * ps + pos % ps, -1)
    return {"slots": slots.to(torch.int32), "cu": cu.to(torch.int32),
            "kv_lens": torch.where(ok, ctx + new, 0).to(torch.int32), "free_count": left.to(torch.int32), "table": table}


def _own_cache(st):
    import weight_quantized_linear_gb300 as wql
    wql.kv_append_i4(st["k"], st["v"], st["slots"], st["cache"])
    return wql.kv_read_i4(st["cache"], st["slots"])


def _plain_cache(st):
    D, ps, slots = st["case"]["D"], st["case"]["ps"], st["slots"].long()
    out = ([], [])
    for a in range(0, slots.numel(), 2048):  # 64 bits: whether a value is above a border between two codes
        at = slice(a, a + 2048)
        _write_rows(st["cache"], D, slots[at], ps, st["k"][at], st["v"][at], torch.float64)
        for o, x in zip(out, _rows(st["cache"], D, slots[at], ps, torch.float64)):
            o.append(x.to(torch.float16))
    return tuple(torch.cat(o) for o in out)


def _own_decode(st):
    import weight_quantized_linear_gb300 as wql
    return wql.attention_kv_i4(st["q"], st["cache"], st["table"], st["kv_lens"], out=st["out"],
                               workspace=st["workspace"])


def _plain_decode(st):
    case, q = st["case"], st["q"].float()
    B, Lq, Hq, Hkv, D, ps = (case[n] for n in ("B", "Lq", "Hq", "Hkv", "D", "ps"))
    G = Hq // Hkv
    out = torch.zeros((B, Lq, Hq, D), device=DEV, dtype=torch.float32)
    for i, n in enumerate(st["lens"]):
        if n == 0:
            continue
        t = torch.arange(n, device=DEV)
        k, v = _rows(st["cache"], D, st["table"][i].long()[t // ps] * ps + t % ps, ps, torch.float32)
        qi = q[i].view(Lq, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, Lq * G, D)
        s = (qi @ k.permute(1, 2, 0)) / math.sqrt(D)
        row = torch.arange(Lq, device=DEV).repeat_interleave(G)
        seen = t[None] <= (n - Lq + row)[:, None]
        s = s.masked_fill(~seen[None], -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True).clamp_(min=-3e38))
        o = (p @ v.permute(1, 0, 2)) / p.sum(-1, keepdim=True).clamp_(min=1e-37)
        out[i] = o.view(Hkv, Lq, G, D).permute(1, 0, 2, 3).reshape(Lq, Hq, D)
    return out.to(torch.float16)


def _own_prompt(st):
    import weight_quantized_linear_gb300 as wql
    return wql.attention_prompt(st["q"], st["k"], st["v"], st["cu"], out=st["out"])


def _plain_prompt(st):
    Hq, Hkv, D = (st["case"][n] for n in ("Hq", "Hkv", "D"))
    G = Hq // Hkv
    outs, a = [], 0
    for n in st["lens"]:
        if n == 0:
            continue
        q, k, v = (x[a:a + n].float().permute(1, 0, 2) for x in (st["q"], st["k"], st["v"]))
        a += n
        o = torch.empty((n, Hq, D), device=DEV, dtype=torch.float32)
        for r0 in range(0, n, 4096):
            r1 = min(n, r0 + 4096)
            late = torch.arange(r1, device=DEV)[None] > torch.arange(r0, r1, device=DEV)[:, None]
            step = max(1, min(Hkv, 2 ** 28 // (G * (r1 - r0) * r1)))  # heads at once: 1 GB of scores
            for h in range(0, Hkv, step):
                e = min(Hkv, h + step)
                qh = q[h * G:e * G, r0:r1].reshape(e - h, G * (r1 - r0), D)
                s = (qh @ k[h:e, :r1].mT) / math.sqrt(D)
                s = s.view(e - h, G, r1 - r0, r1).masked_fill_(late, -math.inf)
                p = torch.exp_(s.sub_(s.amax(-1, keepdim=True)))
                y = p.view(e - h, G * (r1 - r0), r1) @ v[h:e, :r1]
                y = y.view((e - h) * G, r1 - r0, D) / p.sum(-1).view((e - h) * G, r1 - r0, 1)
                o[r0:r1, h * G:e * G] = y.permute(1, 0, 2)
        outs.append(o.to(torch.float16))
    return torch.cat(outs) if outs else torch.zeros((0, Hq, D), device=DEV, dtype=torch.float16)


# ---------------------------------------------------------------------------------------------
# The definition in 64 bits, and the work of a pass
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "plan":
        return None  # whole numbers
    if case["op"] == "cache":
        return tuple(_exact_row_values(st[n].double()) for n in ("k", "v"))
    if case["op"] == "decode":
        return _exact_decode(st)
    if sum(n * n for n in st["lens"]) * case["Hq"] * case["D"] > 2 ** 41:
        return None  # too long in 64 bits
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    out = torch.zeros_like(q)
    G, a = case["Hq"] // case["Hkv"], 0
    for n in st["lens"]:
        for h in range(case["Hq"]):
            kh, vh = k[a:a + n, h // G], v[a:a + n, h // G]
            for r in range(0, n, 1024):
                e = min(n, r + 1024)
                w = torch.einsum("id,jd->ij", q[a + r:a + e, h], kh[:e]) * case["D"] ** -0.5
                w = w + torch.full((e - r, e), -math.inf, device=DEV, dtype=torch.float64).triu_(r + 1)
                out[a + r:a + e, h] = torch.einsum("ij,jd->id", torch.softmax(w, 1), vh[:e])
        a += n
    return out


def _exact_row_values(x):
    low, high = x.min(2).values, x.max(2).values
    step = ((high - low) / 15.0).half().double()
    step[step == 0] = 1.0
    n = ((x - low[..., None]) / step[..., None]).round().clamp(max=15.0)
    return low[..., None] + n * step[..., None]


def _exact_decode(st):
    case = st["case"]
    B, Lq, Hq, Hkv, D, ps = (case[n] for n in ("B", "Lq", "Hq", "Hkv", "D", "ps"))
    raw, half = st["cache"], D // 2
    out = torch.zeros((B, Lq, Hq, D), device=DEV, dtype=torch.float64)
    for i, n in enumerate(st["lens"]):
        pages = st["table"][i, :(n + ps - 1) // ps].long()
        for h in range(Hkv if n else 0):
            blocks = raw[pages, h].reshape(-1, 16 * (D + 8))
            kv = []
            for codes, par in ((blocks[:, :16 * half], blocks[:, 32 * half:32 * half + 64]),
                               (blocks[:, 16 * half:32 * half], blocks[:, 32 * half + 64:])):
                codes = codes.reshape(-1, half)[:n]
                par = par.contiguous().view(torch.float16).reshape(-1, 2)[:n].double()
                x = torch.empty((n, D), device=DEV, dtype=torch.float64)
                x[:, 0::2], x[:, 1::2] = (codes % 16).double(), (codes // 16).double()
                kv.append(x * par[:, :1] + par[:, 1:])
            for r in range(Lq):
                see = n - Lq + r + 1
                if see > 0:
                    heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                    w = torch.softmax(st["q"][i, r, heads].double() @ kv[0][:see].T * D ** -0.5, 1)
                    out[i, r, heads] = w @ kv[1][:see]
    return out


def work(case):
    op = case["op"]
    if op == "plan":
        B, new = case["B"], case["max_new"]
        tokens = _plan_tokens(case)
        pages = tokens / case["ps"] + (B / 2 if new > 1 else 0)
        return {"bytes": int(B * 20 + tokens * 4 + pages * 8), "flops": int(tokens * 4 + B * 8)}
    D = case["D"]
    if op == "cache":
        rows = case["T"] * case["Hkv"]
        # the rows in, the cache's entries written, their values out
        return {"bytes": rows * (4 * D + D + 8 + 4 * D) + 4 * case["T"], "flops": rows * 12 * D}
    Hq, Hkv, lens = case["Hq"], case["Hkv"], _lens(case, 0)
    if op == "decode":
        B, Lq = case["B"], case["Lq"]
        pairs = sum(max(0, n - Lq + r + 1) for n in lens for r in range(Lq))
        return {"bytes": sum(lens) * Hkv * (D + 8) + B * Lq * Hq * D * 4 + sum(lens) // case["ps"] * 4,
                "flops": 4 * D * Hq * pairs}
    return {"bytes": sum(lens) * (2 * Hq + 2 * Hkv) * D * 2, "flops": 2 * D * Hq * sum(n * (n + 1) for n in lens)}
