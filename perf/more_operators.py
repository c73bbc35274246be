"""Long contexts in the paged 4-bit KV cache, as cases to time and compare: chunks of new tokens attend to the
cache, the tokens' attention weights are added up, and the least attended tokens are left behind.

Every case is one pass through one operator:

  chunk    attention_chunks_kv_i4   attention of packed chunks of new tokens over the paged cache, with the logarithm
                                    of each row's sum of exponentials
  weights  kv_weights_i4            the attention weight that every cached token gets from the chunks, added up
  evict    kv_evict_i4              the heaviest and the newest tokens go into new pages, the others stay behind

``run`` computes them either from elementary torch operations in 32 bits or, with ``own``, through the package.
``exact`` gives the definition in 64 bits.

The cache is uint8 [pages, kv heads, page size / 16, 16 (D + 8)]: each block of 16 tokens holds the K codes
[16, D / 2] (channel 2i in the low half of byte i), the V codes [16, D / 2], then (s, lo) fp16 of the 16
K rows and of the 16 V rows.  A value is code * s + lo, rounded to fp16 as kv_read_i4 gives it.
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
# The cases.  lens: tokens of each sequence, the new ones among them; new: how many of those are queried.
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # the last tokens of a short prompt behind a shared beginning, as many K/V heads as query heads (Llama-7B)
        {"name": "chunk_tail", "op": "chunk", "lens": "each:716", "new": "each:16", "B": 1, "Hq": 32, "Hkv": 32, "D": 128,
         "ps": 16},
        # a decode step of a serving batch whose weights are wanted afterwards: one token each, ragged contexts
        {"name": "chunk_steps", "op": "chunk", "lens": "ragged:8192", "new": "each:1", "B": 64, "Hq": 32, "Hkv": 8, "D": 128,
         "ps": 64},
        # a step of continuous batching: chunks of three prompts among running requests, some refused, heads of 64
        {"name": "chunk_mixed", "op": "chunk", "lens": "padded:6000", "new": "mixed:500", "B": 24, "Hq": 32, "Hkv": 8, "D": 64,
         "ps": 32},
        # chunked prefill: 512 tokens behind a long document
        {"name": "chunk_512", "op": "chunk", "lens": "each:16384", "new": "each:512", "B": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "ps": 64},
        # large chunks of four prompts, as many K/V heads as query heads (Llama-7B)
        {"name": "chunk_2048", "op": "chunk", "lens": "ragged:8190", "new": "each:2048", "B": 4, "Hq": 32, "Hkv": 32, "D": 128,
         "ps": 128},
        # what the last tokens of a long document looked at
        {"name": "weights_window", "op": "weights", "lens": "each:32768", "new": "each:32", "B": 1, "Hq": 32, "Hkv": 8,
         "D": 128, "ps": 64},
        # weights added up in a decode step
        {"name": "weights_steps", "op": "weights", "lens": "ragged:8192", "new": "each:1", "B": 64, "Hq": 32, "Hkv": 8,
         "D": 128, "ps": 64},
        # weights of whole prompts of different lengths, one request refused
        {"name": "weights_prompts", "op": "weights", "lens": "padded:4099", "new": "whole:0", "B": 5, "Hq": 32, "Hkv": 8,
         "D": 64, "ps": 32},
        # a small batch makes room for its next tokens
        {"name": "evict_small", "op": "evict", "lens": "each:1024", "budget": 960, "recent": 64, "B": 4, "Hkv": 8, "D": 128,
         "ps": 16},
        # half of the tokens of a serving batch, short requests keep all of theirs
        {"name": "evict_batch", "op": "evict", "lens": "ragged:4096", "budget": 2048, "recent": 256, "B": 64, "Hkv": 8,
         "D": 128, "ps": 64},
        # a long document after its prefill
        {"name": "evict_long", "op": "evict", "lens": "each:120001", "budget": 16384, "recent": 1000, "B": 1, "Hkv": 8,
         "D": 128, "ps": 64},
        # 32 K/V heads of 64, odd lengths, empty places in the batch
        {"name": "evict_d64", "op": "evict", "lens": "padded:3001", "budget": 1777, "recent": 0, "B": 24, "Hkv": 32, "D": 64,
         "ps": 32},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "weights", "evict"])
    ps, D = rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 128])
    kind = rng.choice(["each", "ragged", "padded"])
    B = rng.choice([1, 1, 2, 3]) if kind == "each" else _log_int(rng, 2, 64)
    Hkv, G = rng.choice([(1, 8), (2, 4), (2, 7), (4, 1), (8, 4), (8, 4), (8, 8), (8, 1), (32, 1), (4, 16), (3, 5)])
    if op == "evict":
        Hkv = rng.choice([1, 2, 8, 8, 32])
        n = _log_int(rng, 1, min(131072, 2000000 // (B * Hkv)))
        budget = _log_int(rng, 1, n + 40)
        return {"op": op, "lens": f"{kind}:{n}", "budget": budget, "recent": rng.choice([0, 1, budget // 8, budget]), "B": B,
                "Hkv": Hkv, "D": D, "ps": ps}
    how = rng.choice(["each", "each", "mixed", "whole"])
    if how == "whole":  # rows x tokens x heads of all sequences, padded, below those of the largest listed case
        n = _log_int(rng, 1, int(math.sqrt(1.5e9 / (B * Hkv * G))))
        return {"op": op, "lens": f"{kind}:{n}", "new": "whole:0", "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "ps": ps}
    n = _log_int(rng, 1, min(131072, 2000000 // (B * Hkv)))
    new = _log_int(rng, 1, max(1, min(n, 2048, int(1.2e9 / (B * n * Hkv * G)))))
    return {"op": op, "lens": f"{kind}:{n}", "new": f"{how}:{new}", "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "ps": ps}


def _lens(case, seed):
    """(tokens of each sequence, new ones of each): one length for all, 'ragged' up to it, or the same with places of
    refused requests, which have a new token but none in the cache.  The work does not hang on the seed: it only shuffles."""
    kind, n = case["lens"].split(":")
    n, B = int(n), case["B"]
    how, m = case.get("new", "each:0").split(":")
    g = torch.Generator().manual_seed(int(seed) + 17)
    lens, new = [0] * B, [0] * B
    for rank, i in enumerate(torch.randperm(B, generator=g).tolist()):
        if kind == "padded" and rank % 5 == 4:
            new[i] = 1
            continue
        lens[i] = n if kind == "each" else max(1, n - (n * rank) // B - (rank % 7 if n > 64 else 0))
        most = {"each": int(m), "mixed": max(1, int(m) - 37 * (rank // 8)) if rank % 8 == 0 else 1, "whole": lens[i]}[how]
        new[i] = min(lens[i], most)
    return lens, new


# ---------------------------------------------------------------------------------------------
# The cache's format, in plain operations
# ---------------------------------------------------------------------------------------------

def _blocks(cache, D):
    """The parts of the cache's blocks as views [pages, heads, blocks, 16, ...]: K codes, V codes, K (s, lo), V (s, lo)."""
    h = D // 2
    kc, vc, kp, vp = torch.split(cache, [16 * h, 16 * h, 64, 64], dim=-1)
    shape = cache.shape[:-1]
    return (kc.unflatten(-1, (16, h)), vc.unflatten(-1, (16, h)),
            kp.view(torch.float16).view(*shape, 16, 2), vp.view(torch.float16).view(*shape, 16, 2))


def _values(codes, par, wide):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(wide)
    return (c * par[..., 0:1].to(wide) + par[..., 1:2].to(wide)).to(torch.float16).to(wide)


def _padded_kv(cache, D, table, ps, L, both=True):
    """K and V of tokens 0 .. L - 1 of each row of the table, [B, heads, L, D] fp32; anything behind a row's pages."""
    t = torch.arange(L, device=DEV)
    page = table.long()[:, t // ps].clamp_(min=0)
    blk, row = ((t % ps) // 16)[None], (t % 16)[None]
    parts = _blocks(cache, D)
    return [_values(codes[page, :, blk, row], par[page, :, blk, row], torch.float32).transpose(1, 2)
            for codes, par in ((parts[0], parts[2]), (parts[1], parts[3]))[:2 if both else 1]]


def _pack_rows(x, pages, ps):
    """fp16 rows [pages * ps, heads, D] as codes [pages, heads, ps / 16, 16, D / 2] and (s, lo) as bytes [.., 16, 4]."""
    v = x.float()
    lo = v.amin(-1, keepdim=True)
    s = ((v.amax(-1, keepdim=True) - lo) / 15).to(torch.float16)
    s = torch.where(s == 0, torch.ones_like(s), s)
    c = torch.round((v - lo) / s.float()).clamp_(0, 15).to(torch.uint8)
    par = torch.cat([s, lo.to(torch.float16)], -1).view(torch.uint8)
    return [y.unflatten(0, (pages, ps // 16, 16)).permute(0, 3, 1, 2, 4) for y in (c[..., 0::2] | (c[..., 1::2] << 4), par)]


def _make_cache(lens, Hkv, D, ps, g, spare):
    """A cache with the sequences' tokens in shuffled pages, `spare` pages more, and anything at all (what earlier requests
    left) in the places that hold no token; the block table; the spare pages."""
    B = len(lens)
    held = torch.tensor([(n + ps - 1) // ps for n in lens], device=DEV)
    width, used = max(1, int(held.max())), int(held.sum())
    pages = used + spare
    perm = torch.randperm(pages, generator=g, device=DEV)
    col = torch.arange(width, device=DEV)[None]
    first = torch.cumsum(held, 0) - held
    mine = col < held[:, None]
    table = torch.where(mine, perm[(first[:, None] + col).clamp_(max=pages - 1)], -1).to(torch.int32)
    fill = torch.zeros((pages,), device=DEV, dtype=torch.int64)  # tokens of each page
    fill[table[mine].long()] = (torch.tensor(lens, device=DEV)[:, None] - col * ps).clamp(max=ps)[mine]
    k = torch.randn((pages * ps, Hkv, D), generator=g, device=DEV)
    off = torch.randn((1, Hkv, D), generator=g, device=DEV)  # a few channels of large offset, as rotary keys have
    k += torch.where(off.abs() > 2.2, 4.0 * off, 0.3 * off)
    v = torch.randn((pages * ps, Hkv, D), generator=g, device=DEV)
    v *= torch.rand((pages * ps, 1, 1), generator=g, device=DEV) + 0.25
    kc, kp = _pack_rows(k.to(torch.float16), pages, ps)
    vc, vp = _pack_rows(v.to(torch.float16), pages, ps)
    token = (torch.arange(ps, device=DEV)[None] < fill[:, None]).view(pages, 1, ps // 16, 16, 1)
    parts = []
    for part in (kc, vc, kp, vp):
        left = torch.randint(0, 256, part.shape, generator=g, device=DEV, dtype=torch.uint8)
        parts.append(torch.where(token, part, left).flatten(-2))
    return torch.cat(parts, -1), table, perm[used:].to(torch.int32)


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = _gen(seed)
    lens, new = _lens(case, seed)
    B, Hkv, D, ps = (case[n] for n in ("B", "Hkv", "D", "ps"))
    kv_lens = torch.tensor(lens, device=DEV, dtype=torch.int32)
    if case["op"] == "evict":
        width = (case["budget"] + 256 + ps - 1) // ps  # room for the kept tokens and the next 256
        held = [(min(n, case["budget"]) + ps - 1) // ps for n in lens]
        cache, table, free = _make_cache(lens, Hkv, D, ps, g, sum(held) + 2)
        col = torch.arange(width, device=DEV)[None]
        h = torch.tensor(held, device=DEV)
        first = torch.cumsum(h, 0) - h
        new_table = torch.where(col < h[:, None], free[(first[:, None] + col).clamp_(max=free.numel() - 1)], -1)
        # sums of attention weights: a few heavy tokens, many light ones, some never looked at
        w = torch.randn((B, Hkv, table.shape[1] * ps), generator=g, device=DEV).mul_(2.5).exp_()
        w[torch.rand(w.shape, generator=g, device=DEV) < 0.2] = 0.0
        return {"case": case, "cache": cache, "table": table, "kv_lens": kv_lens, "new_table": new_table.to(torch.int32),
                "weights": w}
    Hq = case["Hq"]
    T = sum(new) + 3  # a padded step: the last rows belong to nobody
    cache, table, _ = _make_cache(lens, Hkv, D, ps, g, 4)
    # a view of the fused QKV projection's output
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEV)
    qkv[:, :Hq] *= 0.5 + torch.rand((1, Hq, 1), generator=g, device=DEV)
    cu = torch.zeros((B + 1,), dtype=torch.int64)
    cu[1:] = torch.cumsum(torch.tensor(new), 0)
    st = {"case": case, "q": qkv.to(torch.float16)[:, :Hq], "cache": cache, "table": table, "kv_lens": kv_lens,
          "cu": cu.to(device=DEV, dtype=torch.int32), "longest": (max(lens), max(new))}
    if case["op"] == "chunk":
        st["out"] = torch.zeros((T, Hq, D), device=DEV, dtype=torch.float16)
        st["lse"] = torch.zeros((T, Hq), device=DEV)
    else:  # what attention over the chunks left, and the sums so far
        st["lse"] = _plain_chunk(st)[1]
        st["weights"] = torch.rand((B, Hkv, table.shape[1] * ps), generator=g, device=DEV)
        st["weights"][torch.arange(table.shape[1] * ps, device=DEV)[None, None].expand_as(st["weights"])
                      >= (kv_lens - (cu[1:] - cu[:-1]).to(DEV))[:, None, None]] = 0.0
    return st


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"chunk": _own_chunk, "weights": _own_weights, "evict": _own_evict}[op](state)
    return {"chunk": _plain_chunk, "weights": _plain_weights, "evict": _plain_evict}[op](state)


def _own_chunk(st):
    import weight_quantized_linear_gb300 as wql
    if "workspace" not in st:  # a program keeps one
        n = wql.attention_chunks_kv_i4_workspace_bytes(st["q"].shape[0], st["kv_lens"].shape[0], st["q"].shape[1],
                                                       st["cache"].shape[1], st["q"].shape[2])
        st["workspace"] = torch.empty((n,), device=DEV, dtype=torch.uint8)
    wql.attention_chunks_kv_i4(st["q"], st["cache"], st["table"], st["cu"], st["kv_lens"], out=st["out"], lse=st["lse"],
                               workspace=st["workspace"])
    return st["out"], st["lse"]


def _own_weights(st):
    import weight_quantized_linear_gb300 as wql
    return wql.kv_weights_i4(st["q"], st["cache"], st["table"], st["cu"], st["kv_lens"], st["lse"], st["weights"])


def _own_evict(st):
    import weight_quantized_linear_gb300 as wql
    kept, weights, lens = wql.kv_evict_i4(st["weights"], st["cache"], st["table"], st["kv_lens"], st["new_table"],
                                          st["case"]["budget"], st["case"]["recent"])
    # rows are moved, not computed: the cache's bytes are compared as the whole numbers that they are
    return {"kept": kept, "weights": weights, "lens": lens, "cache": st["cache"]}


def _scores(st, k):
    """Scaled scores [B, Hkv, rows, G, L] of each sequence's new tokens, padded to the longest; those that a row does not see
    are minus infinity."""
    Hq, Hkv, D = (st["case"][n] for n in ("Hq", "Hkv", "D"))
    L, rows = st["longest"]
    B, G = st["kv_lens"].numel(), Hq // Hkv
    cu, lens = st["cu"].long(), st["kv_lens"].long()
    n = cu[1:] - cu[:-1]
    r = torch.arange(rows, device=DEV)
    q = st["q"][(cu[:-1, None] + r).clamp_(max=st["q"].shape[0] - 1)].float()  # [B, rows, Hq, D]
    q = q.view(B, rows, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, rows * G, D)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, rows, G, L)
    last = torch.where(r < n[:, None], (lens - n)[:, None] + r, -1)  # the last token that a row sees
    late = torch.arange(L, device=DEV) > last[..., None]
    return s.masked_fill_(late[:, None, :, None], -math.inf)


def _row_of(st):
    """Sequence and row in it of each token of q, and whether it is of a sequence at all."""
    cu = st["cu"].long()
    t = torch.arange(st["q"].shape[0], device=DEV)
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp_(max=cu.numel() - 2)
    return b, (t - cu[b]).clamp_(max=st["longest"][1] - 1), t < cu[-1]


def _plain_chunk(st):
    case = st["case"]
    Hq, Hkv, D = (case[n] for n in ("Hq", "Hkv", "D"))
    L, rows = st["longest"]
    B, G = st["kv_lens"].numel(), Hq // Hkv
    k, v = _padded_kv(st["cache"], D, st["table"], case["ps"], L)
    behind = torch.arange(L, device=DEV)[None] >= st["kv_lens"][:, None]
    v.masked_fill_(behind[:, None, :, None], 0.0)
    s = _scores(st, k)
    m = s.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, rows * G, L), v).view(B, Hkv, rows, G, D) / total.clamp(min=1e-37)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)[..., 0]
    b, r, some = _row_of(st)
    out = torch.where(some[:, None, None], o.transpose(1, 2).reshape(B, rows, Hq, D)[b, r], 0.0)
    return out.to(torch.float16), torch.where(some[:, None], lse.transpose(1, 2).reshape(B, rows, Hq)[b, r], 0.0)


def _plain_weights(st):
    case = st["case"]
    Hq, Hkv, D = (case[n] for n in ("Hq", "Hkv", "D"))
    L, rows = st["longest"]
    B, G = st["kv_lens"].numel(), Hq // Hkv
    k, = _padded_kv(st["cache"], D, st["table"], case["ps"], L, both=False)
    r = torch.arange(rows, device=DEV)
    at = (st["cu"].long()[:-1, None] + r).clamp_(max=st["q"].shape[0] - 1)
    lse = st["lse"][at].view(B, rows, Hkv, G).transpose(1, 2)[..., None]
    s = _scores(st, k)
    p = torch.where(s > -math.inf, torch.exp(s - lse), 0.0)
    st["weights"][:, :, :L] += p.sum((2, 3))
    return st["weights"]


def _plain_evict(st):
    case, w = st["case"], st["weights"]
    ps, D, budget = case["ps"], case["D"], case["budget"]
    B, H, cap = w.shape
    lens = st["kv_lens"].long()
    t = torch.arange(cap, device=DEV)[None]
    new = t >= (lens - min(case["recent"], budget))[:, None]
    key = torch.where(new[:, None], math.inf, w).masked_fill((t >= lens[:, None])[:, None], -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    if cap < budget:
        order = torch.nn.functional.pad(order, (0, budget - cap))
    n_kept = lens.clamp(max=budget)
    i = torch.arange(budget, device=DEV)
    there = (i < n_kept[:, None])[:, None]
    kept = torch.sort(torch.where(there, order[..., :budget], cap), dim=-1).values
    there = there.expand_as(kept)
    b, h, at = torch.nonzero(there, as_tuple=True)
    src = kept[there]
    page, to = st["table"][b, src // ps].long(), st["new_table"][b, at // ps].long()
    for part in _blocks(st["cache"], D):
        part[to, h, (at % ps) // 16, at % 16] = part[page, h, (src % ps) // 16, src % 16]
    weights = torch.zeros((B, H, st["new_table"].shape[1] * ps), device=DEV)
    weights[b, h, at] = w[b, h, src]
    return {"kept": torch.where(there, kept, -1).to(torch.int32), "weights": weights, "lens": n_kept.to(torch.int32),
            "cache": st["cache"]}


# ---------------------------------------------------------------------------------------------
# The definition in 64 bits, and the work of a pass
# ---------------------------------------------------------------------------------------------

def _exact_rows(st, i, head, n, which):
    """K (0) or V (1) of the first n tokens of sequence i, [n, D] fp64."""
    case = st["case"]
    half, ps = case["D"] // 2, case["ps"]
    pages = st["table"][i, :(n + ps - 1) // ps].long()
    blocks = st["cache"][pages, head].reshape(-1, 16 * (case["D"] + 8))
    codes = blocks[:, 16 * half * which:16 * half * (which + 1)].reshape(-1, half)[:n]
    par = blocks[:, 32 * half + 64 * which:32 * half + 64 * which + 64].contiguous().view(torch.float16).reshape(-1, 2)[:n].double()
    x = torch.empty((n, case["D"]), device=DEV, dtype=torch.float64)
    x[:, 0::2], x[:, 1::2] = (codes % 16).double(), (codes // 16).double()
    return x.mul_(par[:, :1]).add_(par[:, 1:]).half().double()


def exact(case, seed):
    if case["op"] == "evict":
        return _exact_evict(prepare(case, seed))
    lens, new = _lens(case, seed)
    if sum(n * m for n, m in zip(lens, new)) * case["Hq"] * case["D"] > 2 ** 41:
        return None  # too long in 64 bits
    st = prepare(case, seed)
    Hq, Hkv, D = (case[n] for n in ("Hq", "Hkv", "D"))
    G, T = Hq // Hkv, st["q"].shape[0]
    out = torch.zeros((T, Hq, D), device=DEV, dtype=torch.float64)
    lse = torch.zeros((T, Hq), device=DEV, dtype=torch.float64)
    weights = st["weights"].double() if case["op"] == "weights" else None
    a = 0
    for i, (n, m) in enumerate(zip(lens, new)):
        lse[a:a + m] = -math.inf
        for h in range(Hkv if n else 0):
            k, heads = _exact_rows(st, i, h, n, 0), slice(h * G, (h + 1) * G)
            v = _exact_rows(st, i, h, n, 1) if weights is None else None
            for r in range(0, m, 512):
                e = min(m, r + 512)
                z = torch.einsum("rgd,td->grt", st["q"][a + r:a + e, heads].double(), k) / math.sqrt(D)
                z = z + torch.full((e - r, n), -math.inf, device=DEV, dtype=torch.float64).triu_(n - m + r + 1)
                if weights is None:
                    out[a + r:a + e, heads] = torch.einsum("grt,td->rgd", torch.softmax(z, -1), v)
                    lse[a + r:a + e, heads] = torch.logsumexp(z, -1).T
                else:
                    weights[i, h, :n] += torch.exp(z - st["lse"][a + r:a + e, heads].double().T[..., None]).sum((0, 1))
        a += m
    return (out, lse) if weights is None else weights


def _exact_evict(st):
    """The sums that go with the kept tokens, found by counting the heavier ones; the rest are whole numbers."""
    case, w = st["case"], st["weights"].double()
    lens, budget = st["kv_lens"].tolist(), case["budget"]
    if sum(n * n for n in lens) * case["Hkv"] > 2 ** 38:
        return None
    B, H, _ = w.shape
    weights = torch.zeros((B, H, st["new_table"].shape[1] * case["ps"]), device=DEV, dtype=torch.float64)
    for i, n in enumerate(lens):
        old = max(0, n - min(case["recent"], budget))
        for h in range(H):
            x, t = w[i, h, :old], torch.arange(old, device=DEV)
            ahead = torch.zeros((old,), device=DEV, dtype=torch.int64)
            for a in range(0, old, 4096):
                y, u = x[a:a + 4096, None], t[a:a + 4096, None]
                ahead[a:a + 4096] = ((x > y) | ((x == y) & (t < u))).sum(1)
            stay = torch.cat([ahead < budget - (n - old), torch.ones((n - old,), device=DEV, dtype=torch.bool)])
            weights[i, h, :min(n, budget)] = w[i, h, :n][stay]
    return {"kept": None, "weights": weights, "lens": None, "cache": None}


def work(case):
    lens, new = _lens(case, 0)
    Hkv, D, ps = case["Hkv"], case["D"], case["ps"]
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        room = (case["budget"] + 256 + ps - 1) // ps * ps * len(lens)
        # the sums, the kept rows read and written, their places, and their sums with the zeros behind them
        return {"bytes": Hkv * (4 * sum(lens) + kept * 2 * (D + 8) + 4 * case["budget"] * len(lens) + 4 * room),
                "flops": Hkv * sum(lens)}
    Hq = case["Hq"]
    pairs = sum(m * n - m * (m - 1) // 2 for n, m in zip(lens, new) if n)
    tables = sum((n + ps - 1) // ps for n in lens) * 4
    if case["op"] == "weights":
        return {"bytes": sum(lens) * Hkv * (D // 2 + 4 + 8) + sum(new) * Hq * (2 * D + 4) + tables, "flops": 2 * D * Hq * pairs}
    return {"bytes": sum(lens) * Hkv * (D + 8) + sum(new) * Hq * (4 * D + 4) + tables, "flops": 4 * D * Hq * pairs}
