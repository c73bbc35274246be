"""Plain 64-bit restatements of the paged 4-bit KV cache, the page plan and the attention over both kinds of K and V,
with elementwise error bounds derived from the roundings that include/wql.h allows.  No code is shared with the
library.  Everything works on CPU and CUDA tensors.

Bounds (half a step of fp16 is u = 2^-11 relative, 2^-25 below 2^-14; fp32 sums are off by at most 2^-23 of the sum
of magnitudes per addition, which also covers tensor-core sums that truncate):
  scores   d = (D + 8) 2^-23 scale sum |q_c k_c|, with |k_c| <= code s + |lo| for the 4-bit cache, plus 2^-20 for the
           base-2 exponential and its argument
  weights  each is off by a factor e^d, then rounded to fp16: u relative, or 2^-25 absolute against weights whose
           largest is at least 2^-8 of 1 (a running maximum may lag by 2^8 upwards, which only helps)
  output   u |o| for the last rounding (2^-25 below 2^-14), 2^-18 |o| for the sums and the division
"""
from __future__ import annotations

import math

import numpy as np
import torch

U16 = 2.0 ** -11


def quantise(x: torch.Tensor):
    """x [..., D] fp16 -> (codes uint8, s fp16 [...], lo fp16 [...]) in exact-enough 64-bit arithmetic."""
    v = x.double()
    lo, hi = v.min(-1, keepdim=True).values, v.max(-1, keepdim=True).values
    finite = torch.isfinite(v).all(-1, keepdim=True)
    s = ((hi - lo) / 15).half()
    s = torch.where(s == 0, torch.ones_like(s), s)
    c = torch.round((v - lo) / s.double()).clamp(0, 15)
    c = torch.where(finite, c, torch.zeros_like(c)).to(torch.uint8)
    nan = torch.full_like(s, math.nan)
    return c, torch.where(finite, s, nan)[..., 0], torch.where(finite, lo.half(), nan)[..., 0]


def write(cache: torch.Tensor, slots, k: torch.Tensor, v: torch.Tensor) -> None:
    """Rows k, v [T, H, D] into the cache [pages, H, blocks, 16 (D + 8)] at slots (negative ones passed over)."""
    D = k.shape[-1]
    ps = cache.shape[2] * 16
    slots = torch.as_tensor(slots, device=cache.device).long()
    keep = slots >= 0
    slots, k, v = slots[keep], k[keep], v[keep]
    if slots.numel() == 0:
        return
    page, blk, row = slots // ps, slots % ps // 16, slots % 16
    h = D // 2
    for x, c_at, p_at in ((k, 0, 32 * h), (v, 16 * h, 32 * h + 64)):
        c, s, lo = quantise(x)
        packed = c[..., 0::2] + 16 * c[..., 1::2]  # [T, H, h]
        par = torch.stack([s, lo], -1).contiguous().view(torch.uint8)  # [T, H, 4]
        cache[:, :, :, c_at:c_at + 16 * h].unflatten(-1, (16, h))[page, :, blk, row] = packed
        cache[:, :, :, p_at:p_at + 64].unflatten(-1, (16, 4))[page, :, blk, row] = par


def read_parts(cache: torch.Tensor, slots):
    """(codes, s, lo) of K and of V at slots: codes [T, H, D] float64, s and lo [T, H, 1] float64."""
    D = cache.shape[3] // 16 - 8
    ps = cache.shape[2] * 16
    h = D // 2
    slots = torch.as_tensor(slots, device=cache.device).long()
    page, blk, row = slots // ps, slots % ps // 16, slots % 16
    out = []
    for c_at, p_at in ((0, 32 * h), (16 * h, 32 * h + 64)):
        c = cache[:, :, :, c_at:c_at + 16 * h].unflatten(-1, (16, h))[page, :, blk, row]
        par = cache[:, :, :, p_at:p_at + 64].unflatten(-1, (16, 4))[page, :, blk, row].contiguous().view(torch.float16)
        codes = torch.stack([c % 16, c // 16], -1).flatten(-2).double()
        out.append((codes, par[..., 0:1].double(), par[..., 1:2].double()))
    return out


def read(cache: torch.Tensor, slots):
    """The fp16 values of K and V at slots (code * s + lo has at most 40 bits: exact in 64, rounded once)."""
    return [(c * s + lo).half() for c, s, lo in read_parts(cache, slots)]


def attend(q, k, v, kmag, vmag, first_unseen, scale):
    """One K/V head: q [R, D], k, v [n, D] float64, keys t < first_unseen[r] visible.  kmag, vmag bound |k| and the
    factor that the rounded weight multiplies.  Returns (o [R, D], bound [R, D])."""
    R, D = q.shape
    n = k.shape[0]
    o, b = torch.zeros((R, D), dtype=torch.float64, device=q.device), None
    b = torch.zeros_like(o)
    see = torch.arange(n, device=q.device)[None] < first_unseen[:, None]
    some = see.any(-1)
    if not bool(some.any()):
        return o, b
    s = torch.where(see, q @ k.T * scale, -math.inf)
    d = torch.where(see, (q.abs() @ kmag.T) * abs(scale), 0.0).amax(-1, keepdim=True) * (D + 8) * 2.0 ** -23 + 2.0 ** -20
    top = s.amax(-1, keepdim=True).clamp(min=-1e300)
    e = torch.exp(s - top)
    l = e.sum(-1, keepdim=True).clamp(min=1e-300)
    zero_v, zero_m = torch.nan_to_num(v), torch.nan_to_num(vmag)
    o = e @ zero_v / l
    size = e @ zero_m / l
    spread = e @ zero_v.abs() / l
    seen = see.double()
    under = 2.0 ** -25 * (seen @ zero_m) / l * 2.0  # every weight may lie below fp16's normal numbers
    b = 2 * d * (spread + o.abs()) + U16 * size + under + (U16 + 2.0 ** -18) * o.abs() + 2.0 ** -25
    return torch.where(some[:, None], o, 0.0), torch.where(some[:, None], b, 0.0)


def kv_i4(q, cache, table, lens, scale=None):
    """(o, bound) float64 [B, Lq, Hq, D] of attention over the 4-bit cache."""
    B, Lq, Hq, D = q.shape
    Hkv, ps = cache.shape[1], cache.shape[2] * 16
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        t = torch.arange(n, device=q.device)
        slots = table[b].long()[t // ps] * ps + t % ps
        (kc, ks, klo), (vc, vs, vlo) = read_parts(cache, slots)
        k, v = kc * ks + klo, vc * vs + vlo
        kmag, vmag = kc * ks + klo.abs(), vc * vs
        # a weight below fp16's normal range is off by 2^-25 of the largest p s, not of 1
        unseen = (n - Lq + 1 + torch.arange(Lq, device=q.device)).repeat_interleave(G)
        for h in range(Hkv):
            qh = q[b, :, h * G:(h + 1) * G].reshape(Lq * G, D).double()
            oo, bb = attend(qh, k[:, h], v[:, h], kmag[:, h], vmag[:, h], unseen, scale)
            extra = 2.0 ** -25 * 2 * 15 * n * float(torch.nan_to_num(vs[:, h]).max())
            o[b, :, h * G:(h + 1) * G] = oo.view(Lq, G, D)
            bound[b, :, h * G:(h + 1) * G] = (bb + extra * (bb > 0)).view(Lq, G, D)
    return o, bound


def prompt(q, k, v, cu, scale=None):
    """(o, bound) float64 [T, Hq, D] of causal attention over packed prompts (rows of no sequence are NaN)."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    o = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    for a, e in zip(cu[:-1], cu[1:]):
        if e <= a:
            continue
        for h in range(Hq):
            kk, vv = k[a:e, h // G].double(), v[a:e, h // G].double()
            for r in range(a, e, 2048):
                z = min(e, r + 2048)
                unseen = torch.arange(r - a + 1, z - a + 1, device=q.device)
                o[r:z, h], bound[r:z, h] = attend(q[r:z, h].double(), kk[:z - a], vv[:z - a], kk[:z - a].abs(),
                                                  vv[:z - a].abs(), unseen, scale)
    return o, bound


def plan(ctx, new, table, free, n_free, ps, T):
    """The page plan, request by request.  Returns (slots, cu, kv_lens, left, table) as numpy int32."""
    table = np.array(table, dtype=np.int64)
    n_free = min(max(int(n_free), 0), len(free))
    slots = np.full((T,), -1, dtype=np.int64)
    cu, kv_lens, before, taken = [0], [], 0, 0
    for i, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(int(c), 0), max(int(n), 0)
        held, total = -(-c // ps), -(-(c + n) // ps)
        need = total - held if total <= table.shape[1] else None
        ok = need is not None and (need == 0 or before + need <= n_free)
        if ok:
            for j in range(need):
                table[i, held + j] = free[n_free - 1 - before - j]
            taken += need
            for j in range(n):
                if cu[-1] + j < T:
                    page = table[i, (c + j) // ps]
                    slots[cu[-1] + j] = page * ps + (c + j) % ps if page >= 0 else -1
        before += need or 0
        kv_lens.append(c + n if ok else 0)
        cu.append(cu[-1] + n)
    i32 = lambda x: np.asarray(x, dtype=np.int32)  # noqa: E731
    return i32(slots), i32(cu), i32(kv_lens), n_free - taken, i32(table)


def paged_case(B, lens, Lq, Hq, Hkv, D, ps, seed, device="cuda", spread=0.0):
    """A cache of random bytes (so that what no request holds is anything at all, NaN params included) with the
    requests' rows written into shuffled pages.  spread: decades over which V's magnitude varies between tokens."""
    g = torch.Generator().manual_seed(seed)
    width = max(1, max(-(-n // ps) for n in lens)) + 1
    pages = sum(-(-n // ps) for n in lens) + 3
    perm = torch.randperm(pages, generator=g)
    cache = torch.randint(0, 256, (pages, Hkv, ps // 16, 16 * (D + 8)), generator=g, dtype=torch.uint8).to(device)
    table = torch.full((B, width), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // ps)
        table[b, :m] = perm[at:at + m]
        at += m
        k = torch.randn((n, Hkv, D), generator=g) + 1.5 * torch.randn((1, Hkv, D), generator=g)
        v = torch.randn((n, Hkv, D), generator=g) * 10.0 ** (spread * (torch.rand((n, 1, 1), generator=g) - 0.5))
        t = torch.arange(n)
        slots = table[b].long()[t // ps] * ps + t % ps
        write(cache, slots.to(device), k.half().to(device), v.half().to(device))
    q = (torch.randn((B, Lq, Hq, D), generator=g) * (0.5 + 2 * torch.rand((B, 1, Hq, 1), generator=g))).half().to(device)
    return q, cache, table.to(device), torch.tensor(lens, dtype=torch.int32, device=device)
