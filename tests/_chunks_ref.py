"""Plain 64-bit restatements of attention over packed chunks, of the attention weights that cached tokens get, and of
leaving the least attended tokens behind.  No code is shared with the library; everything works on CPU and CUDA tensors.

Bounds, beside those of _attn_ref.attend for the outputs (half a step of fp32 is 2^-24 relative; every addition, and the
tensor cores', is taken as off by up to 2^-23 of the sum of magnitudes):
  scores   d = (D + 8) 2^-23 |scale| sum |q_c k_c|, and 2^-20 for the base-2 exponential and its argument
  lse      the largest d of the row, the sum's own relative error (a thread adds 64 weights per 128 tokens two by two, then
           the tiles and the parts), 2^-22 of |lse| and of the largest |score| for the maximum, the logarithm and the factor ln 2
  weights  each term exp(s - lse) is off by a factor e^(d + 2^-20 + 2^-21 |lse| + 2^-22 |s|) (the argument's roundings), the
           sum by 2^-23 of itself per addition
"""
from __future__ import annotations

import math

import torch

import _attn_ref as ref


def values(cache, table_row, n, ps):
    """K and V of the first n tokens, [n, H, D] float64: fp16(code * s + lo), 65504 for what rounds to infinity, NaN for a row
    with parameters that are not finite."""
    t = torch.arange(n, device=cache.device)
    out = []
    for c, s, lo in ref.read_parts(cache, table_row.long()[t // ps] * ps + t % ps):
        x = (c * s + lo).half().double().clamp(-65504.0, 65504.0)
        out.append(torch.where(torch.isfinite(s) & torch.isfinite(lo), x, math.nan))
    return out


def _rows(cu, lens, b):
    n = cu[b + 1] - cu[b]
    return cu[b], n, lens[b] - n  # first row, rows, last token that row 0 sees


def chunks(q, cache, table, cu, lens, scale=None):
    """(o, bound [T, Hq, D], lse, bound [T, Hq]) in float64; rows of no sequence are NaN with bound zero."""
    T, Hq, D = q.shape
    Hkv, ps = cache.shape[1], cache.shape[2] * 16
    G, dev = Hq // Hkv, q.device
    scale = D ** -0.5 if scale is None else scale
    o = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64, device=dev)
    ob, lb = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(len(lens)):
        a, n, c = _rows(cu, lens, b)
        if n <= 0:
            continue
        o[a:a + n], lse[a:a + n] = 0.0, -math.inf
        if lens[b] <= 0:
            continue
        k, v = values(cache, table[b], lens[b], ps)
        unseen = (c + 1 + torch.arange(n, device=dev)).repeat_interleave(G)
        see = torch.arange(lens[b], device=dev)[None] < unseen[:, None]
        some = see.any(-1)
        for h in range(Hkv):
            qh = q[a:a + n, h * G:(h + 1) * G].reshape(n * G, D).double()
            kh, vh = k[:, h], v[:, h]
            oo, bb = ref.attend(qh, kh, vh, kh.abs(), vh.abs(), unseen, scale)
            bad = torch.isnan(vh).any(-1)  # a row of V that is not a number reaches those that see it
            oo = torch.where((see & bad[None]).any(-1)[:, None], math.nan, oo)
            s = torch.where(see, qh @ kh.T * scale, -math.inf)
            z = torch.logsumexp(s, -1)
            d = torch.where(see, qh.abs() @ kh.abs().T * abs(scale), 0.0).amax(-1) * (D + 8) * 2.0 ** -23
            top = torch.where(see, s.abs(), 0.0).amax(-1)
            zb = d + (130 + lens[b] / 128) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * (z.abs() + top)
            o[a:a + n, h * G:(h + 1) * G] = oo.view(n, G, D)
            ob[a:a + n, h * G:(h + 1) * G] = bb.view(n, G, D)
            lse[a:a + n, h * G:(h + 1) * G] = torch.where(some, z, -math.inf).view(n, G)
            lb[a:a + n, h * G:(h + 1) * G] = torch.where(some, zb, 0.0).view(n, G)
    return o, ob, lse, lb


def weights(q, cache, table, cu, lens, lse, before, scale=None):
    """(weights, bound) float64, of before's shape [B, Hkv, cap]."""
    T, Hq, D = q.shape
    Hkv, ps = cache.shape[1], cache.shape[2] * 16
    G, dev = Hq // Hkv, q.device
    scale = D ** -0.5 if scale is None else scale
    out = before.double().clone()
    bound = torch.zeros_like(out)
    for b in range(len(lens)):
        a, n, c = _rows(cu, lens, b)
        if n <= 0 or lens[b] <= 0:
            continue
        k = values(cache, table[b], lens[b], ps)[0]
        last = (c + torch.arange(n, device=dev)).repeat_interleave(G)
        see = torch.arange(lens[b], device=dev)[None] <= last[:, None]
        for h in range(Hkv):
            qh = q[a:a + n, h * G:(h + 1) * G].reshape(n * G, D).double()
            z = lse[a:a + n, h * G:(h + 1) * G].reshape(n * G, 1).double()
            s = qh @ k[:, h].T * scale
            p = torch.where(see, torch.exp(s - z), 0.0)
            d = qh.abs() @ k[:, h].abs().T * (abs(scale) * (D + 8) * 2.0 ** -23)
            off = torch.where(see, p * (d + 2.0 ** -20 + 2.0 ** -21 * z.abs() + 2.0 ** -22 * s.abs()) * 2, 0.0)
            add = p.sum(0)
            out[b, h, :lens[b]] += add
            bound[b, h, :lens[b]] = off.sum(0) + (n * G + 2) * 2.0 ** -23 * add + 2.0 ** -23 * out[b, h, :lens[b]].abs() + 1e-30
    return out, bound


def evict(weights, lens, budget, recent):
    """Tokens kept by each sequence and head, token by token: lists [B][H] of ascending numbers."""
    out = []
    for b, n in enumerate(lens):
        new = min(recent, budget, n)
        heads = []
        for row in weights[b].tolist():
            order = sorted(range(n - new), key=lambda t: (-math.inf if math.isnan(row[t]) else -row[t],
                                                          0 if math.isnan(row[t]) else 1, t))
            heads.append(sorted(order[:min(n, budget) - new] + list(range(n - new, n))))
        out.append(heads)
    return out


def case(lens, new, Hq, Hkv, D, ps, seed, pad=0, lead=0, device="cuda", spread=0.0):
    """(q [T, Hq, D], cache, table, cu list): `lead` rows before the first sequence and `pad` behind the last one."""
    _, cache, table, _ = ref.paged_case(len(lens), lens, 1, Hkv, Hkv, D, ps, seed, device=device, spread=spread)
    g = torch.Generator().manual_seed(seed + 1)
    T = lead + sum(new) + pad
    q = (torch.randn((T, Hq, D), generator=g) * (0.5 + 2 * torch.rand((1, Hq, 1), generator=g))).half().to(device)
    cu = [lead]
    for n in new:
        cu.append(cu[-1] + n)
    return q, cache, table, cu
