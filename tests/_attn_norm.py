"""A sharp criterion for attention over the 4-bit cache: the error of an output row, as a vector, against what its
roundings can come to when their signs are independent.  Works on CPU and CUDA tensors; shares no code with the library.

Token t enters a row's output with its weight p_t, whose rounding (u = 2^-11 relative, half a step of fp16) meets
s_t (code_t - 7.5), and whose score's error (d relative, the worst case of tests/_attn_ref.py) meets v_t - o.  So its
vector of errors is no longer than
    a_t = p_t (u |s_t| |code_t - 7.5| + d |v_t - o|) + w 2^-32 |code_t - 7.5|,   w the largest p |s| of the row:
a weight below 2^-14, fp16's normal numbers, is off by 2^-25 where the largest one is at least 2^7.  A constant row of V
(all codes 0, whatever its s) adds its value exactly.  n vectors with independent signs add up to
3 sqrt(sum a_t^2) with room to spare (a rounding's error is 0.41 u on average, so that this is seven standard deviations;
for n <= 9 no signs can exceed it), where their worst case grows with n.  The output's own rounding adds u |o|, or 2^-25 per
channel below 2^-14.
"""
from __future__ import annotations

import math

import torch

import _attn_ref as ref

U16 = 2.0 ** -11


def rows(q, k, v, dev, smax, kmag, unseen, scale, drop=None):
    """One K/V head: q [R, D], k, v, kmag [n, D], dev = s (code - 7.5) [n, D], smax [n] = |s|, float64; keys t < unseen[r]
    visible, but for token `drop`.  Returns (o [R, D], tolerance [R])."""
    D, n = q.shape[1], k.shape[0]
    see = torch.arange(n, device=q.device)[None] < unseen[:, None]
    if drop is not None:
        see[:, drop] = False
    s = torch.where(see, q @ k.T * scale, -math.inf)
    d = torch.where(see, (q.abs() @ kmag.T) * abs(scale), 0.0).amax(-1, keepdim=True) * (D + 8) * 2.0 ** -23 + 2.0 ** -20
    e = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300))
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
    o = p @ v
    far = (v.square().sum(-1)[None] + o.square().sum(-1, keepdim=True) - 2 * o @ v.T).clamp(min=0).sqrt()
    size = dev.norm(dim=-1)[None]
    units = torch.where(smax > 0, size[0] / smax.clamp(min=1e-30), size[0])[None]  # |code - 7.5|
    a = p * (U16 * size + d * far) + 2.0 ** -32 * (p * smax[None]).amax(-1, keepdim=True) * units * see
    tol = 3 * a.square().sum(-1).sqrt() + (U16 * o).square().sum(-1).sqrt() + D ** 0.5 * 2.0 ** -25
    return o, tol


def kv_i4(q, cache, table, lens, scale=None, drop=None):
    """(o [B, Lq, Hq, D], tolerance [B, Lq, Hq]) float64 of attention over the 4-bit cache."""
    B, Lq, Hq, D = q.shape
    Hkv, ps = cache.shape[1], cache.shape[2] * 16
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros(q.shape[:3], dtype=torch.float64, device=q.device)
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        t = torch.arange(n, device=q.device)
        (kc, ks, klo), (vc, vs, vlo) = ref.read_parts(cache, table[b].long()[t // ps] * ps + t % ps)
        some = vc.any(-1, keepdim=True)
        k, v, dev = kc * ks + klo, vc * vs + vlo, torch.where(some, vs * (vc - 7.5), 0.0)
        smax, kmag = torch.where(some, vs.abs(), 0.0)[..., 0], kc * ks.abs() + klo.abs()
        unseen = (n - Lq + 1 + torch.arange(Lq, device=q.device)).repeat_interleave(G)
        for h in range(Hkv):
            qh = q[b, :, h * G:(h + 1) * G].reshape(Lq * G, D).double()
            y, x = rows(qh, k[:, h], v[:, h], dev[:, h], smax[:, h], kmag[:, h], unseen, scale, drop)
            o[b, :, h * G:(h + 1) * G], tol[b, :, h * G:(h + 1) * G] = y.view(Lq, G, D), x.view(Lq, G)
    return o, tol


def within(y, o, tol, what=""):
    err = (y.double() - o).norm(dim=-1)
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / tol)[bad].max()), bad.nonzero()[0].tolist())
