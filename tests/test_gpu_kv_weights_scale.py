"""GPU tests of attention weights of large scores: a weight is the exponential of a small difference of large numbers, which has to be
formed without rounding them first.

Scores here are exact in fp32: codes 0 .. 15 with s = 1 and lo = 0, whole numbers of up to 2^11 in q, sums below 2^24.  So of
exp(scale q . k - lse), t = scale q . k - lse, what is left to be off is
  t itself, rounded once, times log2 e, which is rounded to fp32, and that product: 2^-24 |t| + 2^-24 |t| + 2^-24 |t|
  the base-2 exponential: 2^-21 of itself (its documented bound is 2 units in the last place)
  sums: 2^-23 of the sum per addition
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import _attn_ref as ref  # noqa: E402


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


def exact_scores(n, rows, Hq, Hkv, D, big, seed):
    """(q, cache, table, q . k as [Hq, rows, n] float64): half of the channels carry a constant of about `big` D times 7.5, the
    others differences of some units."""
    g = torch.Generator().manual_seed(seed)
    _, cache, table, _ = ref.paged_case(1, [n], 1, Hkv, Hkv, D, 16, seed)
    k = torch.randint(0, 16, (n, Hkv, D), generator=g).float()
    k[..., ::2] = 15.0
    k[..., 1] = 0.0
    q = torch.randint(-1, 2, (rows, Hq, D), generator=g).float()
    q[..., ::2] = big
    t = torch.arange(n)
    ref.write(cache, (table[0].long().cpu()[t // 16] * 16 + t % 16).cuda(), k.half().cuda(), torch.ones_like(k).half().cuda())
    s = torch.einsum("rhd,thd->hrt", q.double(), k.double().repeat_interleave(Hq // Hkv, 1))
    assert float(s.abs().max()) < 2 ** 24
    return q.half().cuda(), cache, table, s.cuda()


# few rows and many: one and two groups of warps that add up
@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 4, 4)])
@pytest.mark.parametrize("big,scale", [(0.0, 0.1), (16.0, 0.37), (256.0, -0.37), (1024.0, 0.37), (1024.0, 0.011), (1024.0, 37.0)])
def test_weights_of_large_scores(wql, big, scale, D, Hq, Hkv, rows):
    n, G = 300, Hq // Hkv
    q, cache, table, s = exact_scores(n, rows, Hq, Hkv, D, big, 3)
    scale = float(torch.tensor(scale, dtype=torch.float32))  # as the kernel takes it
    see = torch.arange(n, device="cuda")[None] <= (n - rows + torch.arange(rows, device="cuda"))[:, None]
    s = torch.where(see, s * scale, -torch.inf)
    lse = torch.logsumexp(s, -1).T.float().contiguous()  # [rows, Hq], rounded: what is added up is the formula's of these
    t = s - lse.T[..., None].double()
    p = torch.exp(t)
    off = torch.where(p > 0, p * (3 * 2.0 ** -24 * t.abs() + 2.0 ** -21) * 1.01, 0.0)
    want, bound = (x.view(Hkv, G * rows, n).sum(1) for x in (p, off))
    bound = bound + (G * rows + 2) * 2.0 ** -23 * want + 1e-30
    w = torch.zeros((1, Hkv, table.shape[1] * 16), device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    wql.kv_weights_i4(q, cache, table, i32([0, rows]), i32([n]), lse, w, scale)
    wql.device_status()
    far = (w[0, :, :n].double() - want).abs()
    assert bool((far <= bound).all()), (float((far / want.clamp(min=1e-3)).max()), float((far - bound).max()))
    # a row's weights add up to what its lse, rounded once, says; to one if it were not rounded
    assert float((want.sum(-1) / (G * rows)).log().abs().max()) <= float(lse.abs().max()) * 2.0 ** -24 + 1e-9
