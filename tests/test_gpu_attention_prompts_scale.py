"""GPU tests of attention_prompt with scores of almost any size that fp32 holds: the keys with the largest score decide."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("scale", [1e8, -1e8, 3e12, -2.0 ** 64])
@pytest.mark.parametrize("n", [1, 40, 700])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (3, 1, 64)])
def test_prompt_keys_of_the_largest_score_decide(wql, scale, n, Hq, Hkv, D):
    q = torch.zeros((n, Hq, D), dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    k = torch.zeros((n, Hkv, D), dtype=torch.float16, device="cuda")
    k[..., 0] = -(2 + torch.arange(n, device="cuda") % 8 / 8).half()[:, None]
    v = torch.randn((n, Hkv, D), generator=torch.Generator().manual_seed(n)).half().cuda()
    y = wql.attention_prompt(q, k, v, i32([0, n]), scale=scale)
    wql.device_status()
    s = k[:, 0, 0].double() * scale
    for r in {0, n // 2, n - 1}:
        best = s[:r + 1] == s[:r + 1].max()
        o = v[:r + 1][best].double().mean(0).repeat_interleave(Hq // Hkv, 0)
        size = v[:r + 1][best].double().abs().mean(0).repeat_interleave(Hq // Hkv, 0)
        assert bool(((y[r].double() - o).abs() <= 2.0 ** -10 * size + 2.0 ** -24).all())


@pytest.mark.parametrize("n", [1, 100, 300])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (4, 2, 64), (3, 1, 128)])
def test_prompt_rows_of_the_largest_numbers(wql, n, Hq, Hkv, D):
    # scores of up to 4.9e10, all the same for one half of the heads' rows, rising for the other half
    q = torch.full((n, Hq, D), 65504.0, dtype=torch.float16, device="cuda")
    k = torch.full((n, Hkv, D), 60000.0, dtype=torch.float16, device="cuda")
    v = torch.randn((n, Hkv, D), generator=torch.Generator().manual_seed(n)).half().cuda()
    y = wql.attention_prompt(q, k, v, i32([0, n]))
    wql.device_status()
    count = torch.arange(1, n + 1, device="cuda", dtype=torch.float64)[:, None, None]
    o = (v.double().cumsum(0) / count).repeat_interleave(Hq // Hkv, 1)
    size = (v.double().abs().cumsum(0) / count).repeat_interleave(Hq // Hkv, 1)
    assert bool(((y.double() - o).abs() <= 2.0 ** -10 * size + 2.0 ** -24).all())
    k = k - torch.arange(n, 0, -1, device="cuda").half()[:, None, None] * 64  # every key above the one before it
    y = wql.attention_prompt(q, k, v, i32([0, n]))
    assert torch.equal(y, v.repeat_interleave(Hq // Hkv, 1))
    y = wql.attention_prompt(-q, k, v, i32([0, n]))
    assert torch.equal(y, v[:1].repeat_interleave(Hq // Hkv, 1).expand(n, -1, -1))
    wql.device_status()


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_rows_of_huge_scores_do_not_touch_their_neighbours(wql, D):
    n, Hq, Hkv = 400, 4, 2
    g = torch.Generator().manual_seed(D)
    q, k, v = (torch.randn((n, h, D), generator=g).half().cuda() for h in (Hq, Hkv, Hkv))
    y = wql.attention_prompt(q, k, v, i32([0, n]))
    pick = torch.arange(n, device="cuda") % 29 == 3
    q2 = torch.where(pick[:, None, None], q * 20000, q).clamp(-65504, 65504)
    k2 = k.clone()
    z = wql.attention_prompt(q2, k2, v, i32([0, n]), scale=1e4)
    w = wql.attention_prompt(q, k2, v, i32([0, n]), scale=1e4)
    wql.device_status()
    assert torch.equal(z[~pick].view(torch.int16), w[~pick].view(torch.int16))
    assert torch.isfinite(z).all() and torch.isfinite(y).all()
