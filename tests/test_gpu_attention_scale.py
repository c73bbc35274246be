"""GPU tests of attention over the 4-bit cache with scales so large that scores are of almost any size that fp32 holds: the
keys with the largest score decide."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import _attn_ref as ref  # noqa: E402


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("scale", [1e8, -1e12, 2.0 ** 64, -2.0 ** 64])
@pytest.mark.parametrize("n", [1, 40, 3000])
@pytest.mark.parametrize("G,D", [(1, 128), (8, 64), (16, 128)])
@pytest.mark.parametrize("big", [1.0, 60000.0])
def test_cached_keys_of_the_largest_score_decide(wql, scale, n, G, D, big):
    # scores are -scale * (2 + key's number % 8 / 8): every 8th key has the largest, or the smallest where scale is negative
    q = torch.zeros((1, G, D), dtype=torch.float16, device="cuda")
    q[..., 0] = big
    k = torch.zeros((n, 1, D), dtype=torch.float16, device="cuda")
    k[:, 0, 0] = -(2 + torch.arange(n, device="cuda") % 8 / 8).half()
    v = torch.randn((n, 1, D), generator=torch.Generator().manual_seed(n)).half().cuda()
    ps = 16
    pages = -(-n // ps)
    cache = wql.kv_cache_i4(pages, 1, D, ps)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    wql.kv_append_i4(k, v, slots, cache)
    y = wql.attention_kv_i4(q, cache, slots[:pages].view(1, pages).contiguous(), i32([n]), scale=scale)
    wql.device_status()
    (kc, ks, klo), (vc, vs, vlo) = ref.read_parts(cache, slots)
    score = (kc * ks + klo)[:, 0, 0] * scale * big
    best = score >= score.max() - abs(float(score.max())) * 1e-3
    o = (vc * vs + vlo)[best, 0].mean(0)
    # scores that differ by less than fp32's rounding of them share the weight in any proportion: here they are equal
    assert bool((score[best] == score.max()).all())
    assert bool(((y[0].double() - o).abs() <= 2.0 ** -10 * (vc * vs + vlo)[best, 0].abs().mean(0) + 2.0 ** -11 * 4 * vs[best].max()).all())


def test_scales_beyond_the_limit_are_refused(wql):
    q = torch.zeros((2, 2, 64), dtype=torch.float16, device="cuda")
    cache = wql.kv_cache_i4(1, 2, 64, 16)
    for scale in (2.0 ** 65, -2.0 ** 65, 3e38):
        with pytest.raises(wql.WQLError, match="2\\^64"):
            wql.attention_prompt(q, q, q, i32([0, 2]), scale=scale)
        with pytest.raises(wql.WQLError, match="2\\^64"):
            wql.attention_kv_i4(q, cache, i32([[0], [0]]), i32([1, 1]), scale=scale)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("n", [1, 50, 2000])
@pytest.mark.parametrize("G,D", [(1, 128), (8, 64), (16, 128)])
def test_cached_keys_of_the_largest_numbers_at_the_largest_scale(wql, sign, n, G, D):
    # all scores are +-2^64 D 60000^2 = +-8.5e30 (D = 128): the values' mean
    q = torch.full((1, G, D), 60000.0, dtype=torch.float16, device="cuda")
    k = torch.full((n, 1, D), -60000.0, dtype=torch.float16, device="cuda")
    v = torch.randn((n, 1, D), generator=torch.Generator().manual_seed(n)).half().cuda()
    pages = -(-n // 16)
    cache = wql.kv_cache_i4(pages, 1, D, 16)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    wql.kv_append_i4(k, v, slots, cache)
    y = wql.attention_kv_i4(q, cache, slots[:pages].view(1, pages).contiguous(), i32([n]), scale=sign * 2.0 ** 64)
    wql.device_status()
    vc, vs, vlo = ref.read_parts(cache, slots)[1]
    x = (vc * vs + vlo)[:, 0]
    # each weight rounded once against code - 7.5, at most 2^-11 s 7.5, the sums in fp32, the output rounded once
    bound = 2.0 ** -11 * 7.5 * vs.max() + 2.0 ** -18 * x.abs().max() + 2.0 ** -11 * x.mean(0).abs() + 2.0 ** -25
    assert bool(((y[0].double() - x.mean(0)).abs() <= bound).all())
