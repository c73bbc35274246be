"""GPU tests of attention over caches that the format allows and kv_append_i4 does not write: scales of V (and K) that are zero
or negative, written by another quantiser."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import _attn_norm as norm  # noqa: E402
import _attn_ref as ref  # noqa: E402


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


def params(cache, D):
    """(s, lo) of K and of V as views [pages, H, blocks, 16] fp16."""
    p = cache[..., 16 * D:].view(torch.float16).unflatten(-1, (2, 16, 2))
    return p[..., 0, :, 0], p[..., 0, :, 1], p[..., 1, :, 0], p[..., 1, :, 1]


SHAPES = [([3, 64, 700], 1, 8, 2, 128), ([3, 64, 700], 1, 8, 1, 64), ([5, 1500], 2, 8, 1, 128), ([6000], 1, 16, 1, 64), ([40], 5, 8, 1, 128)]


def random_cache(lens, Lq, Hq, Hkv, D, seed, s_of):
    q, cache, table, kv_lens = ref.paged_case(len(lens), lens, Lq, Hq, Hkv, D, 16, seed)
    g = torch.Generator().manual_seed(seed)
    ks, klo, vs, vlo = params(cache, D)
    r = lambda x: torch.rand(x.shape, generator=g).cuda()  # noqa: E731
    ks.copy_(r(ks) * 0.2 - 0.1)
    klo.copy_(r(klo) - 0.5)
    vs.copy_(s_of(r(vs)))
    vlo.copy_(r(vlo) * 4 - 2)
    return q, cache, table, kv_lens


@pytest.mark.parametrize("kind", ["negative", "either sign", "zero", "some zero", "minus one"])
@pytest.mark.parametrize("lens,Lq,Hq,Hkv,D", SHAPES)
def test_any_finite_scale_of_v(wql, lens, Lq, Hq, Hkv, D, kind):
    s_of = {"negative": lambda x: -0.05 - 0.2 * x, "either sign": lambda x: x - 0.5, "zero": lambda x: x * 0,
            "some zero": lambda x: torch.where(x < 0.3, 0.0, x - 0.3), "minus one": lambda x: torch.where(x < 0.5, -1.0, 1.0)}[kind]
    q, cache, table, kv_lens = random_cache(lens, Lq, Hq, Hkv, D, 4, s_of)
    y = wql.attention_kv_i4(q, cache, table, kv_lens, scale=0.5)  # scores of tens
    wql.device_status()
    o, tol = norm.kv_i4(q, cache, table, lens, scale=0.5)
    norm.within(y, o, tol, kind)


def test_a_cache_of_zeros_gives_zeros(wql):
    cache = wql.kv_cache_i4(4, 2, 128, 16)
    for G in (1, 8):
        q = torch.randn((1, 2 * G, 128), device="cuda").half()
        table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
        y = wql.attention_kv_i4(q, cache, table, torch.tensor([41], dtype=torch.int32, device="cuda"))
        assert not y.any() and torch.isfinite(y).all()
    wql.device_status()
