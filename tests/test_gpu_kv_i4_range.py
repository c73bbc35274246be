"""GPU tests of the 4-bit cache at the end of fp16's range: a finite row whose largest value lies between fp16's largest
number and infinity once its scale is rounded."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import _attn_ref as ref  # noqa: E402


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


@pytest.mark.parametrize("D", [64, 128])
def test_finite_rows_beyond_fp16_read_as_infinity_and_attend_as_they_are(wql, D):
    x = torch.zeros((5, 1, D), dtype=torch.float64)
    x[0, 0, 1::2] = 65504            # s = 4368: 65520
    x[1, 0, 1::2] = -65504           # 15 s + lo = 16: the other end has no such row
    x[2, 0, ::2], x[2, 0, 1::2] = -65504, 65504
    x[3, 0, 1::2] = 60000            # s = 4000
    x = x.half().cuda()
    cache = wql.kv_cache_i4(1, 1, D, 16)
    slots = torch.arange(5, dtype=torch.int32, device="cuda")
    wql.kv_append_i4(torch.zeros_like(x), x, slots, cache)
    want = torch.zeros_like(cache)
    ref.write(want, slots, torch.zeros_like(x), x)
    assert torch.equal(cache, want)
    _, v = wql.kv_read_i4(cache, slots)
    assert torch.equal(v.view(torch.int16), ref.read(cache, slots)[1].view(torch.int16))
    top = v[:, 0, 1::2].double()
    assert bool((top[0] == math.inf).all()) and bool((top[1] == -65504).all()) and bool((top[2] == math.inf).all())
    assert bool((top[3] == 60000).all()) and not v[:4, 0, ::2][[0, 3]].any()
    # equal weights: a fifth of 65520 + 0 - 65504 + 65536 + 60000 is no infinity, for few rows and for many
    for G in (1, 8, 16):
        y = wql.attention_kv_i4(torch.zeros((1, G, D), dtype=torch.float16, device="cuda"), cache,
                                torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                                torch.tensor([5], dtype=torch.int32, device="cuda"))
        o, bound = ref.kv_i4(torch.zeros((1, 1, G, D), dtype=torch.float16, device="cuda"), cache,
                             torch.zeros((1, 1), dtype=torch.int32, device="cuda"), [5])
        assert torch.isfinite(y).all() and bool(((y[:, None].double() - o).abs() <= bound).all())
    wql.device_status()
