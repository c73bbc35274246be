"""GPU tests of attention over chunks of many rows whose scores are so large that one token gets all the weight."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import _chunks_ref as cref  # noqa: E402


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


@pytest.mark.parametrize("scale", [2.0 ** 12, 2.0 ** 20, -(2.0 ** 40), 2.0 ** 64])
@pytest.mark.parametrize("D,Hq,Hkv,n,new", [(128, 2, 1, 300, 50), (64, 4, 4, 700, 60), (128, 8, 2, 2000, 100)])
def test_most_rows_choose_one_token(wql, D, Hq, Hkv, n, new, scale):
    # A row counts where its greatest score, as fp32 may see it, is 1000 beyond the next: both are off by (D + 8) 2^-23 of the sum of
    # magnitudes at most, and exp(-1000) is zero.  Most rows have to be of that kind.
    q, cache, table, cu = cref.case([n], [new], Hq, Hkv, D, 16, 10)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lse = torch.zeros((new, Hq), device="cuda")
    y = wql.attention_chunks_kv_i4(q, cache, table, i32(cu), i32([n]), scale, lse=lse)
    wql.device_status()
    k, v = cref.values(cache, table[0], n, 16)
    chosen = 0
    for h in range(Hq):
        kh, vh, qh = k[:, h * Hkv // Hq], v[:, h * Hkv // Hq], q[:, h].double()
        see = torch.arange(n, device="cuda")[None] <= torch.arange(n - new, n, device="cuda")[:, None]
        s = torch.where(see, qh @ kh.T * math.copysign(1.0, scale), -math.inf)
        off = (qh.abs() @ kh.abs().T).amax(-1) * (D + 8) * 2.0 ** -23
        two = s.topk(2, dim=-1)
        clear = (two.values[:, 0] - two.values[:, 1] - 2 * off) * abs(scale) > 1000
        want = vh[two.indices[:, 0]]
        # the token's own weight is rounded once, and the output: 2^-11 each, with room for fp32 sums and the division
        assert bool(((y[:, h].double() - want).abs() <= want.abs() * (2.0 ** -10 + 2.0 ** -18) + 2.0 ** -24)[clear].all()), h
        # its score is the log-sum: off by as much, and by 2^-22 of itself for the maximum, the logarithm and ln 2
        top = two.values[:, 0] * abs(scale)
        assert bool(((lse[:, h].double() - top).abs() <= off * abs(scale) + 2.0 ** -21 * top.abs() + 2.0 ** -20)[clear].all()), h
        chosen += int(clear.sum())
    assert chosen > 0.8 * new * Hq, chosen
