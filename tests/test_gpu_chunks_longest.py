"""GPU tests of attention over chunks and of attention weights at the longest context that a table may hold, 2^31 - 16 tokens: numbers of
tokens, steps and tiles that pass 32 bits where they are added up carelessly would lose or repeat some.

Every entry of the table is page 0 and q is zero, so all tokens have the score 0, the weight 2^7 and the values of their channel:
  out  is the channel's whole number v, whatever the row sees, but for what a long sum loses.  A CTA adds up at most a 148th of the
       tokens, fewer than 2^24.  Tensor cores align products with the sum so far and cut off what lies below its last place, 2^-23 of the
       power of two that it has reached.  A product 2^7 v whose v is a power of two is never cut before 2^24 tokens; another loses what
       lost() adds up: its remainder modulo that last place, for the tokens that the sum takes while it is that large.
       The other sums' roundings, 2^-24 each, are far below fp16's half step, which then makes whole numbers exact
  lse  is ln(tokens seen), off by the roundings of joining 152 parts (2^-23 each at most) and 2^-21 of itself: 3e-5
  weights add exp(-lse) per row and head, off by 2^-19 of themselves; lse is taken as it is
"""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def lost(v, tokens):
    """The part of the sum of `tokens` products 2^7 v that is cut off at most."""
    t, total = 128 * v, 128 * v * tokens
    cut = 0.0
    for e in range(24, 64):
        cut += max(0, min(2 ** (e + 1), total) - 2 ** e) / max(t, 1) * (t % 2 ** (e - 23))
    return cut / max(total, 1)


# one row, a few (kernel for a few rows), a tile that both halves of a CTA share, two tiles
@pytest.mark.parametrize("rows,Hq", [(1, 2), (4, 2), (40, 2), (100, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_longest_context(wql, D, rows, Hq):
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    ps, width = 16, 2 ** 27 - 1
    n = ps * width
    cache = wql.kv_cache_i4(1, 1, D, ps)
    whole = (torch.arange(D) % 16).half().view(1, 1, D).expand(16, 1, D).contiguous().cuda()
    ref.write(cache, torch.arange(16, device="cuda"), torch.randn((16, 1, D)).half().cuda(), whole)
    table = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    q = torch.zeros((rows, Hq, D), dtype=torch.float16, device="cuda")
    lse = torch.zeros((rows, Hq), device="cuda")
    y = wql.attention_chunks_kv_i4(q, cache, table, i32([0, rows]), i32([n]), lse=lse)
    wql.device_status()
    want = whole[0, 0].double()
    off = torch.tensor([lost(int(v), n // 148 + 128) for v in want.tolist()], dtype=torch.float64, device="cuda")
    assert [int(v) for v, x in zip(want.tolist()[:16], off.tolist()) if x == 0] == [0, 1, 2, 4, 8]
    assert bool((y.double() <= want).all()) and bool((y.double() >= want * (1 - off) * torch.where(off > 0, 1 - 2.0 ** -11, 1.0)).all())
    seen = n - rows + 1 + torch.arange(rows, dtype=torch.float64, device="cuda")
    assert float((lse.double() - seen.log()[:, None]).abs().max()) < 3e-5
    weights = torch.zeros((1, 1, n), device="cuda")
    wql.kv_weights_i4(q, cache, table, i32([0, rows]), i32([n]), lse, weights)
    wql.device_status()
    each = torch.exp(-lse.double()).sum(1)  # of a row
    all_see = n - rows + 1
    first, least, most = float(each.sum()), math.inf, 0.0
    for a in range(0, all_see, 1 << 28):
        part = weights[0, 0, a:min(a + (1 << 28), all_see)]
        least, most = min(least, float(part.min())), max(most, float(part.max()))
    assert abs(least / first - 1) < 2.0 ** -19 and abs(most / first - 1) < 2.0 ** -19
    last = each.flip(0).cumsum(0).flip(0)  # token all_see - 1 + r is seen by the rows from r on
    assert float((weights[0, 0, all_see - 1:].double() / last - 1).abs().max()) < 2.0 ** -19
