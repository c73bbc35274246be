"""GPU tests of attention over the paged 4-bit cache where rows of V are constant, against the 64-bit restatement and the
error vectors' criterion of tests/_attn_norm.py."""
import math

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


def case(lens, Lq, Hq, Hkv, D, ps, seed, values):
    """A cache whose V rows [n, Hkv, D] are values(generator, n)."""
    q, cache, table, kv_lens = ref.paged_case(len(lens), lens, Lq, Hq, Hkv, D, ps, seed)
    g = torch.Generator().manual_seed(seed + 1)
    for b, n in enumerate(lens):
        t = torch.arange(n)
        slots = (table[b].cpu().long()[t // ps] * ps + t % ps).cuda()
        keys = (torch.randn((n, Hkv, D), generator=g) * 0.7).half().cuda()
        ref.write(cache, slots, keys, values(g, n).half().cuda())
    return q, cache, table, kv_lens


# lens, Lq, Hq, Hkv, D: 1, 4, 5, 7, 8, 16 and 20 rows per K/V head; short, in one CTA, over several
SHAPES = [([1], 1, 1, 1, 128), ([3, 64], 1, 8, 2, 128), ([3, 64, 700], 1, 10, 2, 128), ([3, 64, 700], 1, 7, 1, 64),
          ([3, 64, 33], 1, 16, 2, 128), ([1, 3, 64], 2, 16, 2, 64), ([64, 1500, 5], 4, 8, 2, 128), ([40, 700], 5, 8, 2, 64),
          ([6000], 1, 8, 1, 128), ([6000], 1, 16, 1, 64)]


@pytest.mark.parametrize("lens,Lq,Hq,Hkv,D", SHAPES)
def test_rows_of_zeros_give_zeros(wql, lens, Lq, Hq, Hkv, D):
    q, cache, table, kv_lens = case(lens, Lq, Hq, Hkv, D, 16, 3, lambda g, n: torch.zeros((n, Hkv, D)))
    y = wql.attention_kv_i4(q, cache, table, kv_lens)
    wql.device_status()
    assert not y.any(), float(y.abs().max())


@pytest.mark.parametrize("size", [0.02, 0.05, 40.0])
@pytest.mark.parametrize("lens,Lq,Hq,Hkv,D", SHAPES)
def test_constant_rows_among_others(wql, lens, Lq, Hq, Hkv, D, size):
    def values(g, n):
        v = torch.randn((n, Hkv, D), generator=g) * size
        const = torch.rand((n, Hkv, 1), generator=g) < 0.1
        const[n // 2] = True
        level = torch.randn((n, Hkv, 1), generator=g) * size * (torch.rand((n, Hkv, 1), generator=g) < 0.5)
        return torch.where(const, level.expand(-1, -1, D), v)

    q, cache, table, kv_lens = case(lens, Lq, Hq, Hkv, D, 16, 5, values)
    y = wql.attention_kv_i4(q, cache, table, kv_lens)
    wql.device_status()
    o, tol = norm.kv_i4(q, cache, table, lens)
    norm.within(y, o, tol, size)


@pytest.mark.parametrize("size", [1e-3, 1.0, 3000.0])
@pytest.mark.parametrize("lens,Lq,Hq,Hkv,D", SHAPES)
def test_only_constant_rows(wql, lens, Lq, Hq, Hkv, D, size):
    q, cache, table, kv_lens = case(lens, Lq, Hq, Hkv, D, 16, 7,
                                    lambda g, n: (torch.randn((n, Hkv, 1), generator=g) * size).expand(-1, -1, D))
    y = wql.attention_kv_i4(q, cache, table, kv_lens)
    wql.device_status()
    o, tol = norm.kv_i4(q, cache, table, lens)
    norm.within(y, o, tol, size)


def test_a_scale_of_one_with_codes_stays_what_it_is(wql):
    # rows from 0 to 15 have s = 1, as constant ones do, and codes that count
    D, n, Hkv = 128, 500, 2
    lens = [n]
    q, cache, table, kv_lens = case(lens, 1, 16, Hkv, D, 16, 9, lambda g, n: torch.randint(0, 16, (n, Hkv, D), generator=g).float()
                                    .index_fill_(2, torch.tensor([0]), 0.0).index_fill_(2, torch.tensor([D - 1]), 15.0))
    t = torch.arange(n, device="cuda")
    parts = ref.read_parts(cache, table[0].long()[t // 16] * 16 + t % 16)
    assert bool((parts[1][1] == 1.0).all())
    y = wql.attention_kv_i4(q, cache, table, kv_lens)
    o, tol = norm.kv_i4(q, cache, table, lens)
    norm.within(y, o, tol)
    # one code alone, in any place of the row
    v = torch.zeros((D, Hkv, D))
    for c in range(D):
        v[c, :, c] = 15.0
    q, cache, table, kv_lens = case([D], 1, 16, Hkv, D, 16, 10, lambda g, n: v[:n])
    y = wql.attention_kv_i4(q, cache, table, kv_lens)
    o, tol = norm.kv_i4(q, cache, table, [D])
    norm.within(y, o, tol)
    wql.device_status()
