"""GPU tests of attention over chunks where sequences have a few rows: single tokens, drafted ones, groups of many heads, on
both sides of what the kernel for them takes, against the 64-bit restatements."""
import math
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import _attn_ref as ref  # noqa: E402
import _chunks_ref as cref  # noqa: E402
from test_gpu_chunks import check, i32, within  # noqa: E402


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


def attend(wql, lens, new, Hq, Hkv, D, ps, seed, **kw):
    check(wql, *cref.case(lens, new, Hq, Hkv, D, ps, seed, **kw), lens, weights=False, what=(lens, new, Hq, Hkv, D, ps))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (4, 1), (5, 1), (14, 2), (16, 2), (9, 1), (16, 1), (17, 1), (33, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_around_what_is_few(wql, D, Hq, Hkv):
    # rows of a K/V head: below, at and above 8 and 16, in batches whose mean is each of these
    lens = [300, 41, 7, 130, 1, 77]
    for new in ([1] * 6, [2] * 5 + [1], [4, 2, 4, 3, 1, 4], [8, 9, 7, 16, 1, 17], [1, 1, 1, 64, 1, 1], [3, 1, 0, 2, 1, 0]):
        attend(wql, lens, [min(n, m) for n, m in zip(lens, new)], Hq, Hkv, D, 16, Hq, pad=1, lead=2)


@pytest.mark.parametrize("new", [1, 2, 4, 8, 15, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_one_sequence(wql, D, new):
    for n in (new, 16, 17, 33, 64, 65, 500, 5000):
        if n >= new:
            attend(wql, [n], [new], 2, 2, D, 16, n)


@pytest.mark.parametrize("D,Hq,Hkv,new", [(128, 8, 2, 1), (128, 8, 2, 2), (128, 8, 2, 4), (64, 4, 4, 1), (64, 4, 4, 16), (64, 16, 1, 1)])
def test_lengths(wql, D, Hq, Hkv, new):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 95, 96, 97, 127, 128, 129, 1000]
    attend(wql, lens, [new] * len(lens), Hq, Hkv, D, 16, new)  # rows that see nothing among them


@pytest.mark.parametrize("ps", [16, 48, 80, 128, 1024])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(wql, D, ps):
    attend(wql, [1, 200, 1025, 33, 160], [1, 1, 2, 1, 2], 4, 1, D, ps, ps)
    attend(wql, [16, 200, 1025, 33, 160], [16, 3, 9, 14, 10], 2, 2, D, ps, ps)


def test_long_contexts(wql):
    attend(wql, [60007], [1], 1, 1, 128, 64, 1)
    attend(wql, [30001, 100, 9000], [2, 2, 1], 8, 2, 128, 64, 2)
    attend(wql, [40000, 5], [4, 4], 4, 1, 64, 32, 3)


def test_many_sequences(wql):
    r = random.Random(8)
    lens = [r.choice([0, 1, 5, 64, 130, 333]) for _ in range(1300)]
    attend(wql, lens, [r.choice([1, 1, 1, min(1 + n, 3)]) for n in lens], 4, 1, 64, 16, 4, pad=2)


@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_are_not_numbers_reach_only_those_that_see_them(wql, D):
    for new in ([4, 1, 2], [8, 2, 6]):
        lens = [300, 200, 50]
        q, cache, table, cu = cref.case(lens, new, 4, 2, D, 16, 12)
        g = torch.Generator().manual_seed(0)
        for b, t, which in ((0, 297, "k"), (0, 298, "v"), (1, 0, "v"), (1, 131, "v"), (2, 49, "k")):
            k, v = (torch.randn((1, 2, D), generator=g).half().cuda() for _ in range(2))
            (k if which == "k" else v)[0, t % 2, 3] = math.inf if b == 0 else math.nan
            ref.write(cache, [int(table[b, t // 16]) * 16 + t % 16], k, v)
        check(wql, q, cache, table, cu, lens, weights=False, what=new)


@pytest.mark.parametrize("D", [64, 128])
def test_values_beyond_fp16_are_the_largest(wql, D):
    # 65504 in a row from 0: s is rounded up, 15 s is 65520; and parameters just below where that is looked for
    for new in (1, 4, 8):
        lens = [200, 90]
        q, cache, table, cu = cref.case(lens, [new, new], 2, 1, D, 16, 13)
        for t, top in ((5, 65504.0), (130, -65504.0), (140, 30000.0), (150, -16380.0), (160, 60000.0)):
            v = torch.zeros((1, 1, D)).half()
            v[0, 0, 2::3] = top
            ref.write(cache, [int(table[0, t // 16]) * 16 + t % 16], torch.randn((1, 1, D)).half().cuda(), v.cuda())
        k = torch.zeros((1, 1, D)).half()
        k[0, 0, 1::2] = 65504.0
        ref.write(cache, [int(table[1, 3]) * 16], k.cuda(), torch.ones((1, 1, D)).half().cuda())
        check(wql, q * 2.0 ** -14, cache, table, cu, lens, weights=False, what=new)


@pytest.mark.parametrize("D", [64, 128])
def test_maxima_that_move(wql, D):
    # keys that grow along the context, so that weights pass every running maximum by far; and ones that fall
    for sign, new in ((1.0, 1), (-1.0, 1), (1.0, 4), (-1.0, 4)):
        n = 1500
        q, cache, table, cu = cref.case([n, n], [new, new], 4, 2, D, 16, 14)
        t = torch.arange(n)
        for b in range(2):
            k = (torch.randn((n, 2, D)) * 0.2 + sign * (t / 90.0).view(n, 1, 1)).half().cuda()
            v = torch.randn((n, 2, D)).half().cuda()
            ref.write(cache, (table[b].long().cpu()[t // 16] * 16 + t % 16).cuda(), k, v)
        check(wql, q.abs(), cache, table, cu, [n, n], weights=False)


@pytest.mark.parametrize("scale", [0.0, 1e-36, -0.11, 7.5])
@pytest.mark.parametrize("new", [1, 4])
def test_scales(wql, scale, new):
    lens = [400, 33, 90]
    check(wql, *cref.case(lens, [new] * 3, 4, 1, 128, 16, 9), lens, scale=scale, weights=False)


@pytest.mark.parametrize("scale", [2.0 ** 20, -(2.0 ** 64), 2.0 ** 64])
@pytest.mark.parametrize("new", [1, 4])
def test_scores_of_millions_choose_one_token(wql, scale, new):
    lens = [300] * 12
    q, cache, table, cu = cref.case(lens, [new] * 12, 2, 1, 128, 16, 10)
    y = wql.attention_chunks_kv_i4(q, cache, table, i32(cu), i32(lens), scale)
    chosen = 0
    for b in range(12):
        k, v = cref.values(cache, table[b], 300, 16)
        for j in range(new):
            r = b * new + j
            s = q[r].double() @ k[:301 - new + j, 0].T * math.copysign(1.0, scale)
            two = s.topk(2, dim=-1)
            gap = two.values[:, 0] - two.values[:, 1]
            clear = (gap * abs(scale) > 1e3) & (gap > 2e-3)  # far beyond what fp32 sums are off
            want = v[two.indices[:, 0], 0]
            assert bool(((y[r].double() - want).abs() <= want.abs() * 2.0 ** -10 + 2.0 ** -24)[clear].all()), r
            chosen += int(clear.sum())
    assert chosen > 12 * new
    wql.device_status()


def test_bad_pages_and_sequences_among_short_ones(wql):
    lens, new = [100, 60, 40, 70], [2, 1, 3, 1]
    q, cache, table, cu = cref.case(lens, new, 4, 2, 128, 16, 15)
    o, ob, z, zb = cref.chunks(q, cache, table, cu, lens)
    for page in (-1, cache.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[1, 2], t[2, 0] = page, page
        lse = torch.zeros((7, 4), device="cuda")
        y = wql.attention_chunks_kv_i4(q, cache, t, i32(cu), i32(lens), lse=lse)
        with pytest.raises(wql.WQLError):
            wql.device_status()
        keep = [0, 1, 6]
        within(y[keep], o[keep], ob[keep], page)
        within(lse[keep], z[keep], zb[keep], page)
    y = torch.full_like(q, 7.0)
    wql.attention_chunks_kv_i4(q, cache, table, i32([0, 2, 1, 6, 8]), i32(lens), out=y)  # the second ends early, the last too late
    with pytest.raises(wql.WQLError):
        wql.device_status()
    within(y[:1], o[:1], ob[:1])
    assert bool((y[6:] == 7.0).all())


@pytest.mark.parametrize("seed", range(16))
def test_drawn_cases(wql, seed):
    r = random.Random(100 + seed)
    Hkv, G = r.choice([(1, 1), (2, 4), (1, 7), (3, 2), (2, 16), (4, 1), (8, 8), (1, 11)])
    lens, new = [], []
    for _ in range(r.choice([1, 2, 7, 40])):
        n = r.choice([0, r.randrange(1, 40), r.randrange(1, 700), r.randrange(1, 5000)])
        lens.append(n)
        new.append(r.choice([0, 1, 1, 1, 2, 4, r.randrange(1, 20)]) if r.random() < 0.9 else min(n, 70))
    attend(wql, lens, new, Hkv * G, Hkv, r.choice([64, 128]), r.choice([16, 32, 48, 64, 128]), seed, pad=r.choice([0, 1, 9]),
           lead=r.choice([0, 0, 2]))
