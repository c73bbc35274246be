"""GPU tests of attention over packed chunks and of the attention weights that cached tokens get, against 64-bit
restatements with derived bounds."""
import math
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import _attn_ref as ref  # noqa: E402
import _chunks_ref as cref  # noqa: E402
from _gpu_util import Guarded  # noqa: E402


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def within(y, want, bound, what=""):
    """Equal up to the bound; infinities and NaN in the same places."""
    y = y.double()
    assert torch.equal(torch.isnan(y), torch.isnan(want)), (what, "NaN", int(torch.isnan(y).sum()), int(torch.isnan(want).sum()))
    far = torch.where(y == want, 0.0, (y - want).abs())
    bad = ~torch.isnan(want) & ~(far <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float(far[bad].max()), float(bound[bad].max()), bad.nonzero()[0].tolist())


def check(wql, q, cache, table, cu, lens, scale=None, what="", weights=True):
    """Both operators on one case, against the restatements; rows of no sequence and entries behind the lengths stay."""
    T, Hq, D = q.shape
    Hkv, ps, B = cache.shape[1], cache.shape[2] * 16, len(lens)
    c, n = i32(cu), i32(lens)
    out, lse = Guarded((T, Hq, D), torch.float16), Guarded((T, Hq), torch.float32)
    y = wql.attention_chunks_kv_i4(q, cache, table, c, n, scale, out=out.t, lse=lse.t)
    assert y.data_ptr() == out.t.data_ptr()
    wql.device_status()
    out.check(), lse.check()
    o, ob, z, zb = cref.chunks(q, cache, table, cu, lens, scale)
    mine = torch.zeros((T,), dtype=torch.bool, device="cuda")
    mine[cu[0]:cu[-1]] = True
    assert bool((out.t[~mine].view(torch.int16) == 0x7e00).all()) and bool((lse.t[~mine].view(torch.int32) == 0x7fc00000).all()), what
    within(out.t[mine], o[mine], ob[mine], (what, "out"))
    within(lse.t[mine], z[mine], zb[mine], (what, "lse"))
    without = wql.attention_chunks_kv_i4(q, cache, table, c, n, scale)
    assert torch.equal(without[mine].view(torch.int16), out.t[mine].view(torch.int16)), what
    if not weights:
        return
    g = torch.Generator().manual_seed(5)
    before = torch.rand((B, Hkv, table.shape[1] * ps), generator=g).cuda()
    w = Guarded(tuple(before.shape), torch.float32)
    w.t.copy_(before)
    wql.kv_weights_i4(q, cache, table, c, n, lse.t, w.t, scale)
    wql.device_status()
    w.check()
    want, wb = cref.weights(q, cache, table, cu, lens, lse.t, before, scale)
    within(w.t, want, wb, (what, "weights"))
    for b in range(B):
        at = max(lens[b], 0) if cu[b + 1] > cu[b] else 0
        assert torch.equal(w.t[b, :, at:], before[b, :, at:]), (what, b)


@pytest.mark.parametrize("n,m", [(1, 1), (2, 1), (16, 16), (17, 3), (127, 127), (128, 128), (129, 129), (128, 1), (130, 2), (255, 100),
                                 (256, 256), (257, 257), (300, 40), (513, 129), (1000, 5), (384, 384)])
@pytest.mark.parametrize("D", [64, 128])
def test_one_sequence(wql, n, m, D):
    check(wql, *cref.case([n], [m], 8, 2, D, 16, n + m, pad=2), [n])


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (5, 1), (6, 2), (7, 1), (14, 2), (4, 4), (16, 1), (32, 2), (20, 1),
                                    (64, 1), (71, 1), (65, 1), (128, 1), (127, 1), (96, 3), (33, 33)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads(wql, Hq, Hkv, D):
    lens, new = [203, 64, 9], [70, 1, 9]
    check(wql, *cref.case(lens, new, Hq, Hkv, D, 32, Hq, pad=1), lens)


@pytest.mark.parametrize("ps", [16, 48, 80, 128, 144, 256, 1024])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes(wql, ps, D):
    lens, new = [700, 129, 3], [33, 129, 1]
    check(wql, *cref.case(lens, new, 8, 2, D, ps, ps, pad=1), lens)


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 4, 4), (128, 7, 1)])
def test_mixed_batches(wql, D, Hq, Hkv):
    lens = [900, 0, 1, 300, 0, 77, 512, 5, 128, 2000, 3, 640]
    new = [1, 4, 1, 300, 0, 1, 256, 9, 0, 40, 3, 1]  # refused with rows, whole prompts, rows that see nothing, no rows
    check(wql, *cref.case(lens, new, Hq, Hkv, D, 32, 1, pad=3, lead=5), lens)


@pytest.mark.parametrize("D", [64, 128])
def test_long_contexts_are_split_and_joined(wql, D):
    for lens, new, Hq, Hkv in (([20011], [3], 8, 1), ([9000, 40, 5000], [70, 40, 1], 8, 2), ([12345], [130], 4, 4)):
        check(wql, *cref.case(lens, new, Hq, Hkv, D, 64, 7), lens, what=lens)


def test_many_sequences(wql):
    r = random.Random(3)
    lens = [r.choice([0, 1, 5, 64, 130, 333]) for _ in range(700)]
    new = [min(n, r.choice([0, 1, 1, 1, 20])) + (r.random() < 0.1) for n in lens]
    check(wql, *cref.case(lens, new, 4, 2, 64, 16, 4, pad=2), lens)


@pytest.mark.parametrize("scale", [0.0, 1e-4, -0.11, 1.0, 7.5, 1e-36])
@pytest.mark.parametrize("D", [64, 128])
def test_scales(wql, scale, D):
    # a weight's bound grows with the scores: from 7.5 on they reach hundreds
    lens, new = [400, 33], [20, 33]
    check(wql, *cref.case(lens, new, 4, 2, D, 16, 9), lens, scale=scale)


@pytest.mark.parametrize("scale", [2.0 ** 20, -(2.0 ** 64), 2.0 ** 64])
def test_scores_of_millions_choose_one_token(wql, scale):
    # scores this far apart leave one token (or those that share its score): the row of V with the greatest score
    lens, new = [300], [50]
    q, cache, table, cu = cref.case(lens, new, 2, 1, 128, 16, 10)
    y = wql.attention_chunks_kv_i4(q, cache, table, i32(cu), i32(lens), scale)
    k, v = cref.values(cache, table[0], 300, 16)
    for r in range(50):
        s = q[r].double() @ k[:251 + r, 0].T * math.copysign(1.0, scale)
        two = s.topk(2, dim=-1)
        clear = (two.values[:, 0] - two.values[:, 1]) * abs(scale) > 1e3  # far beyond what fp32 sums are off, 1e-5 of 1e8
        clear &= (two.values[:, 0] - two.values[:, 1]) > 2e-3
        want = v[two.indices[:, 0], 0]
        assert bool(((y[r].double() - want).abs() <= want.abs() * 2.0 ** -10 + 2.0 ** -24)[clear].all()), r
    wql.device_status()


def test_views_of_a_fused_projection(wql):
    lens, new = [150, 40], [60, 40]
    q, cache, table, cu = cref.case(lens, new, 6, 2, 128, 16, 11, pad=2)
    qkv = torch.randn((q.shape[0], 10, 128), device="cuda").half()
    qkv[:, :6] = q
    check(wql, qkv[:, :6], cache, table, cu, lens)
    wide = torch.zeros((2 * q.shape[0], 10, 128), device="cuda", dtype=torch.float16)
    wide[::2, :6] = q
    check(wql, wide[::2, :6], cache, table, cu, lens)
    one = qkv[:1, :6]  # one token: its stride says nothing
    check(wql, one, cache, table[:1], [0, 1], [150])


@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_are_not_numbers_reach_only_those_that_see_them(wql, D):
    lens, new = [300, 200], [100, 200]
    q, cache, table, cu = cref.case(lens, new, 4, 2, D, 16, 12)
    g = torch.Generator().manual_seed(0)
    for t, which in ((250, "k"), (270, "v"), (299, "k")):
        k, v = (torch.randn((1, 2, D), generator=g).half().cuda() for _ in range(2))
        (k if which == "k" else v)[0, 1, 3] = math.inf
        ref.write(cache, [int(table[0, t // 16]) * 16 + t % 16], k, v)
    for t in (0, 131):
        k, v = (torch.randn((1, 2, D), generator=g).half().cuda() for _ in range(2))
        v[0, 0, 3] = math.nan
        ref.write(cache, [int(table[1, t // 16]) * 16 + t % 16], k, v)
    check(wql, q, cache, table, cu, lens)
    q[3, 1, 5], q[110, 0, 0] = math.nan, math.inf  # rows of q: their own alone
    y = wql.attention_chunks_kv_i4(q, cache, table, i32(cu), i32(lens))
    assert bool(torch.isnan(y[3, 1]).all()) and not bool(torch.isnan(y[:50, [0, 2, 3]]).any())
    wql.device_status()


@pytest.mark.parametrize("D", [64, 128])
def test_values_beyond_fp16_are_the_largest(wql, D):
    # 65504 in a row from 0: s is rounded up, 15 s is 65520
    lens, new = [200], [20]
    q, cache, table, cu = cref.case(lens, new, 2, 1, D, 16, 13)
    for t in (5, 130, 195):
        v = torch.zeros((1, 1, D)).half()
        v[0, 0, 2::3] = 65504.0 if t != 130 else -65504.0
        ref.write(cache, [int(table[0, t // 16]) * 16 + t % 16], torch.randn((1, 1, D)).half().cuda(), v.cuda())
    k = torch.zeros((1, 1, D)).half()
    k[0, 0, 1::2] = 65504.0
    ref.write(cache, [int(table[0, 3]) * 16], k.cuda(), torch.ones((1, 1, D)).half().cuda())
    check(wql, q * 2.0 ** -14, cache, table, cu, lens)


@pytest.mark.parametrize("D", [64, 128])
def test_maxima_that_grow_in_every_tile(wql, D):
    # keys that grow along the context, so that weights pass every running maximum by far; and ones that fall
    for sign in (1.0, -1.0):
        n = 1500
        q, cache, table, cu = cref.case([n], [60], 4, 2, D, 16, 14)
        t = torch.arange(n)
        k = (torch.randn((n, 2, D)) * 0.2 + sign * (t / 90.0).view(n, 1, 1)).half().cuda()
        v = torch.randn((n, 2, D)).half().cuda()
        ref.write(cache, (table[0].long().cpu()[t // 16] * 16 + t % 16).cuda(), k, v)
        check(wql, q.abs(), cache, table, cu, [n])


def test_bad_sequences_lengths_and_pages_are_left_out_and_recorded(wql):
    lens, new = [100, 60, 40], [10, 5, 7]
    q, cache, table, cu = cref.case(lens, new, 4, 2, 64, 16, 15)
    o, ob, _, _ = cref.chunks(q, cache, table, cu, lens)
    w = torch.zeros((3, 2, table.shape[1] * 16), device="cuda")

    def recorded():
        with pytest.raises(wql.WQLError) as e:
            wql.device_status()
        assert e.value.status == 1

    for bad in ([0, 10, 15, 23], [-3, 10, 15, 22], [0, 23, 15, 22]):
        out = torch.full_like(q, 7.0)
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        wql.attention_chunks_kv_i4(q, cache, table, i32(bad), i32(lens), out=out, lse=lse)
        recorded()
        for b in range(3):
            a, e = bad[b], bad[b + 1]
            if 0 <= a <= e <= 22 and [a, e] == cu[b:b + 2]:
                within(out[a:e], o[a:e], ob[a:e], bad)
        left = [r for r in range(22) if not any(0 <= bad[b] <= r < bad[b + 1] <= 22 for b in range(3))]
        assert bool((out[left] == 7.0).all()) and bool((lse[left] == 7.0).all())
        wql.kv_weights_i4(q, cache, table, i32(bad), i32(lens), lse, w.clone())
        recorded()
    # a length beyond the table is cut to what it holds
    cap = table.shape[1] * 16
    full = table.clone()
    full[full < 0] = 0
    cut = wql.attention_chunks_kv_i4(q, cache, full, i32(cu), i32([cap + 1, 60, 40]))
    recorded()
    o, ob, z, zb = cref.chunks(q, cache, full, cu, [cap, 60, 40])
    within(cut, o, ob, "cut")
    # page numbers: the other sequences do not notice
    for page in (-1, cache.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[1, 2] = page
        y = wql.attention_chunks_kv_i4(q, cache, t, i32(cu), i32(lens))
        recorded()
        o, ob, z, zb = cref.chunks(q, cache, table, cu, lens)
        keep = [r for r in range(22) if not 10 <= r < 15]
        within(y[keep], o[keep], ob[keep], page)
        ww = w.clone()
        wql.kv_weights_i4(q, cache, t, i32(cu), i32(lens), torch.nan_to_num(z).float(), ww)
        recorded()
        want, wb = cref.weights(q, cache, table, cu, lens, torch.nan_to_num(z).float(), w)
        within(ww[[0, 2]], want[[0, 2]], wb[[0, 2]], page)


def test_lse_that_is_not_a_number_stays_in_its_sums(wql):
    lens, new = [100, 60], [10, 5]
    q, cache, table, cu = cref.case(lens, new, 4, 2, 64, 16, 16)
    lse = torch.zeros((15, 4), device="cuda")
    wql.attention_chunks_kv_i4(q, cache, table, i32(cu), i32(lens), lse=lse)
    lse[2, 3] = math.nan
    w = torch.zeros((2, 2, table.shape[1] * 16), device="cuda")
    wql.kv_weights_i4(q, cache, table, i32(cu), i32(lens), lse, w)
    assert bool(torch.isnan(w[0, 1, :93]).all()) and not bool(torch.isnan(w[0, 1, 93:]).any())
    assert not bool(torch.isnan(w[0, 0]).any()) and not bool(torch.isnan(w[1]).any())
    # the weights of a row add up to one
    total = w[1, :, :60].double().sum(-1)
    assert bool(((total - 10.0).abs() < 10 * 1e-5).all())
    wql.device_status()


@pytest.mark.parametrize("seed", range(12))
def test_drawn_cases(wql, seed):
    r = random.Random(seed)
    Hkv, G = r.choice([(1, 1), (2, 4), (1, 7), (3, 2), (2, 16), (4, 1), (1, 33), (8, 8)])
    D, ps = r.choice([64, 128]), r.choice([16, 32, 48, 64, 128])
    lens, new = [], []
    for _ in range(r.choice([1, 2, 5, 13])):
        n = r.choice([0, r.randrange(1, 40), r.randrange(1, 700), r.randrange(1, 3500)])
        lens.append(n)
        new.append(r.choice([0, 1, min(n, r.randrange(1, 64)), min(n, r.randrange(1, 400)), n + r.choice([0, 0, 3]) if n < 600 else 1]))
    scale = r.choice([None, None, 0.2, -0.05])
    check(wql, *cref.case(lens, new, Hkv * G, Hkv, D, ps, seed, pad=r.choice([0, 1, 9]), lead=r.choice([0, 0, 2])), lens, scale=scale,
          what=(lens, new, Hkv, G, D, ps))
