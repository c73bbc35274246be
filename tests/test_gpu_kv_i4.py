"""GPU tests of the paged 4-bit KV cache: page planning, quantise-and-append, read back -- bit-exact against the
64-bit restatement -- and their run together."""
import math

import numpy as np
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


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


# ---- plan ------------------------------------------------------------------------------------

def _plan_case(B, ps, max_ctx, max_new, seed, spare, width_cut=0):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, max_ctx + 1, B)
    new = rng.integers(0, max_new + 1, B)
    width = max(1, -(-(max_ctx + max_new) // ps) - width_cut)
    ctx = np.minimum(ctx, width * ps)
    held = -(-ctx // ps)
    need = int((-(-(ctx + new) // ps) - held).sum())
    pages = int(held.sum()) + max(0, need + spare)
    perm = rng.permutation(pages + 2)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = perm[at:at + max(0, need + spare)]
    return ctx, new, table, free


@pytest.mark.parametrize("B,ps,max_ctx,max_new,spare,width_cut", [
    (1, 16, 0, 1, 0, 0), (1, 16, 40, 1, 3, 0), (8, 16, 4096, 1, 5, 0), (33, 64, 500, 300, 0, 0), (257, 48, 100, 40, 9, 0),
    (300, 16, 64, 200, -50, 0),   # the free list runs out
    (64, 32, 900, 300, 4, 12),    # some tables are too short
    (100, 16, 300, 200, -40, 5),  # both
    (4096, 128, 50, 3, 1, 0), (3, 16, 16, 5000, 0, 0)])
def test_plan(wql, B, ps, max_ctx, max_new, spare, width_cut):
    ctx, new, table, free = _plan_case(B, ps, max_ctx, max_new, B + ps, spare, width_cut)
    for extra in (0, 7):
        T = int(new.sum()) + extra
        r_slots, r_cu, r_len, r_left, r_table = ref.plan(ctx, new, table, free, len(free), ps, T)
        t = i32(table)
        f = i32(free) if len(free) else torch.empty((0,), dtype=torch.int32, device="cuda")
        for _ in range(2):  # the second call finds the table written
            slots, cu, lens, left = wql.kv_plan_pages(i32(ctx), i32(new), t, f, i32([len(free)]), ps, T)
            assert np.array_equal(cu.cpu().numpy(), r_cu)
            assert np.array_equal(lens.cpu().numpy(), r_len)
            assert int(left) == r_left
            assert np.array_equal(t.cpu().numpy(), r_table)
            assert np.array_equal(slots.cpu().numpy(), r_slots)
    wql.device_status()


def test_plan_fewer_slots_than_tokens_and_empty(wql):
    ctx, new, table, free = _plan_case(20, 16, 50, 60, 3, 0)
    T = int(new.sum()) - 33
    r = ref.plan(ctx, new, table, free, len(free), 16, T)
    slots, cu, lens, left = wql.kv_plan_pages(i32(ctx), i32(new), i32(table), i32(free), i32([len(free)]), 16, T)
    assert np.array_equal(slots.cpu().numpy(), r[0]) and np.array_equal(cu.cpu().numpy(), r[1])
    e = torch.empty((0,), dtype=torch.int32, device="cuda")
    slots, cu, lens, left = wql.kv_plan_pages(e, e, torch.empty((0, 4), dtype=torch.int32, device="cuda"), i32(free),
                                              i32([len(free)]), 16, 5)
    assert slots.tolist() == [-1] * 5 and cu.tolist() == [0] and int(left) == len(free)
    # lengths below zero count as zero, a free count above the list's size as its size
    slots, cu, lens, left = wql.kv_plan_pages(i32([-5, 3]), i32([2, -1]), i32([[-1, -1], [7, -1]]), i32([4, 9]),
                                              i32([50]), 16, 3)
    assert slots.tolist() == [9 * 16, 9 * 16 + 1, -1] and lens.tolist() == [2, 3] and int(left) == 1


def test_plan_pages_beyond_every_slot(wql):
    # 16 * 2^30 = 0 in 32 bits: such a page must not stand for page 0
    table = i32([[2 ** 30], [2 ** 27 - 1], [-3], [-1]])
    slots, cu, lens, left = wql.kv_plan_pages(i32([4, 15, 2, 0]), i32([1, 1, 1, 2]), table, i32([2 ** 31 - 1]), i32([1]), 16, 6)
    assert slots.tolist() == [-1, 2 ** 31 - 1, -1, -1, -1, -1]
    assert cu.tolist() == [0, 1, 2, 3, 5] and lens.tolist() == [5, 16, 3, 2] and int(left) == 0
    assert int(table[3, 0]) == 2 ** 31 - 1
    wql.device_status()


# ---- append and read ---------------------------------------------------------------------------

def _kv(T, H, D, seed, fused):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((2, T, H, D), generator=g) * 10.0 ** (4 * torch.rand((2, T, 1, 1), generator=g) - 2)
    x[:, :, :, : D // 32] *= 8
    x = x.clamp(-65000, 65000).half().cuda()
    if not fused:
        return x[0].contiguous(), x[1].contiguous()
    qkv = torch.zeros((T, 5 * H, D), dtype=torch.float16, device="cuda")
    qkv[:, 3 * H:4 * H], qkv[:, 4 * H:] = x[0], x[1]
    return qkv[:, 3 * H:4 * H], qkv[:, 4 * H:]


@pytest.mark.parametrize("T,H,D,ps,fused", [(1, 1, 128, 16, False), (1, 1, 64, 16, True), (7, 3, 128, 48, True),
                                           (16, 8, 128, 16, True), (129, 2, 64, 32, False), (1000, 4, 128, 64, True),
                                           (2050, 8, 64, 128, True)])
def test_append_and_read_bit_exact(wql, T, H, D, ps, fused):
    k, v = _kv(T, H, D, T + H, fused)
    g = torch.Generator().manual_seed(T)
    pages = -(-T // ps) + 4
    slots = torch.randperm(pages * ps, generator=g)[:T].to(torch.int32).cuda()
    if T > 4:
        slots[T // 2] = -1
        slots[T - 1] = -9
    cache = torch.randint(0, 256, (pages, H, ps // 16, 16 * (D + 8)), generator=g, dtype=torch.uint8).cuda()
    want = cache.clone()
    ref.write(want, slots, k, v)
    assert wql.kv_append_i4(k, v, slots, cache) is cache
    assert torch.equal(cache, want)  # and nothing else was touched
    kk, vv = wql.kv_read_i4(cache, slots)
    keep = slots >= 0
    rk, rv = ref.read(cache, slots[keep])
    assert same_bits(kk[keep], rk) and same_bits(vv[keep], rv)
    assert not kk[~keep].any() and not vv[~keep].any()
    twice = torch.cat([slots, slots.flip(0)])  # reading a slot more than once
    k2, _ = wql.kv_read_i4(cache, twice)
    assert same_bits(k2[:T], kk) and same_bits(k2[T:].flip(0), kk)
    wql.device_status()


@pytest.mark.parametrize("T,H,D", [(8191, 9, 64), (8191, 9, 128), (4001, 40, 64), (5, 700, 128), (17, 400, 64)])
def test_append_many_rows_bit_exact(wql, T, H, D):
    # both numbers of tokens that a warp may take, with a ragged end
    k, v = _kv(T, H, D, T, True)
    pages = -(-T // 32) + 1
    slots = torch.randperm(pages * 32, generator=torch.Generator().manual_seed(H))[:T].to(torch.int32).cuda()
    slots[T // 3] = -1
    cache, want = wql.kv_cache_i4(pages, H, D, 32), wql.kv_cache_i4(pages, H, D, 32)
    ref.write(want, slots, k, v)
    wql.kv_append_i4(k, v, slots, cache)
    assert torch.equal(cache, want)
    wql.device_status()


def test_append_ties_constant_rows_and_non_finite(wql):
    D, T = 128, 9
    x = torch.zeros((T, 1, D), dtype=torch.float64)
    c = torch.arange(D) % 31
    x[0, 0] = (c * 0.5).clamp(max=15)             # s = 1: every second value an exact tie between two codes
    x[1, 0] = -3.0 + (c * 0.5).clamp(max=15) / 8  # the same around -3, s = 1/8
    x[2, 0] = 1234.0                              # a constant row: s = 1, codes 0
    x[3, 0] = 2.0 ** -24 * (c % 23)               # fp16 subnormals
    x[4, 0, ::2], x[4, 0, 1::2] = 65504, -65504   # the widest row
    x[5, 0] = c * 2.0 ** -24
    x[5, 0, 0] = 60000                            # a difference that fp32 cannot hold
    x[6, 0, 5] = math.inf
    x[7, 0, 9] = math.nan
    x[8, 0] = -0.0
    # scales that lie in the middle between two fp16 numbers: (max - lo) / 15 = (2 m + 1) 2^-11 for 2^10 <= 2m+1 < 2^11...
    x = x.half()
    more = []
    for odd in (2049, 2051, 2053, 4095):
        r = torch.zeros((D,), dtype=torch.float64)
        r[1] = 15.0 * odd * 2.0 ** -12  # needs up to 16 bits: keep those that fp16 pairs can span
        hi = torch.tensor(float(r[1])).half()
        r[1], r[2] = float(hi), float(hi) - 15.0 * odd * 2.0 ** -12
        more.append(r.half()[None])
    x = torch.cat([x, torch.stack(more)]).cuda()
    T = x.shape[0]
    cache = torch.zeros((1, 1, 1, 16 * (D + 8)), dtype=torch.uint8, device="cuda")
    want = cache.clone()
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    y = x.flip(0).contiguous()
    ref.write(want, slots, x, y)
    wql.kv_append_i4(x, y, slots, cache)
    kk, vv = wql.kv_read_i4(cache, slots)
    nan = torch.zeros((T,), dtype=torch.bool, device="cuda")
    nan[6:8] = True
    assert torch.isnan(kk[nan]).all() and torch.isnan(vv[nan.flip(0)]).all()
    # NaN params may differ in their payload: compare the finite rows' bytes
    rk, rv = ref.read(want, slots)
    assert same_bits(kk[~nan], rk[~nan]) and same_bits(vv[~nan.flip(0)], rv[~nan.flip(0)])
    a, b = ref.read_parts(cache, slots), ref.read_parts(want, slots)
    for (c0, s0, l0), (c1, s1, l1), ok in ((a[0], b[0], ~nan), (a[1], b[1], ~nan.flip(0))):
        assert torch.equal(c0[ok], c1[ok]) and torch.equal(s0[ok], s1[ok]) and torch.equal(l0[ok], l1[ok])
    wql.device_status()


@pytest.mark.parametrize("D", [64, 128])
def test_append_many_random_fp16_patterns_bit_exact(wql, D):
    # every fp16 exponent, few mantissa bits: scales and quotients meet ties far more often than real rows do
    g = torch.Generator().manual_seed(D)
    T, H, ps = 8192, 4, 64
    e = torch.randint(-12, 12, (T, H, 1), generator=g) + torch.randint(-4, 1, (T, H, D), generator=g)
    x = (torch.randint(-16, 17, (T, H, D), generator=g) * torch.exp2(e.double())).half().cuda()
    y = (torch.randint(-2000, 2001, (T, H, D), generator=g) * torch.exp2(e.double() - 6)).half().cuda()
    cache = wql.kv_cache_i4(T // ps, H, D, ps)
    want = cache.clone()
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    ref.write(want, slots, x, y)
    wql.kv_append_i4(x, y, slots, cache)
    assert torch.equal(cache, want)


def test_slots_out_of_range_are_left_out_and_recorded(wql):
    k, v = _kv(4, 2, 64, 1, False)
    cache = wql.kv_cache_i4(2, 2, 64, 16)
    want = cache.clone()
    slots = i32([0, 32, 31, 2 ** 31 - 1])
    ref.write(want, [0, -1, 31, -1], k, v)
    wql.kv_append_i4(k, v, slots, cache)
    with pytest.raises(wql.WQLError) as e:
        wql.device_status()
    assert e.value.status == 1 and "out of range" in str(e.value)
    wql.device_status()  # reported once
    assert torch.equal(cache, want)
    kk, vv = wql.kv_read_i4(cache, slots)
    with pytest.raises(wql.WQLError):
        wql.device_status()
    assert not kk[1].any() and not vv[3].any() and same_bits(kk[0], ref.read(cache, [0])[0][0])


def test_cache_offsets_beyond_32_bits(wql):
    # a pool of 2.3 GB: the last page lies past 2^31 bytes
    D, H, ps = 128, 8, 64
    pages = 2300000000 // (H * ps * (D + 8))
    cache = torch.empty((pages, H, ps // 16, 16 * (D + 8)), dtype=torch.uint8, device="cuda")
    k, v = _kv(3, H, D, 5, False)
    slots = i32([pages * ps - 1, 5, (pages - 1) * ps])
    wql.kv_append_i4(k, v, slots, cache)
    kk, vv = wql.kv_read_i4(cache, slots)
    small = wql.kv_cache_i4(1, H, D, 16)
    wql.kv_append_i4(k, v, i32([0, 1, 2]), small)
    sk, sv = wql.kv_read_i4(small, i32([0, 1, 2]))
    assert same_bits(kk, sk) and same_bits(vv, sv)
    q = torch.randn((2, 1, H, D), device="cuda").half()
    table = i32([[pages - 1], [0]])
    big = wql.attention_kv_i4(q, cache, table, i32([1, 0]))
    wql.kv_append_i4(k[2:], v[2:], i32([0]), small)
    little = wql.attention_kv_i4(q, small, i32([[0], [0]]), i32([1, 0]))
    assert same_bits(big, little)
    wql.device_status()
