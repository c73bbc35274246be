"""GPU tests of leaving the least attended tokens of the 4-bit cache behind, against a restatement token by token, and of
the whole run from page planning to decode steps over the smaller cache."""
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


def make(lens, H, D, ps, budget, seed, extra=0, distinct=None):
    """Cache of random bytes with the sequences' pages and as many new ones; weights with ties, zeros of both signs."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // ps) for n in lens]
    new = [-(-min(n, budget) // ps) for n in lens]
    width, new_width = max(1, max(held)) + 1, -(-budget // ps) + extra
    pages = sum(held) + sum(new) + 2
    perm = torch.randperm(pages, generator=g)
    table, new_table = torch.full((len(lens), width), -5, dtype=torch.int32), torch.full((len(lens), new_width), -5, dtype=torch.int32)
    at = 0
    for t, counts in ((table, held), (new_table, new)):
        for b, m in enumerate(counts):
            t[b, :m] = perm[at:at + m]
            at += m
    cache = torch.randint(0, 256, (pages, H, ps // 16, 16 * (D + 8)), generator=g, dtype=torch.uint8)
    w = torch.randn((len(lens), H, width * ps), generator=g)
    if distinct is not None:
        w = torch.randint(0, distinct, w.shape, generator=g).float() * 0.5 - 0.5
        w[torch.rand(w.shape, generator=g) < 0.1] = -0.0
    return cache.cuda(), table.cuda(), new_table.cuda(), w.cuda()


def rows(cache, slots, H, D):
    """Codes and parameters [tokens, H, D + 8] bytes at slots [tokens, H], each head's own."""
    h, ps = D // 2, cache.shape[2] * 16
    page, blk, row = slots // ps, slots % ps // 16, slots % 16
    heads = torch.arange(H, device=cache.device)[None]
    parts = ((0, h), (16 * h, h), (32 * h, 4), (32 * h + 64, 4))
    return torch.cat([cache[..., a:a + 16 * n].unflatten(-1, (16, n))[page, heads, blk, row] for a, n in parts], -1)


def check(wql, lens, H, D, ps, budget, recent, seed, extra=0, distinct=None, weights=None, what=""):
    cache, table, new_table, w = make(lens, H, D, ps, budget, seed, extra, distinct)
    if weights is not None:
        w = weights(w)
    B, before = len(lens), cache.clone()
    kept, nw, nl = Guarded((B, H, budget), torch.int32), Guarded((B, H, new_table.shape[1] * ps), torch.float32), Guarded((B,), torch.int32)
    got = wql.kv_evict_i4(w, cache, table, i32(lens), new_table, budget, recent, kept.t, nw.t, nl.t)
    wql.device_status()
    kept.check(), nw.check(), nl.check()
    assert [x.data_ptr() for x in got] == [kept.t.data_ptr(), nw.t.data_ptr(), nl.t.data_ptr()]
    want = cref.evict(w.cpu(), lens, budget, recent)
    assert nl.t.tolist() == [min(n, budget) for n in lens], what
    k = kept.t.cpu()
    for b, n in enumerate(lens):
        m = min(n, budget)
        for h in range(H):
            assert k[b, h, :m].tolist() == want[b][h], (what, b, h)
        assert bool((k[b, :, m:] == -1).all())
        src = torch.tensor(want[b], device="cuda").long().T.reshape(m, H)  # [m, H]
        assert torch.equal(nw.t[b, :, :m].view(torch.int32), w[b].gather(1, src.T).view(torch.int32)), (what, b)
        assert not bool(nw.t[b, :, m:].any())
        i = torch.arange(m, device="cuda")
        to = (new_table[b].long()[i // ps] * ps + i % ps)[:, None].expand(m, H)
        assert torch.equal(rows(cache, to, H, D), rows(before, table[b].long()[src // ps] * ps + src % ps, H, D)), (what, b)
        # everything else is as it was
        expect = rows(before, table[b].long()[src // ps] * ps + src % ps, H, D)
        hh = D // 2
        at = 0
        for a, size in ((0, hh), (16 * hh, hh), (32 * hh, 4), (32 * hh + 64, 4)):
            before[..., a:a + 16 * size].unflatten(-1, (16, size))[to // ps, torch.arange(H, device="cuda")[None], to % ps // 16, to % 16] = \
                expect[..., at:at + size]
            at += size
    assert torch.equal(cache, before), what


@pytest.mark.parametrize("n,budget,recent", [(1, 1, 0), (1, 5, 2), (2, 1, 0), (2, 1, 1), (16, 16, 4), (17, 16, 16), (33, 16, 40),
                                             (1000, 1, 0), (1000, 999, 0), (1000, 999, 998), (1025, 512, 100), (1024, 1000, 0),
                                             (2049, 1024, 7), (5000, 4097, 4096), (5000, 33, 1), (4096, 4096, 0), (4097, 2048, 2048)])
@pytest.mark.parametrize("D", [64, 128])
def test_one_sequence(wql, n, budget, recent, D):
    check(wql, [n], 3, D, 16, budget, recent, n + budget)


@pytest.mark.parametrize("ps", [16, 48, 128, 1024])
def test_batches(wql, ps):
    lens = [700, 0, 1, 350, 349, 351, 2000, 16]
    check(wql, lens, 2, 128, ps, 350, 30, ps, extra=1)
    check(wql, lens, 5, 64, ps, 350, 0, ps + 1, distinct=3)


@pytest.mark.parametrize("distinct", [1, 2, 3, 50])
@pytest.mark.parametrize("n", [100, 1500, 9000])
def test_equal_weights_keep_the_first(wql, n, distinct):
    for budget in (1, n // 3, n - 1):
        check(wql, [n, n // 2], 2, 64, 16, budget, budget // 4, distinct, distinct=distinct, what=(n, distinct, budget))


def test_special_weights(wql):
    def odd(w):
        g = torch.Generator().manual_seed(1)
        x = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-45, -1e-45, 1e-38, 3e38, -math.nan])
        pick = torch.randint(0, 10, w.shape, generator=g)
        return torch.where(torch.rand(w.shape, generator=g).cuda() < 0.5, x[pick].cuda(), w)

    for budget in (1, 77, 200, 399, 500, 699):
        check(wql, [700, 300], 2, 64, 16, budget, 5, budget, weights=odd, what=budget)
    check(wql, [2500], 1, 64, 16, 600, 0, 3, weights=lambda w: torch.full_like(w, math.nan))
    check(wql, [2500], 1, 64, 16, 600, 0, 3, weights=lambda w: torch.full_like(w, -math.inf))


@pytest.mark.parametrize("n,budget", [(40000, 8192), (120001, 30000), (65536, 65535), (131072, 100)])
def test_long_contexts(wql, n, budget):
    check(wql, [n], 2, 64, 64, budget, budget // 10, 5)
    check(wql, [n, 5000], 1, 128, 128, budget, 0, 6, weights=lambda w: w.exp())


@pytest.mark.parametrize("seed", range(10))
def test_drawn_cases(wql, seed):
    r = random.Random(seed)
    ps = r.choice([16, 32, 64, 96])
    top = r.choice([50, 600, 5000])
    lens = [r.choice([0, r.randrange(1, top), r.randrange(1, top)]) for _ in range(r.choice([1, 3, 9]))]
    budget = r.randrange(1, top + 10)
    check(wql, lens, r.choice([1, 2, 8]), r.choice([64, 128]), ps, budget, r.choice([0, 1, budget // 2, budget + 5]), seed,
          extra=r.choice([0, 3]), distinct=r.choice([None, 2, 40]), what=(lens, budget, ps))


def test_bad_lengths_and_pages_are_recorded(wql):
    lens = [100, 60]
    cache, table, new_table, w = make(lens, 2, 64, 16, 40, 3)

    def recorded():
        with pytest.raises(wql.WQLError) as e:
            wql.device_status()
        assert e.value.status == 1

    cap = table.shape[1] * 16
    t = table.clone()
    t[t < 0] = 0
    kept, nw, nl = wql.kv_evict_i4(w, cache.clone(), t, i32([cap + 5, -3]), new_table, 40, 2)
    recorded()
    assert nl.tolist() == [40, 0] and kept[0].tolist() == cref.evict(w.cpu(), [cap, 0], 40, 2)[0] and not nw[1].any()
    for page in (-1, cache.shape[0], 2 ** 31 - 1):
        for which in range(2):
            a, b = table.clone(), new_table.clone()
            (b if which else a)[0, 1] = page
            c = cache.clone()
            good, _, _ = wql.kv_evict_i4(w, cache.clone(), table, i32(lens), new_table, 40, 2)
            wql.device_status()
            kept, nw, nl = wql.kv_evict_i4(w, c, a, i32(lens), b, 40, 2)
            recorded()
            assert torch.equal(kept, good)
            ref_c = cache.clone()
            wql.kv_evict_i4(w, ref_c, table, i32(lens), new_table, 40, 2)
            m = new_table[1, :3].long()
            assert torch.equal(c[m], ref_c[m])  # the other sequence's


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 4, 4)])
def test_from_planned_pages_to_decode_over_what_is_kept(wql, D, Hq, Hkv):
    ps, B, budget = 16, 3, 120
    g = torch.Generator().manual_seed(2)
    prompts = [200, 90, 333]
    free = torch.randperm(120, generator=g).to(torch.int32).cuda()
    left = i32([120])
    cache = wql.kv_cache_i4(120, Hkv, D, ps)
    table = torch.full((B, 24), -1, dtype=torch.int32, device="cuda")
    weights = torch.zeros((B, Hkv, 24 * ps), device="cuda")
    held = i32([0] * B)
    want = weights.double()
    for step in range(6):  # prompts in chunks of up to 64 tokens
        new = [max(0, min(64, n - 64 * step)) for n in prompts]
        T = sum(new) + 2
        slots, cu, lens, left = wql.kv_plan_pages(held, i32(new), table, free, left, ps, T)
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g).half().cuda()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        wql.kv_append_i4(k, v, slots, cache)
        lse = torch.zeros((T, Hq), device="cuda")
        y = wql.attention_chunks_kv_i4(q, cache, table, cu, lens, lse=lse)
        o, ob, z, zb = cref.chunks(q, cache, table, cu.tolist(), lens.tolist())
        some = sum(new)
        assert bool(((y[:some].double() - o[:some]).abs() <= ob[:some]).all())
        before = weights.clone()
        wql.kv_weights_i4(q, cache, table, cu, lens, lse, weights)
        want, wb = cref.weights(q, cache, table, cu.tolist(), lens.tolist(), lse, before)
        assert bool(((weights.double() - want).abs() <= wb).all())
        held = lens
    assert held.tolist() == prompts
    # every row's weights add up to one
    assert bool(((weights.double().sum(-1) - held[:, None] * (Hq // Hkv)).abs() < 1e-4 * held[:, None] * (Hq // Hkv)).all())
    new_table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    _, _, planned, left = wql.kv_plan_pages(i32([0] * B), torch.clamp(held, max=budget), new_table, free, left, ps, B * budget)
    k_before = [ref.read(cache, table[b].long()[torch.arange(prompts[b], device="cuda") // ps] * ps
                         + torch.arange(prompts[b], device="cuda") % ps) for b in range(B)]
    kept, w2, lens2 = wql.kv_evict_i4(weights, cache, table, held, new_table, budget, 32)
    assert lens2.tolist() == planned.tolist() == [min(n, budget) for n in prompts]
    assert kept.tolist() == [[x + [-1] * (budget - len(x)) for x in heads] for heads in cref.evict(weights.cpu(), prompts, budget, 32)]
    # a decode step over what is kept: a token more, in the new pages, and its weights behind the kept ones
    slots, cu, lens3, left = wql.kv_plan_pages(lens2, i32([1] * B), new_table, free, left, ps, B)
    qkv = torch.randn((B, Hq + 2 * Hkv, D), generator=g).half().cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    wql.kv_append_i4(k, v, slots, cache)
    y = wql.attention_kv_i4(q, cache, new_table, lens3)
    lse = torch.zeros((B, Hq), device="cuda")
    y2 = wql.attention_chunks_kv_i4(q, cache, new_table, cu, lens3, lse=lse)
    wql.kv_weights_i4(q, cache, new_table, cu, lens3, lse, w2)
    wql.device_status()
    new_k, new_v = wql.kv_read_i4(cache, slots)
    for b in range(B):
        m = min(prompts[b], budget)
        for h in range(Hq):
            kh = h * Hkv // Hq
            at = kept[b, kh, :m].long()
            kk = torch.cat([k_before[b][0][at, kh], new_k[b:b + 1, kh]]).double()
            vv = torch.cat([k_before[b][1][at, kh], new_v[b:b + 1, kh]]).double()
            oo, bb = ref.attend(q[b:b + 1, h].double(), kk, vv, kk.abs(), vv.abs(), i32([m + 1]), D ** -0.5)
            assert bool(((y2[b, h].double() - oo[0]).abs() <= bb[0]).all())
            # the decode kernel takes code * s + lo unrounded: K and V are off by half a step, and a score by |q| |k| of those
            slack = float((q[b, h].double().abs() @ kk.abs().T).max()) * D ** -0.5 * 2.0 ** -11 * 2
            assert bool(((y[b, h].double() - oo[0]).abs() <= bb[0] + (slack + 2.0 ** -10) * float(vv.abs().max())).all())
    assert bool((w2[torch.arange(B), :, lens2.long()] > 0).all())  # the new token looked at itself


@pytest.mark.parametrize("B,H,n,budget", [(20, 16, 900, 400), (5, 8, 900, 700), (3, 8, 2000, 1500), (30, 16, 2000, 300), (2, 8, 4000, 2000),
                                          (3, 8, 7000, 3000), (10, 8, 4000, 1000), (10, 8, 20000, 500), (9, 5, 40000, 700), (40, 8, 9000, 200),
                                          (2, 8, 16000, 16000), (2, 4, 70000, 9000)])
def test_heads_and_widths_that_choose_the_ctas(wql, B, H, n, budget):
    # few and many heads with narrow and wide tables, so that heads have one to eight CTAs and read their weights once or again
    r = random.Random(B * n)
    lens = [max(1, n - (n * i) // (2 * B) - r.randrange(0, 40)) for i in range(B)]
    lens[-1] = 5
    g = torch.Generator().manual_seed(n)
    D, ps = 64, 64
    held = [-(-x // ps) for x in lens]
    width, nw = -(-n // ps), -(-budget // ps)
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b, m in enumerate(held):
        table[b, :m] = torch.randperm(64, generator=g).repeat(m // 64 + 1)[:m].int()  # a pool of 64 pages, read again and again
    cache = torch.randint(0, 256, (64 + B * nw, H, ps // 16, 16 * (D + 8)), generator=g, dtype=torch.uint8).cuda()
    before, table = cache.clone(), table.cuda()
    new_table = (64 + torch.arange(B * nw)).view(B, nw).int().cuda()
    w = torch.randint(-40, 400, (B, H, width * ps), generator=g).float().cuda() / 16  # many equal ones
    kept, kw, kn = wql.kv_evict_i4(w, cache, table, i32(lens), new_table, budget, 20)
    wql.device_status()
    assert kn.tolist() == [min(x, budget) for x in lens] and torch.equal(cache[:64], before[:64])
    for b, x in enumerate(lens):
        m = min(x, budget)
        new = min(20, budget, x)
        # of the others the greatest, of equal ones the first: a stable sort
        order = torch.sort(w[b, :, :x - new], dim=-1, descending=True, stable=True).indices[:, :m - new]
        want = torch.cat([order.sort(-1).values, torch.arange(x - new, x, device="cuda").expand(H, new)], -1)
        assert torch.equal(kept[b, :, :m].long(), want) and bool((kept[b, :, m:] == -1).all()), b
        assert torch.equal(kw[b, :, :m], w[b].gather(1, want)) and not bool(kw[b, :, m:].any())
        i = torch.arange(m, device="cuda")[:, None].expand(m, H)
        src = want.T
        assert torch.equal(rows(cache, new_table[b].long()[i // ps] * ps + i % ps, H, D),
                           rows(before, table[b].long()[src // ps] * ps + src % ps, H, D)), b
