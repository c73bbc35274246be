"""GPU tests of attention over the paged 4-bit cache that see one lost or doubled token of a long context (the criterion of
tests/_attn_norm.py), and of chunks of a prompt over its cached beginning."""
import math

import pytest

torch = pytest.importorskip("torch")

import _attn_norm as norm  # noqa: E402
import _attn_ref as ref  # noqa: E402

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


def within(y, o, bound, what=""):
    err = (y.double() - o).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float(err[bad].max()), bad.nonzero()[0].tolist())


# lens, Lq, Hq, Hkv, D, ps: 1 to 40 rows per K/V head, contexts over many blocks of the grid
LONG = [([9001, 17], 2, 16, 1, 64, 128), ([5003], 1, 8, 2, 128, 64), ([7001, 300], 1, 16, 2, 128, 64), ([6007], 5, 6, 2, 128, 16),
        ([3001] * 5, 4, 16, 4, 64, 32), ([12000], 1, 16, 1, 128, 64), ([4500, 9000, 1], 4, 20, 2, 64, 16), ([20011], 1, 5, 1, 128, 32),
        ([2000] * 40, 1, 8, 1, 64, 64)]


@gpu
@pytest.mark.parametrize("lens,Lq,Hq,Hkv,D,ps", LONG)
def test_rows_of_long_contexts_lose_no_token(wql, lens, Lq, Hq, Hkv, D, ps):
    q, cache, table, kv_lens = ref.paged_case(len(lens), lens, Lq, Hq, Hkv, D, ps, seed=sum(lens))
    q = (q * 0.5).half()  # flat weights: many tokens count
    y = wql.attention_kv_i4(q, cache, table, kv_lens)
    wql.device_status()
    o, tol = norm.kv_i4(q, cache, table, lens)
    norm.within(y, o, tol)


def test_the_criterion_sees_one_lost_token():
    # flat weights over 3000 tokens: without any one of them the outputs are off by more than the tolerance allows
    q, cache, table, lens = ref.paged_case(1, [3000], 1, 8, 1, 64, 32, seed=1, device="cpu")
    q = q * 0
    o, tol = norm.kv_i4(q, cache, table, [3000])
    for t in (0, 31, 32, 1499, 2976, 2999):
        z, _ = norm.kv_i4(q, cache, table, [3000], drop=t)
        assert bool(((z - o).norm(dim=-1) > 1.5 * tol).all())
    q, cache, table, lens = ref.paged_case(1, [3000], 1, 8, 1, 64, 32, seed=1, device="cpu")
    o, tol = norm.kv_i4(q, cache, table, [3000])
    assert bool((tol < 0.02 * o.norm(dim=-1)).all())


@gpu
@pytest.mark.parametrize("Lq,Hq,Hkv,D", [(1, 4, 1, 128), (1, 8, 1, 128), (1, 16, 1, 64), (3, 8, 1, 64), (2, 20, 1, 128)])
def test_each_token_at_a_border_counts_once(wql, Lq, Hq, Hkv, D):
    # V is zero but for one token: the output is its weight times its value, neither nothing nor twice that
    n, ps = 2500, 32
    q, cache, table, kv_lens = ref.paged_case(1, [n], Lq, Hq, Hkv, D, ps, seed=D + Hq)
    q = (q * 0.25).half()
    g = torch.Generator().manual_seed(2)
    one = torch.randn((1, Hkv, D), generator=g).half().cuda() * 100
    keys, _ = ref.read(cache, table[0].long()[torch.arange(n, device="cuda") // ps] * ps + torch.arange(n, device="cuda") % ps)
    zero = torch.zeros((1, Hkv, D), dtype=torch.float16, device="cuda")
    at = torch.arange(n, device="cuda")
    ref.write(cache, table[0].long()[at // ps] * ps + at % ps, keys, zero.expand(n, -1, -1))
    for t in [t for t in range(n) if t < 3 or t >= n - 3 or t % 32 in (0, 15, 16, 31) and t % 3 == 0]:
        slot = int(table[0, t // ps]) * ps + t % ps
        ref.write(cache, torch.tensor([slot]), keys[t:t + 1], one)
        y = wql.attention_kv_i4(q, cache, table, kv_lens)
        o, tol = norm.kv_i4(q, cache, table, [n])
        norm.within(y, o, tol, t)
        ref.write(cache, torch.tensor([slot]), keys[t:t + 1], zero)
    wql.device_status()


# lens, Lq: chunks behind a cached beginning, from the first token on, longer than some sequences, ending inside pages
@gpu
@pytest.mark.parametrize("lens,Lq,Hq,Hkv,D,ps", [([700], 256, 8, 2, 128, 64), ([300], 300, 8, 2, 64, 16), ([1000, 130, 90, 0], 100, 4, 1, 128, 48),
                                                 ([2048], 512, 4, 1, 128, 64), ([517, 33], 33, 6, 2, 64, 32), ([400], 129, 3, 3, 128, 16)])
def test_a_chunk_of_a_prompt_over_its_cached_beginning(wql, lens, Lq, Hq, Hkv, D, ps):
    B = len(lens)
    q, cache, table, kv_lens = ref.paged_case(B, lens, Lq, Hq, Hkv, D, ps, seed=Lq)
    out = torch.full((B, Lq, Hq, D), math.nan, dtype=torch.float16, device="cuda")
    wql.attention_kv_i4(q, cache, table, kv_lens, out=out)
    wql.device_status()
    o, bound = ref.kv_i4(q, cache, table, lens)
    within(out, o, bound)
    o, tol = norm.kv_i4(q, cache, table, lens)
    norm.within(out, o, tol)
    for b, n in enumerate(lens):  # rows of a sequence shorter than the chunk
        if n < Lq:
            assert not out[b, :Lq - n].any()


@gpu
def test_chunks_in_turn_are_the_whole_prompt(wql):
    # a prompt of 300 tokens in chunks of 128, 128 and 44, as an engine feeds them: plan, append, attention over the cache
    Hq, Hkv, D, ps, n = 8, 2, 128, 16, 300
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn((n, Hq + 2 * Hkv, D), generator=g).half().cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = wql.kv_cache_i4(24, Hkv, D, ps)
    table, free, count = torch.full((1, 24), -1, dtype=torch.int32, device="cuda"), torch.arange(24, dtype=torch.int32, device="cuda"), i32([24])
    held, outs = i32([0]), []
    for a in range(0, n, 128):
        e = min(n, a + 128)
        slots, _, held, count = wql.kv_plan_pages(held, i32([e - a]), table, free, count, ps, e - a)
        wql.kv_append_i4(k[a:e], v[a:e], slots, cache)
        outs.append(wql.attention_kv_i4(q[None, a:e], cache, table, held)[0])
    y = torch.cat(outs)
    wql.device_status()
    assert held.tolist() == [n] and int(count) == 24 - 19
    o, bound = ref.kv_i4(q[None], cache, table, [n])
    within(y[None], o, bound)
    o, tol = norm.kv_i4(q[None], cache, table, [n])
    norm.within(y[None], o, tol)
    # and the prompt's own attention over the values that the cache holds, but for their rounding to fp16
    t = torch.arange(n, device="cuda")
    kk, vv = wql.kv_read_i4(cache, (table[0].long()[t // ps] * ps + t % ps).to(torch.int32))
    whole = wql.attention_prompt(q, kk, vv, i32([0, n]))
    assert float((whole.double() - y.double()).norm() / y.double().norm()) < 2e-3
