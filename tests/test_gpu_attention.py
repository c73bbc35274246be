"""GPU tests of attention over the paged 4-bit cache and over packed prompts, against 64-bit restatements with
elementwise bounds derived from the roundings (tests/_attn_ref.py), and of the serving run that uses them together."""
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


def within(y, o, bound, what=""):
    err = (y.double() - o).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float(err[bad].max()), bad.nonzero()[0].tolist())


# ---- 4-bit cache ---------------------------------------------------------------------------------

CASES = [
    # lens, Lq, Hq, Hkv, D, ps
    ([1], 1, 1, 1, 128, 16), ([1], 1, 1, 1, 64, 16), ([2, 1], 1, 8, 1, 128, 16),
    ([15, 16, 17, 31, 32, 33, 47, 48, 49], 1, 4, 2, 128, 16), ([15, 16, 17, 31, 32, 33, 47, 48, 49], 1, 4, 2, 64, 48),
    ([0, 700, 0, 3, 0], 1, 32, 8, 128, 64), ([0, 0, 0], 1, 4, 4, 128, 16), ([700], 1, 32, 32, 128, 16),
    ([513, 1024, 100], 1, 14, 2, 128, 32), ([513, 1024, 100], 1, 64, 4, 64, 32),   # 7 and 16 query heads per K/V head
    ([300, 5], 4, 32, 8, 128, 16), ([300, 5, 2, 0], 3, 8, 8, 64, 80), ([9], 5, 24, 2, 128, 16),  # rows that see nothing
    ([130, 40], 7, 40, 2, 64, 16),     # 140 rows of a K/V head: several row blocks
    ([5003], 1, 8, 2, 128, 64), ([9001, 17], 2, 16, 1, 64, 128),
]


@pytest.mark.parametrize("lens,Lq,Hq,Hkv,D,ps", CASES)
def test_kv_i4_attention(wql, lens, Lq, Hq, Hkv, D, ps):
    B = len(lens)
    q, cache, table, kv_lens = ref.paged_case(B, lens, Lq, Hq, Hkv, D, ps, seed=sum(lens) + Lq)
    out = torch.full((B, Lq, Hq, D), math.nan, dtype=torch.float16, device="cuda")
    y = wql.attention_kv_i4(q, cache, table, kv_lens, out=out)
    assert y is out
    wql.device_status()
    o, bound = ref.kv_i4(q, cache, table, lens)
    within(y, o, bound)
    z = wql.attention_kv_i4(q, cache, table, kv_lens)
    assert torch.equal(y.view(torch.int16), z.view(torch.int16))  # the same again


@pytest.mark.parametrize("seed", range(4))
def test_kv_i4_attention_ragged_batch(wql, seed):
    g = torch.Generator().manual_seed(seed)
    B = [40, 3, 161, 700][seed]
    lens = (torch.rand((B,), generator=g) ** 3 * [3000, 9000, 700, 90][seed]).long().tolist()
    Lq, Hq, Hkv, D, ps = [(1, 8, 2, 128, 16), (1, 12, 4, 128, 64), (2, 6, 3, 64, 32), (1, 4, 1, 64, 16)][seed]
    q, cache, table, kv_lens = ref.paged_case(B, lens, Lq, Hq, Hkv, D, ps, seed)
    y = wql.attention_kv_i4(q, cache, table, kv_lens)
    wql.device_status()
    o, bound = ref.kv_i4(q, cache, table, lens)
    within(y, o, bound)


def test_kv_i4_attention_scales_that_differ_by_decades(wql):
    # V rows of very different size: a rounded weight must be small against its own contribution
    for seed, D in ((1, 128), (2, 64)):
        q, cache, table, kv_lens = ref.paged_case(2, [400, 77], 1, 8, 2, D, 16, seed, spread=6.0)
        y = wql.attention_kv_i4(q, cache, table, kv_lens)
        o, bound = ref.kv_i4(q, cache, table, [400, 77])
        within(y, o, bound)
        # against the largest contribution of the row, not of the cache
        rel = (y.double() - o).norm(dim=-1) / o.norm(dim=-1)
        assert float(rel.max()) < 8 * ref.U16


@pytest.mark.parametrize("Lq,Hq,Hkv,D", [(1, 8, 2, 128), (4, 2, 2, 64), (1, 6, 2, 128), (2, 4, 2, 128), (1, 2, 2, 64)])
def test_kv_i4_attention_of_up_to_four_rows_keeps_what_rounding_its_weights_leaves(wql, Lq, Hq, Hkv, D):
    # Outputs that nearly always round as the 64-bit ones do.  For normally distributed outputs an error of relative
    # size 1e-5 (scores of size 20 summed in 32 bits: 20 * 2^-24 * sqrt(D / 16) / log2 e, less over many tokens)
    # moves 5 % of them to a neighbour, 2e-5 moves 8.5 %; weights rounded to 11 bits (2.3e-4) move 45 %.
    lens = [2900, 333]
    q, cache, table, kv_lens = ref.paged_case(2, lens, Lq, Hq, Hkv, D, 32, seed=5 + D + Hq)
    y = wql.attention_kv_i4(q, cache, table, kv_lens)
    o, bound = ref.kv_i4(q, cache, table, lens)
    within(y, o, bound)
    assert float((y == o.half()).double().mean()) > 0.9


def test_kv_i4_attention_sharp_and_flat_scores(wql):
    q, cache, table, kv_lens = ref.paged_case(2, [1500, 64], 1, 16, 4, 128, 16, 11)
    for scale in (0.0, 1e-3, 1.0, 4.0, -0.3):
        y = wql.attention_kv_i4(q, cache, table, kv_lens, scale=scale)
        o, bound = ref.kv_i4(q, cache, table, [1500, 64], scale)
        within(y, o, bound, scale)


def test_kv_i4_attention_non_finite_rows_reach_only_those_who_see_them(wql):
    lens, Lq = [200], 3
    q, cache, table, kv_lens = ref.paged_case(1, lens, Lq, 4, 2, 128, 16, 5)
    y0 = wql.attention_kv_i4(q, cache, table, kv_lens)
    k = torch.randn((1, 2, 128), device="cuda").half()
    v = k.clone()
    v[0, 1, 3] = math.nan
    slot = int(table[0, 199 // 16]) * 16 + 199 % 16  # the last token: seen by the last row only
    old_k, old_v = wql.kv_read_i4(cache, i32([slot]))
    wql.kv_append_i4(k, v, i32([slot]), cache)
    y = wql.attention_kv_i4(q, cache, table, kv_lens)
    assert torch.equal(y[:, :2].view(torch.int16), y0[:, :2].view(torch.int16))
    assert torch.isnan(y[0, 2, 2:]).all() and torch.isfinite(y[0, 2, :2]).all()
    # a query of infinities spoils its own rows alone
    q2 = q.clone()
    q2[0, 0, 1] = math.inf
    y2 = wql.attention_kv_i4(q2, cache, table, kv_lens)
    keep = torch.ones((Lq, 4), dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    assert torch.equal(torch.nan_to_num(y2[0][keep], nan=7.0), torch.nan_to_num(y[0][keep], nan=7.0))


def test_kv_i4_attention_strided_queries_other_stream_and_graph(wql):
    lens = [333, 50]
    q, cache, table, kv_lens = ref.paged_case(2, lens, 2, 8, 2, 128, 32, 8)
    y = wql.attention_kv_i4(q, cache, table, kv_lens)
    qkv = torch.zeros((4, 12, 128), dtype=torch.float16, device="cuda")
    qkv[:, :8] = q.view(4, 8, 128)
    view = qkv.view(2, 2, 12, 128)[:, :, :8]
    assert torch.equal(wql.attention_kv_i4(view, cache, table, kv_lens), y)
    one = q[:, 0].contiguous()
    assert torch.equal(wql.attention_kv_i4(one, cache, table, kv_lens),
                       wql.attention_kv_i4(one[:, None].contiguous(), cache, table, kv_lens)[:, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        z = wql.attention_kv_i4(q, cache, table, kv_lens)
    s.synchronize()
    assert torch.equal(z, y)
    # a captured call follows the lengths' contents
    out = torch.empty_like(y)
    ws = torch.empty((wql.attention_kv_i4_workspace_bytes(2, 2, 8, 2, 128),), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wql.attention_kv_i4(q, cache, table, kv_lens, out=out, workspace=ws)
    for new in ([333, 50], [100, 0], [1, 49], [333, 50]):
        kv_lens.copy_(i32(new))
        ws.random_(0, 256)  # nothing is kept in the workspace between calls
        graph.replay()
        o, bound = ref.kv_i4(q, cache, table, new)
        within(out, o, bound, new)
    wql.device_status()


def test_kv_i4_attention_bad_pages_and_lengths_are_recorded(wql):
    q, cache, table, kv_lens = ref.paged_case(3, [100, 60, 40], 1, 4, 2, 64, 16, 9)
    good = wql.attention_kv_i4(q, cache, table, kv_lens)
    wql.device_status()
    for page in (-1, cache.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[1, 2] = page
        y = wql.attention_kv_i4(q, cache, t, kv_lens)
        with pytest.raises(wql.WQLError) as e:
            wql.device_status()
        assert e.value.status == 1
        assert torch.equal(y[0], good[0]) and torch.equal(y[2], good[2])
    t = table[:, :4].contiguous()  # 64 tokens: the first length is cut
    y = wql.attention_kv_i4(q, cache, t, kv_lens)
    with pytest.raises(wql.WQLError):
        wql.device_status()
    assert torch.equal(y[1:], good[1:])
    y = wql.attention_kv_i4(q, cache, table, i32([100, -3, 40]))
    wql.device_status()
    assert not y[1].any() and torch.equal(y[0], good[0])


# ---- prompts -----------------------------------------------------------------------------------

PROMPTS = [
    # lens, Hq, Hkv, D
    ([1], 1, 1, 128), ([1], 2, 1, 64), ([2, 1, 3], 4, 2, 128), ([63, 64, 65], 2, 2, 64),
    ([127, 128, 129, 0, 1, 255, 256, 257], 4, 1, 128), ([127, 128, 129, 0, 1, 255, 256, 257], 4, 2, 64),
    ([385, 511, 513], 7, 1, 128), ([640], 3, 3, 128), ([1000, 24], 16, 2, 64), ([2049], 4, 2, 128), ([3000, 1], 2, 1, 64),
    ([1] * 150, 2, 1, 128), ([7, 0, 0, 90] * 40, 2, 2, 64),
]


def _prompt(lens, Hq, Hkv, D, seed, behind=0):
    T = sum(lens) + behind
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g)
    qkv[:, :Hq] *= 0.5 + 2 * torch.rand((1, Hq, 1), generator=g)
    qkv[:, Hq:Hq + Hkv] += torch.randn((1, Hkv, D), generator=g)
    qkv = qkv.half().cuda()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], cu


@pytest.mark.parametrize("lens,Hq,Hkv,D", PROMPTS)
def test_prompt_attention(wql, lens, Hq, Hkv, D):
    q, k, v, cu = _prompt(lens, Hq, Hkv, D, seed=sum(lens) + Hq)
    out = torch.full(q.shape, math.nan, dtype=torch.float16, device="cuda")
    y = wql.attention_prompt(q, k, v, i32(cu), out=out)
    assert y is out
    wql.device_status()
    o, bound = ref.prompt(q, k, v, cu)
    within(y, o, bound)
    z = wql.attention_prompt(q.contiguous(), k.contiguous(), v.contiguous(), i32(cu))
    assert torch.equal(y.view(torch.int16), z.view(torch.int16))


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_attention_tensors_on_16_byte_boundaries(wql, D):
    # every tensor a view that begins 16 bytes behind a 32-byte boundary
    q, k, v, cu = _prompt([150], 4, 2, D, seed=3)
    cu = i32(cu)
    y = wql.attention_prompt(q, k, v, cu)

    def shifted(x):
        z = torch.zeros(x.numel() + 16, dtype=x.dtype, device="cuda")[8:8 + x.numel()].view(x.shape)
        assert z.data_ptr() % 32 == 16
        return z.copy_(x)

    out = shifted(torch.zeros_like(q))
    assert wql.attention_prompt(shifted(q), shifted(k), shifted(v), cu, out=out) is out
    wql.device_status()
    assert torch.equal(out.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("D", [64, 128])
def test_kv_i4_tensors_on_16_byte_boundaries(wql, D):
    q, cache, table, lens = ref.paged_case(3, [40, 700, 9], 2, 8, 2, D, 32, seed=4)
    y = wql.attention_kv_i4(q, cache, table, lens)

    def shifted(x):
        n = 16 // x.element_size()
        z = torch.zeros(x.numel() + 2 * n, dtype=x.dtype, device="cuda")[n:n + x.numel()].view(x.shape)
        assert z.data_ptr() % 32 == 16
        return z.copy_(x)

    work = torch.zeros(wql.attention_kv_i4_workspace_bytes(3, 2, 8, 2, D), dtype=torch.uint8, device="cuda")
    out = wql.attention_kv_i4(shifted(q), shifted(cache), shifted(table), shifted(torch.nn.functional.pad(lens, (0, 1)))[:3],
                              out=shifted(torch.zeros_like(q)), workspace=shifted(work))
    wql.device_status()
    assert torch.equal(out.view(torch.int16), y.view(torch.int16))
    slots = torch.arange(96, dtype=torch.int32, device="cuda")
    k, v = wql.kv_read_i4(cache, slots)
    k2, v2 = wql.kv_read_i4(shifted(cache), shifted(slots), shifted(torch.zeros_like(k)), shifted(torch.zeros_like(v)))
    assert torch.equal(k.view(torch.int16), k2.view(torch.int16)) and torch.equal(v.view(torch.int16), v2.view(torch.int16))
    k, v = torch.randn_like(k), torch.randn_like(v)
    a, b = torch.zeros_like(cache), shifted(torch.zeros_like(cache))
    wql.kv_append_i4(k, v, slots, a)
    wql.kv_append_i4(shifted(k), shifted(v), shifted(slots), b)
    wql.device_status()
    assert torch.equal(a, b)


def test_prompt_attention_rows_of_no_sequence_stay(wql):
    q, k, v, cu = _prompt([100, 70], 4, 2, 128, 1, behind=90)
    out = torch.full(q.shape, 3.0, dtype=torch.float16, device="cuda")
    wql.attention_prompt(q, k, v, i32(cu), out=out)
    o, bound = ref.prompt(q, k, v, cu)
    within(out[:170], o[:170], bound[:170])
    assert bool((out[170:] == 3.0).all())
    gap = [20, 100, 170]  # starts behind the first rows
    out.fill_(3.0)
    wql.attention_prompt(q, k, v, i32(gap), out=out)
    o, bound = ref.prompt(q, k, v, gap)
    within(out[20:170], o[20:170], bound[20:170])
    assert bool((out[:20] == 3.0).all()) and bool((out[170:] == 3.0).all())


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_attention_non_finite_values_reach_only_later_rows(wql, D):
    lens = [150, 300, 40]
    q, k, v, cu = _prompt(lens, 4, 2, D, 3, behind=30)
    clean = wql.attention_prompt(q, k, v, i32(cu))
    k2, v2 = k.clone(), v.clone()
    k2[480:], v2[480:] = math.nan, math.inf          # behind the last sequence's 490 rows: rows 480.. are seen late
    k2[150 + 290], v2[150 + 200, 1, 5] = math.nan, math.inf
    v2[149, 0, :] = math.nan                          # the first sequence's last row: neighbours are not reached
    y = wql.attention_prompt(q, k2, v2, i32(cu))
    same = lambda r, h=slice(None): torch.equal(y[r, h].view(torch.int16), clean[r, h].view(torch.int16))  # noqa: E731
    assert same(slice(0, 149)) and torch.isnan(y[149, :2]).all()
    assert torch.equal(y[149, 2:], clean[149, 2:])
    assert same(slice(150, 350)) and same(slice(450, 480))
    assert same(slice(350, 440), slice(0, 2))
    assert not torch.isfinite(y[350:440, 2:, 5]).any()
    rest = [c for c in range(D) if c != 5]
    assert torch.equal(y[350:440, 2:][..., rest], clean[350:440, 2:][..., rest])
    assert torch.isnan(y[440:450, :, rest]).all() and not torch.isfinite(y[480:490]).any()
    q2 = q.clone()
    q2[17] = math.nan
    y = wql.attention_prompt(q2, k, v, i32(cu))
    keep = [r for r in range(490) if r != 17]
    assert torch.isnan(y[17]).all() and torch.equal(y[keep], clean[keep])


def test_prompt_attention_scales_and_large_scores(wql):
    q, k, v, cu = _prompt([400], 4, 1, 128, 4)
    for scale in (0.0, 1e-3, 2.0):
        y = wql.attention_prompt(q, k, v, i32(cu), scale=scale)
        o, bound = ref.prompt(q, k, v, cu, scale)
        within(y, o, bound, scale)
    # scores that rise along the keys: the running maximum keeps moving
    up = torch.linspace(0, 12, 400, device="cuda")[:, None, None]
    k2 = (k * 0.05 + up * 0.05).half()
    q2 = (q.abs() + 1).half()
    y = wql.attention_prompt(q2, k2, v, i32(cu))
    o, bound = ref.prompt(q2, k2, v, cu)
    within(y, o, bound)


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (3, 3, 128), (4, 1, 64)])
def test_prompt_attention_rows_do_not_depend_on_later_ones(wql, Hq, Hkv, D):
    # to the last bit, although rows from 300 on see scores that grow by thousands
    T, n = 700, 300
    q, k, v, cu = _prompt([T], Hq, Hkv, D, seed=11)
    y = wql.attention_prompt(q, k, v, i32(cu))
    q, k, v = q.clone(), k.clone(), v.clone()
    q[n:] *= 64
    k[n:] *= torch.linspace(1, 64, T - n, device="cuda").half()[:, None, None]
    v[n:] *= -100
    z = wql.attention_prompt(q, k, v, i32(cu))
    short = wql.attention_prompt(q[:n].clone(), k[:n].clone(), v[:n].clone(), i32([0, n]))
    wql.device_status()
    assert torch.equal(y[:n].view(torch.int16), z[:n].view(torch.int16))
    assert torch.equal(y[:n].view(torch.int16), short.view(torch.int16))


def test_prompt_attention_bad_sequences_are_left_out_and_recorded(wql):
    q, k, v, cu = _prompt([50, 60, 70], 2, 1, 64, 6)
    good = wql.attention_prompt(q, k, v, i32(cu))
    for bad in ([0, 50, 40, 180], [0, 50, 110, 181], [-4, 50, 110, 180]):
        out = torch.full(q.shape, 3.0, dtype=torch.float16, device="cuda")
        wql.attention_prompt(q, k, v, i32(bad), out=out)
        with pytest.raises(wql.WQLError) as e:
            wql.device_status()
        assert e.value.status == 1
        if bad[0] == 0:
            n = min(bad[1:3])  # [40, 180) is a sequence too, and shares rows 40 .. 49 with the first
            assert torch.equal(out[:n], good[:n])
        else:
            assert bool((out[:50] == 3.0).all()) and torch.equal(out[50:], good[50:])


def test_prompt_attention_graph_follows_lengths(wql):
    q, k, v, cu = _prompt([300, 212], 4, 2, 128, 7)
    c = i32(cu)
    out = torch.zeros(q.shape, dtype=torch.float16, device="cuda")
    wql.attention_prompt(q, k, v, c, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wql.attention_prompt(q, k, v, c, out=out)
    for new in ([0, 300, 512], [0, 0, 512], [0, 512, 512], [0, 1, 512]):
        c.copy_(i32(new))
        graph.replay()
        o, bound = ref.prompt(q, k, v, new)
        within(out, o, bound, new)


# ---- the run together ----------------------------------------------------------------------------

def test_serving_run_prompt_then_decode(wql):
    """Three requests through one layer as an engine runs it: the QKV projection (W4A16), the page plan, the prompts'
    attention and their K and V into the cache; then decode steps over the cache, one with a request refused for
    want of pages."""
    torch.manual_seed(0)
    Hq, Hkv, D, ps, G = 8, 2, 128, 16, 128
    E = Hq * D
    qkv_w = wql.awq_pack(torch.randn((E, (Hq + 2 * Hkv) * D), device="cuda") * 0.02, G)
    lens = [37, 5, 64]
    T = sum(lens)
    pages = 11
    cache = wql.kv_cache_i4(pages, Hkv, D, ps)
    table = torch.full((3, 6), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages).to(torch.int32).cuda()
    n_free = i32([pages])

    def project(x):
        return wql.w4a16_gemm(x, *qkv_w, G).view(x.shape[0], Hq + 2 * Hkv, D)

    qkv = project(torch.randn((T, E), device="cuda").half())
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    slots, cu, kv_lens, n_free = wql.kv_plan_pages(i32([0, 0, 0]), i32(lens), table, free, n_free, ps, T)
    wql.kv_append_i4(k, v, slots, cache)
    y = wql.attention_prompt(q, k, v, cu)
    o, bound = ref.prompt(q, k, v, [0, 37, 42, 106])
    within(y, o, bound)
    assert int(n_free) == pages - 8 and kv_lens.tolist() == lens
    keys, values = wql.kv_read_i4(cache, slots)
    step = (k.float().amax(-1) - k.float().amin(-1))[..., None] / 15
    assert bool(((keys.float() - k.float()).abs() <= 0.51 * step + 1e-2).all())

    held, rows = kv_lens.clone(), {b: (keys[a:a + n], values[a:a + n]) for b, (a, n) in enumerate(((0, 37), (37, 5), (42, 64)))}
    for it in range(14):
        qkv = project(torch.randn((3, E), device="cuda").half())
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        slots, cu, kv_lens, n_free = wql.kv_plan_pages(held, i32([1, 1, 1]), table, free, n_free, ps, 4)
        assert int(slots[3]) == -1
        wql.kv_append_i4(k, v, slots[:3], cache)
        y = wql.attention_kv_i4(q, cache, table, kv_lens)
        kk, vv = wql.kv_read_i4(cache, slots)
        for b in range(3):
            if int(kv_lens[b]) == 0:
                assert not y[b].any()
                continue
            rows[b] = tuple(torch.cat([r, x[b:b + 1]]) for r, x in zip(rows[b], (kk, vv)))
            n = int(kv_lens[b])
            assert rows[b][0].shape[0] == n == int(held[b]) + 1
        held = torch.where(kv_lens > 0, kv_lens, held)
        o, bound = ref.kv_i4(q[:, None], cache, table, kv_lens.tolist())
        within(y[:, None], o, bound, it)
    # what the cache holds is what was appended, in order
    for b in range(3):
        t = torch.arange(int(held[b]), device="cuda")
        kk, vv = wql.kv_read_i4(cache, (table[b].long()[t // ps] * ps + t % ps).to(torch.int32))
        assert torch.equal(kk, rows[b][0]) and torch.equal(vv, rows[b][1])
    wql.device_status()
