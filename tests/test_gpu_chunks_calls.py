"""GPU tests of how attention over chunks, attention weights and eviction are called: repeated, on two streams at once, captured
and replayed with a shared workspace, over workspaces of any contents, one behind the other without a wait, empty, and refused."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import _attn_ref as ref  # noqa: E402
import _chunks_ref as cref  # noqa: E402


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def within(y, o, bound, what=""):
    err = (y.double() - o).abs()
    bad = ~(err <= bound) & (y.double() != o)
    assert not bool(bad.any()), (what, int(bad.sum()), float(err[bad].max()), bad.nonzero()[0].tolist())


CASES = [([9000, 33, 0, 700], [1, 1, 2, 1], 8, 2, 128, 64), ([4000] * 3, [4, 200, 1], 16, 4, 64, 16), ([60, 800, 5], [60, 300, 5], 14, 2, 128, 32),
         ([20000], [1], 4, 4, 64, 128), ([700, 700], [16, 16], 8, 8, 128, 16)]


class Call:
    """One case and both calls on it."""

    def __init__(self, wql, case, seed=3):
        self.wql, (self.lens, new, Hq, Hkv, D, ps) = wql, case
        self.q, self.cache, self.table, self.cu = cref.case(self.lens, new, Hq, Hkv, D, ps, seed, pad=1)
        self.c, self.n = i32(self.cu), i32(self.lens)
        T, B = self.q.shape[0], len(self.lens)
        self.chunk_bytes = wql.attention_chunks_kv_i4_workspace_bytes(T, B, Hq, Hkv, D)
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros((T, Hq), device="cuda")
        self.before = torch.rand((B, Hkv, self.table.shape[1] * ps), generator=torch.Generator().manual_seed(seed)).cuda()
        self.sums = self.before.clone()

    def chunks(self, **kw):
        self.wql.attention_chunks_kv_i4(self.q, self.cache, self.table, self.c, self.n, out=self.out, lse=self.lse, **kw)

    def weights(self, **kw):
        self.sums.copy_(self.before)
        self.wql.kv_weights_i4(self.q, self.cache, self.table, self.c, self.n, self.lse, self.sums, **kw)

    def bits(self):
        return [x.contiguous().view(torch.int16 if x.dtype == torch.float16 else torch.int32).clone() for x in (self.out, self.lse, self.sums)]

    def check(self):
        o, ob, z, zb = cref.chunks(self.q, self.cache, self.table, self.cu, self.lens)
        a = self.cu[-1]
        within(self.out[:a], o[:a], ob[:a])
        within(self.lse[:a], z[:a], zb[:a])
        w, wb = cref.weights(self.q, self.cache, self.table, self.cu, self.lens, self.lse, self.before)
        within(self.sums, w, wb)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("case", CASES)
def test_repeats_bit_for_bit_without_a_wait_between(wql, case):
    # items and units that CTAs share are joined in their order: the result must not show who did what
    c = Call(wql, case)
    ws = torch.empty((c.chunk_bytes,), dtype=torch.uint8, device="cuda")
    ww = torch.empty((wql.kv_weights_i4_workspace_bytes(),), dtype=torch.uint8, device="cuda")
    c.chunks(workspace=ws)
    c.weights(workspace=ww)
    first = c.bits()
    c.check()
    kept = []
    for _ in range(150):
        c.chunks(workspace=ws)
        c.weights(workspace=ww)
        kept.append(c.bits())
    assert all(same(k, first) for k in kept)
    wql.device_status()


@pytest.mark.parametrize("fill", [0x00, 0xff, 0x7f, "random"])
@pytest.mark.parametrize("case", [CASES[0], CASES[1]])
def test_workspace_may_hold_anything(wql, case, fill):
    c = Call(wql, case)
    band = 4096
    for n, call in ((c.chunk_bytes, c.chunks), (wql.kv_weights_i4_workspace_bytes(), c.weights)):
        ws = torch.empty((n + 2 * band,), dtype=torch.uint8, device="cuda")
        if fill == "random":
            ws.random_(0, 256)
        else:
            ws.fill_(fill)
        before = ws.clone()
        call(workspace=ws[band:band + n])
        assert torch.equal(ws[:band], before[:band]) and torch.equal(ws[band + n:], before[band + n:])
        with pytest.raises(wql.WQLError):
            call(workspace=ws[:n - 16])
    c.weights()  # the refused call left the sums as they were set
    c.check()
    wql.device_status()


def test_calls_on_two_streams_at_once(wql):
    cs = [Call(wql, CASES[0], 20), Call(wql, CASES[1], 21)]
    want = []
    for c in cs:
        c.chunks()
        c.weights()
        want.append(c.bits())
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(25):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):  # a workspace each, allocated on its stream
                cs[i].chunks()
                cs[i].weights()
                got[i].append(cs[i].bits())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(g, want[i]) for g in got[i])
    wql.device_status()


def test_two_graphs_share_workspaces_one_after_the_other(wql):
    cs = [Call(wql, CASES[0], 30), Call(wql, CASES[2], 31)]
    ws = torch.empty((max(c.chunk_bytes for c in cs),), dtype=torch.uint8, device="cuda")
    ww = torch.empty((wql.kv_weights_i4_workspace_bytes(),), dtype=torch.uint8, device="cuda")
    want, graphs = [], []
    for c in cs:
        c.chunks(workspace=ws)
        c.weights(workspace=ww)
        want.append(c.bits())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.chunks(workspace=ws)
            c.weights(workspace=ww)
        graphs.append(g)
    for k in range(30):
        cs[k % 2].out.fill_(0)
        cs[k % 2].lse.fill_(0)
        graphs[k % 2].replay()
        assert same(cs[k % 2].bits(), want[k % 2]), k
    wql.device_status()


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 4, 4)])
def test_captured_step_with_eviction_follows_the_lengths(wql, D, Hq, Hkv):
    # plan, append, attention, weights and eviction of one step in a graph; the contents of the lengths decide what it does
    B, ps, budget = 2, 16, 40
    cache = wql.kv_cache_i4(40, Hkv, D, ps)
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    new_table = i32([[30, 31, 32], [33, 34, 35]])
    free, count = torch.randperm(30).to(torch.int32).cuda(), i32([30])
    held, new = i32([0, 0]), i32([0, 0])
    T = 24
    qkv = torch.empty((T, Hq + 2 * Hkv, D), dtype=torch.float16, device="cuda")
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    sums = torch.zeros((B, Hkv, 8 * ps), device="cuda")
    lse, out = torch.zeros((T, Hq), device="cuda"), torch.zeros((T, Hq, D), dtype=torch.float16, device="cuda")

    def step():
        slots, cu, lens, left = wql.kv_plan_pages(held, new, table, free, count, ps, T)
        wql.kv_append_i4(k, v, slots, cache)
        wql.attention_chunks_kv_i4(q, cache, table, cu, lens, out=out, lse=lse)
        wql.kv_weights_i4(q, cache, table, cu, lens, lse, sums)
        kept = wql.kv_evict_i4(sums, cache, table, lens, new_table, budget, 4)
        held.copy_(lens)
        count.copy_(left)
        return (cu, lens) + kept

    state = [x.clone() for x in (held, count, table, sums)]
    qkv.normal_()
    step()
    for x, y in zip((held, count, table, sums), state):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cu, lens, kept, new_sums, new_lens = step()
    for x, y in zip((held, count, table, sums), state):
        x.copy_(y)
    for adds in ([5, 0], [20, 1], [1, 23], [0, 0], [17, 7], [1, 1], [9, 15]):
        new.copy_(i32(adds))
        qkv.normal_()
        before = sums.clone()
        g.replay()
        n, c = lens.tolist(), cu.tolist()
        o, ob, z, zb = cref.chunks(q, cache, table, c, n)
        a = c[-1]
        within(out[:a], o[:a], ob[:a], adds)
        within(lse[:a], z[:a], zb[:a], adds)
        w, wb = cref.weights(q, cache, table, c, n, lse, before)
        within(sums, w, wb, adds)
        want = cref.evict(sums.cpu(), n, budget, 4)
        assert new_lens.tolist() == [min(x, budget) for x in n]
        for b in range(B):
            for h in range(Hkv):
                m = min(n[b], budget)
                assert kept[b, h, :m].tolist() == want[b][h]
                at = torch.tensor(want[b][h], dtype=torch.int64, device="cuda")
                slots = (table[b].long()[at // ps] * ps + at % ps).int()
                i = torch.arange(m, device="cuda")
                mine = wql.kv_read_i4(cache, (new_table[b].long()[i // ps] * ps + i % ps).int())
                old = wql.kv_read_i4(cache, slots)
                for x, y in zip(mine, old):
                    assert torch.equal(x[:, h], y[:, h])
    wql.device_status()


def test_eviction_repeats_and_leaves_its_inputs(wql):
    g = torch.Generator().manual_seed(0)
    for lens, H, D, ps, budget in (([4000, 3, 900] * 8, 8, 128, 64, 700), ([50000], 3, 64, 64, 9000), ([300], 2, 128, 16, 299)):
        _, cache, table, kv_lens = ref.paged_case(len(lens), lens, 1, H, H, D, ps, 4)
        width = -(-budget // ps)
        cache = torch.cat([cache, torch.zeros((len(lens) * width,) + cache.shape[1:], dtype=torch.uint8, device="cuda")])
        new_table = (cache.shape[0] - 1 - torch.arange(len(lens) * width)).view(len(lens), width).int().cuda()
        w = torch.randn((len(lens), H, table.shape[1] * ps), generator=g).cuda()
        saved = [x.clone() for x in (w, table, kv_lens, new_table)]
        first, after = None, None
        for _ in range(20):
            got = [x.clone() for x in wql.kv_evict_i4(w, cache, table, kv_lens, new_table, budget, 10)]
            if first is None:
                first, after = got, cache.clone()
            assert all(torch.equal(x, y) for x, y in zip(got, first)) and torch.equal(cache, after)
        assert all(torch.equal(x, y) for x, y in zip((w, table, kv_lens, new_table), saved))
    wql.device_status()


def test_shared_pages_are_read_by_all(wql):
    # two sequences with the same beginning: both attend to it, both keep some of it
    lens, new, ps = [200, 180], [8, 20], 16
    q, cache, table, cu = cref.case(lens, new, 8, 2, 64, ps, 6)
    table[1, :8] = table[0, :8]
    o, ob, z, zb = cref.chunks(q, cache, table, cu, lens)
    lse = torch.zeros((28, 8), device="cuda")
    within(wql.attention_chunks_kv_i4(q, cache, table, i32(cu), i32(lens), lse=lse), o, ob)
    sums = torch.zeros((2, 2, table.shape[1] * ps), device="cuda")
    wql.kv_weights_i4(q, cache, table, i32(cu), i32(lens), lse, sums)
    w, wb = cref.weights(q, cache, table, cu, lens, lse, torch.zeros_like(sums))
    within(sums, w, wb)
    big = torch.cat([cache, torch.zeros((8,) + cache.shape[1:], dtype=torch.uint8, device="cuda")])
    new_table = (cache.shape[0] + torch.arange(8)).view(2, 4).int().cuda()
    kept, _, n = wql.kv_evict_i4(sums, big, table, i32(lens), new_table, 64, 5)
    assert n.tolist() == [64, 64] and kept.tolist() == cref.evict(sums.cpu(), lens, 64, 5)
    assert torch.equal(big[:cache.shape[0]], cache)
    i = torch.arange(64, device="cuda")
    for b in range(2):
        mine = wql.kv_read_i4(big, (new_table[b].long()[i // ps] * ps + i % ps).int())
        for h in range(2):
            at = kept[b, h].long()
            old = wql.kv_read_i4(cache, (table[b].long()[at // ps] * ps + at % ps).int())
            for x, y in zip(mine, old):
                assert torch.equal(x[:, h], y[:, h])
    wql.device_status()


def test_empty_calls(wql):
    cache = wql.kv_cache_i4(2, 2, 64, 16)
    h = lambda *s: torch.empty(s, dtype=torch.float16, device="cuda")  # noqa: E731
    z = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *s: torch.empty(s, dtype=torch.float32, device="cuda")  # noqa: E731
    assert wql.attention_chunks_kv_i4(h(0, 4, 64), cache, z(2, 3), i32([0, 0, 0]), i32([0, 0])).shape == (0, 4, 64)
    x, out = torch.randn((5, 4, 64), device="cuda").half(), torch.full((5, 4, 64), 2.0, dtype=torch.float16, device="cuda")
    lse, sums = torch.full((5, 4), 2.0, device="cuda"), torch.full((3, 2, 48), 2.0, device="cuda")
    table = torch.zeros((3, 3), dtype=torch.int32, device="cuda")
    for cu, n in ((i32([2, 2, 2, 2]), i32([9, 0, 40])),):  # sequences without rows
        wql.attention_chunks_kv_i4(x, cache, table, cu, n, out=out, lse=lse)
        wql.kv_weights_i4(x, cache, table, cu, n, lse, sums)
    wql.attention_chunks_kv_i4(x, cache, z(0, 3), i32([0]), z(0), out=out, lse=lse)  # no sequence
    wql.kv_weights_i4(x, cache, z(0, 3), i32([0]), z(0), lse, f(0, 2, 48))
    assert bool((out == 2.0).all()) and bool((lse == 2.0).all()) and bool((sums == 2.0).all())
    kept, w, n = wql.kv_evict_i4(f(0, 2, 48), cache, z(0, 3), z(0), z(0, 1), 5)
    assert kept.shape == (0, 2, 5) and w.shape == (0, 2, 16) and n.shape == (0,)
    kept, w, n = wql.kv_evict_i4(sums, cache, table, i32([0, 0, 0]), i32([[-1], [-1], [-1]]), 5)  # nothing to keep: pages are not looked at
    assert n.tolist() == [0, 0, 0] and bool((kept == -1).all()) and not bool(w.any())
    wql.device_status()


def test_binding_refusals_on_the_device(wql):
    q, cache, table, cu = cref.case([40, 30], [4, 3], 4, 2, 128, 16, 9)
    c, n = i32(cu), i32([40, 30])
    lse, sums = torch.zeros((7, 4), device="cuda"), torch.zeros((2, 2, table.shape[1] * 16), device="cuda")
    new_table = i32([[0], [1]])
    refused = (TypeError, ValueError, wql.WQLError)
    for bad in (q.float(), q[:, :3], q[..., :64], q.cpu(), q[0], q.transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises(refused):
            wql.attention_chunks_kv_i4(bad, cache, table, c, n)
        with pytest.raises(refused):
            wql.kv_weights_i4(bad, cache, table, c, n, lse, sums)
    for kw in (dict(block_table=table[:1]), dict(block_table=table.long()), dict(cu_new=c[:2]), dict(cu_new=c.cpu()), dict(kv_lens=n.long()),
               dict(out=q[:3]), dict(out=q.float()), dict(lse=lse[:3]), dict(lse=lse.double()), dict(scale=math.nan), dict(scale=2.0 ** 65),
               dict(workspace=torch.empty((1 << 26,), dtype=torch.int8, device="cuda")), dict(workspace=torch.empty((64,), dtype=torch.uint8, device="cuda"))):
        args = dict(q=q, cache=cache, block_table=table, cu_new=c, kv_lens=n)
        args.update(kw)
        with pytest.raises(refused):
            wql.attention_chunks_kv_i4(**args)
    for kw in (dict(lse=lse[:, :3]), dict(lse=None), dict(weights=sums[:, :, :16]), dict(weights=sums.double()), dict(weights=None), dict(scale=math.inf),
               dict(workspace=torch.empty((64,), dtype=torch.uint8, device="cuda"))):
        args = dict(q=q, cache=cache, block_table=table, cu_new=c, kv_lens=n, lse=lse, weights=sums)
        args.update(kw)
        with pytest.raises(refused):
            wql.kv_weights_i4(**args)
    for kw in (dict(weights=sums[:1]), dict(weights=sums.half()), dict(block_table=table.cpu()), dict(new_table=new_table[:1]), dict(new_table=new_table.long()),
               dict(budget=0), dict(budget=17), dict(recent=-1), dict(kept=i32([1])), dict(new_weights=sums), dict(new_lens=n[:1])):
        args = dict(weights=sums, cache=cache, block_table=table, kv_lens=n, new_table=new_table, budget=8)
        args.update(kw)
        with pytest.raises(refused):
            wql.kv_evict_i4(**args)
    many = torch.zeros((7, 258, 128), dtype=torch.float16, device="cuda")
    with pytest.raises(wql.WQLError):  # 129 query heads to a K/V head
        wql.attention_chunks_kv_i4(many, cache, table, c, n)
    assert not bool(lse.any()) and not bool(sums.any())
    wql.device_status()


def test_pool_of_more_than_4_gib(wql):
    # the same sequences in a small pool and at the end of a large one, whose offsets pass 2^32 bytes
    lens, new, D, H, ps = [150, 70], [9, 1], 128, 8, 64
    q, small, table, cu = cref.case(lens, new, 16, H, D, ps, 12)
    held = small.shape[0]
    pages = (1 << 32) // (H * ps * (D + 8)) + 40
    big = torch.empty((pages, H, ps // 16, 16 * (D + 8)), dtype=torch.uint8, device="cuda")
    big[-held:] = small
    shift = pages - held
    c, n = i32(cu), i32(lens)
    got = []
    for cache, by, t in ((small, 0, table), (big, shift, torch.where(table < 0, table, table + shift))):
        lse, sums = torch.zeros((10, 16), device="cuda"), torch.zeros((2, H, table.shape[1] * ps), device="cuda")
        out = wql.attention_chunks_kv_i4(q, cache, t, c, n, lse=lse)
        wql.kv_weights_i4(q, cache, t, c, n, lse, sums)
        room = torch.zeros((2,) + cache.shape[1:], dtype=torch.uint8, device="cuda")
        pool = torch.cat([cache, room]) if by == 0 else cache
        to = i32([[held], [held + 1]]) if by == 0 else i32([[0], [pages - held - 1]])  # from the end to the beginning, and at the end
        kept, kw, kn = wql.kv_evict_i4(sums, pool, t, n, to, 40, 7)
        moved = [pool[int(p), :, :2].clone() for p in to.flatten()]
        got.append([out.view(torch.int16), lse.view(torch.int32), sums.view(torch.int32), kept, kw.view(torch.int32), kn] +
                   [m[:, 0] for m in moved])
    assert same(got[0], got[1])
    o, ob, _, _ = cref.chunks(q, small, table, cu, lens)
    within(got[0][0].view(torch.float16), o, ob)
    wql.device_status()


def test_largest_batch(wql):
    B, ps, H = 4096, 16, 1
    lens = [(i * 37) % 47 for i in range(B)]
    new = [min(n, (1, 1, 2, 5, 0)[i % 5]) for i, n in enumerate(lens)]
    q, cache, table, cu = cref.case(lens, new, 2, H, 64, ps, 13)
    c, n = i32(cu), i32(lens)
    lse, sums = torch.zeros(q.shape[:2], device="cuda"), torch.zeros((B, H, table.shape[1] * ps), device="cuda")
    out = wql.attention_chunks_kv_i4(q, cache, table, c, n, lse=lse)
    o, ob, z, zb = cref.chunks(q, cache, table, cu, lens)
    within(out, o, ob)
    within(lse, z, zb)
    wql.kv_weights_i4(q, cache, table, c, n, lse, sums)
    w, wb = cref.weights(q, cache, table, cu, lens, lse, torch.zeros_like(sums))
    within(sums, w, wb)
    pages = cache.shape[0]
    pool = torch.cat([cache, torch.zeros((B,) + cache.shape[1:], dtype=torch.uint8, device="cuda")])
    kept, _, kn = wql.kv_evict_i4(sums, pool, table, n, (pages + torch.arange(B)).view(B, 1).int().cuda(), 9, 2)
    want = cref.evict(sums.cpu(), lens, 9, 2)
    for b, (k, m) in enumerate(zip(kept.tolist(), kn.tolist())):
        assert m == min(9, lens[b]) and k[0][:m] == want[b][0] and k[0][m:] == [-1] * (9 - m)
    wql.device_status()


def test_most_heads(wql):
    # 65535 heads of their own; 128 query heads to each of two
    for Hq, Hkv, some in ((65535, 65535, [0, 1, 40000, 65534]), (256, 2, [0, 1])):
        lens, new, G = [21, 9], [2, 1], Hq // Hkv
        q, cache, table, cu = cref.case(lens, new, Hq, Hkv, 64, 16, 14)
        c, n = i32(cu), i32(lens)
        lse, sums = torch.zeros((3, Hq), device="cuda"), torch.zeros((2, Hkv, table.shape[1] * 16), device="cuda")
        out = wql.attention_chunks_kv_i4(q, cache, table, c, n, lse=lse)
        wql.kv_weights_i4(q, cache, table, c, n, lse, sums)
        heads = [h * G + g for h in some for g in range(G)]
        o, ob, z, zb = cref.chunks(q[:, heads], cache[:, some], table, cu, lens)
        within(out[:, heads], o, ob, Hq)
        within(lse[:, heads], z, zb, Hq)
        w, wb = cref.weights(q[:, heads], cache[:, some], table, cu, lens, lse[:, heads], torch.zeros_like(sums[:, some]))
        within(sums[:, some], w, wb, Hq)
        # the weights of a row and head add up to one, to 1e-3 (scores are off by 72 * 2^-23 * scale sum |q k| < 1e-4 here)
        assert bool(((sums.double().sum(-1) - i32([2 * G, G])[:, None]).abs() < 2 * G * 1e-3).all())
    wql.device_status()


def test_rows_of_two_sequences_and_pages_twice_in_one(wql):
    # starts 0 5 2 7: rows 0-4 are the first sequence's, 2-6 the third's, the second ends before it begins
    lens, ps = [60, 30, 45], 16
    q, cache, table, _ = cref.case(lens, [5, 1, 1], 8, 2, 128, ps, 15)
    table[0, 2], table[0, 1] = table[0, 0], table[2, 1]  # a page twice, and one of another sequence
    lse = torch.zeros((7, 8), device="cuda")
    y = wql.attention_chunks_kv_i4(q, cache, table, i32([0, 5, 2, 7]), i32(lens), lse=lse)
    with pytest.raises(wql.WQLError):
        wql.device_status()
    first, third = cref.chunks(q, cache, table[:1], [0, 5], lens[:1]), cref.chunks(q, cache, table[2:], [2, 7], lens[2:])
    for got, i in ((y, 0), (lse, 2)):
        within(got[:2], first[i][:2], first[i + 1][:2])
        within(got[5:], third[i][5:], third[i + 1][5:])
        for r in range(2, 5):  # both write these, 16 or 32 bytes at a time and in no order: each value is one of the two
            a = (got[r].double() - first[i][r]).abs() <= first[i + 1][r]
            b = (got[r].double() - third[i][r]).abs() <= third[i + 1][r]
            assert bool((a | b).all())
    # both add to sums of their own
    lse0 = torch.where(torch.arange(7, device="cuda")[:, None] < 5, first[2].nan_to_num(), third[2]).float()
    sums = torch.zeros((3, 2, table.shape[1] * ps), device="cuda")
    wql.kv_weights_i4(q, cache, table, i32([0, 5, 2, 7]), i32(lens), lse0, sums)
    with pytest.raises(wql.WQLError):
        wql.device_status()
    for b, cu in ((0, [0, 5]), (2, [2, 7])):
        w, wb = cref.weights(q, cache, table[b:b + 1], cu, lens[b:b + 1], lse0, torch.zeros_like(sums[:1]))
        within(sums[b:b + 1], w, wb, b)
    assert not bool(sums[1].any())
    pool = torch.cat([cache, torch.zeros((2,) + cache.shape[1:], dtype=torch.uint8, device="cuda")])
    new_table = i32([[cache.shape[0], cache.shape[0] + 1]])
    kept, _, _ = wql.kv_evict_i4(sums[:1].contiguous(), pool, table[:1].contiguous(), i32(lens[:1]), new_table, 25, 3)
    i = torch.arange(25, device="cuda")
    mine = wql.kv_read_i4(pool, (new_table[0].long()[i // ps] * ps + i % ps).int())
    for h in range(2):
        at = kept[0, h].long()
        old = wql.kv_read_i4(cache, (table[0].long()[at // ps] * ps + at % ps).int())
        for a, b in zip(mine, old):
            assert torch.equal(a[:, h], b[:, h])
    wql.device_status()


def test_evictions_at_once_and_captured(wql):
    # on two streams in one pool with pages apart, and in a graph whose weights and lengths change
    g = torch.Generator().manual_seed(2)
    H, D, ps, budget = 4, 128, 64, 200
    _, cache, table, kv_lens = ref.paged_case(4, [3000, 900, 5000, 10], 1, H, H, D, ps, 5)
    pages, width = cache.shape[0], -(-budget // ps)
    cache = torch.cat([cache, torch.zeros((4 * width,) + cache.shape[1:], dtype=torch.uint8, device="cuda")])
    new_table = (pages + torch.arange(4 * width)).view(4, width).int().cuda()
    w = torch.randn((4, H, table.shape[1] * ps), generator=g).cuda()
    want = [x.clone() for x in wql.kv_evict_i4(w, cache, table, kv_lens, new_table, budget, 16)]
    after = cache.clone()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    halves = [[x[2 * i:2 * i + 2].contiguous() for x in (w, table, kv_lens, new_table)] for i in range(2)]
    cache[pages:] = 0
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                a, t, n, nt = halves[i]
                got[i].append([x.clone() for x in wql.kv_evict_i4(a, cache, t, n, nt, budget, 16)])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y[2 * i:2 * i + 2]) for one in got[i] for x, y in zip(one, want))
    assert torch.equal(cache, after)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept, nw, nl = wql.kv_evict_i4(w, cache, table, kv_lens, new_table, budget, 16)
    for lens in ([3000, 900, 5000, 10], [1, 0, 4999, 9], [2500, 201, 0, 3]):  # no more than there are pages for
        w.normal_()
        kv_lens.copy_(i32(lens))
        graph.replay()
        rows = cref.evict(w.cpu(), lens, budget, 16)
        for b, n in enumerate(lens):
            m = min(n, budget)
            assert int(nl[b]) == m and kept[b, :, :m].tolist() == rows[b] and bool((kept[b, :, m:] == -1).all())
    wql.device_status()


def test_ragged_prompts_right_after_allocation(wql):
    # whole prompts of all lengths in small pages, first read from memory that nothing has touched since it was written: copies that
    # land late and out of order must not be taken for others of the same slot
    n, B = 587, 38
    lens = [max(1, n - (n * r) // B - r % 7) for r in range(B)]
    for D, Hq, Hkv, ps, seed in ((128, 8, 2, 32, 1), (128, 32, 8, 16, 2), (64, 8, 2, 32, 3)):
        order = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
        some = [lens[i] for i in order]
        q, cache, table, cu = cref.case(some, some, Hq, Hkv, D, ps, seed, pad=3)
        o, ob, z, zb = cref.chunks(q, cache, table, cu, some)
        first = None
        for _ in range(20):
            cold, other, lse = cache.clone(), torch.empty((1 << 28,), dtype=torch.uint8, device="cuda"), torch.zeros(q.shape[:2], device="cuda")
            other.zero_()  # the caches hold something else
            y = wql.attention_chunks_kv_i4(q, cold, table, i32(cu), i32(some), lse=lse)
            got = [y[:cu[-1]].view(torch.int16), lse[:cu[-1]].view(torch.int32)]
            if first is None:
                first = got
                within(y[:cu[-1]], o[:cu[-1]], ob[:cu[-1]], D)
                within(lse[:cu[-1]], z[:cu[-1]], zb[:cu[-1]], D)
            assert same(got, first)
    wql.device_status()
