"""GPU tests of how the attention and 4-bit cache calls are made: repeated, at the same time on two streams, captured and
replayed with a shared workspace, empty, over workspaces of any contents, and over randomly drawn shapes."""
import math
import random

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


def bits(t):
    return t.contiguous().view(torch.int16).clone()


def within(y, o, bound, what=""):
    err = (y.double() - o).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float(err[bad].max()), bad.nonzero()[0].tolist())


def _prompt(lens, Hq, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((sum(lens), Hq + 2 * Hkv, D), generator=g).half().cuda()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], cu


@pytest.mark.parametrize("lens,Lq,Hq,Hkv,D", [([9000, 33, 0, 700], 1, 8, 2, 128), ([4000] * 3, 4, 16, 4, 64),
                                              ([60, 800, 5], 2, 16, 1, 128)])
def test_kv_attention_repeats_bit_for_bit(wql, lens, Lq, Hq, Hkv, D):
    # units that span CTAs are joined by whichever CTA finds them complete: the result must not show which
    q, cache, table, kv_lens = ref.paged_case(len(lens), lens, Lq, Hq, Hkv, D, 16, 3)
    ws = torch.empty((wql.attention_kv_i4_workspace_bytes(len(lens), Lq, Hq, Hkv, D),), dtype=torch.uint8, device="cuda")
    first = bits(wql.attention_kv_i4(q, cache, table, kv_lens, workspace=ws))
    for _ in range(200):
        assert torch.equal(bits(wql.attention_kv_i4(q, cache, table, kv_lens, workspace=ws)), first)
    wql.device_status()


@pytest.mark.parametrize("fill", [0x00, 0xff, 0x7f, "random"])
def test_kv_attention_workspace_may_hold_anything(wql, fill):
    lens = [5000, 40, 1200]
    q, cache, table, kv_lens = ref.paged_case(3, lens, 1, 8, 2, 128, 32, 4)
    o, bound = ref.kv_i4(q, cache, table, lens)
    n = wql.attention_kv_i4_workspace_bytes(3, 1, 8, 2, 128)
    band = 4096
    ws = torch.empty((n + 2 * band,), dtype=torch.uint8, device="cuda")
    if fill == "random":
        ws.random_(0, 256)
    else:
        ws.fill_(fill)
    before = ws.clone()
    y = wql.attention_kv_i4(q, cache, table, kv_lens, workspace=ws[band:band + n])
    within(y, o, bound)
    assert torch.equal(ws[:band], before[:band]) and torch.equal(ws[band + n:], before[band + n:])
    with pytest.raises(wql.WQLError):
        wql.attention_kv_i4(q, cache, table, kv_lens, workspace=ws[:n - 16])
    wql.device_status()


def test_prompt_attention_repeats_bit_for_bit(wql):
    for lens, Hq, Hkv, D in (([1300, 7, 400], 8, 2, 128), ([900, 129], 3, 3, 64), ([128, 1, 256] * 20, 4, 1, 128)):
        q, k, v, cu = _prompt(lens, Hq, Hkv, D, 5)
        c = i32(cu)
        first = bits(wql.attention_prompt(q, k, v, c))
        for _ in range(100):
            assert torch.equal(bits(wql.attention_prompt(q, k, v, c)), first)
    wql.device_status()


def test_calls_on_two_streams_at_once(wql):
    lens = [[7000, 90], [300, 4100]]
    cases = [ref.paged_case(2, n, 1, 8, 2, 128, 16, 20 + i) for i, n in enumerate(lens)]
    prompts = [_prompt([600 + 100 * i, 50], 4, 2, 128, 30 + i) for i in range(2)]
    cus = [i32(p[3]) for p in prompts]
    want = [bits(wql.attention_kv_i4(*c)) for c in cases]
    wantp = [bits(wql.attention_prompt(*p[:3], cu)) for p, cu in zip(prompts, cus)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):  # a workspace each, allocated on its stream
                got[i].append((wql.attention_kv_i4(*cases[i]), wql.attention_prompt(*prompts[i][:3], cus[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for y, z in got[i]:
            assert torch.equal(bits(y), want[i]) and torch.equal(bits(z), wantp[i])
    wql.device_status()


def test_two_graphs_share_a_workspace_one_after_the_other(wql):
    a = ref.paged_case(2, [3000, 64], 1, 8, 2, 128, 16, 40)
    b = ref.paged_case(3, [10, 5000, 77], 1, 16, 2, 64, 32, 41)
    n = max(wql.attention_kv_i4_workspace_bytes(2, 1, 8, 2, 128), wql.attention_kv_i4_workspace_bytes(3, 1, 16, 2, 64))
    ws = torch.empty((n,), dtype=torch.uint8, device="cuda")
    want = [bits(wql.attention_kv_i4(*x)) for x in (a, b)]
    graphs, outs = [], []
    for x in (a, b):
        out = torch.zeros_like(x[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            wql.attention_kv_i4(*x, out=out, workspace=ws)
        graphs.append(g)
        outs.append(out)
    for k in range(40):
        outs[k % 2].fill_(7)
        graphs[k % 2].replay()
        assert torch.equal(bits(outs[k % 2]), want[k % 2])


def test_captured_decode_step_of_all_calls(wql):
    # plan, append, attention of one step in one graph, replayed as the lengths grow
    Hq, Hkv, D, ps, B = 8, 2, 64, 16, 3
    cache = wql.kv_cache_i4(20, Hkv, D, ps)
    table = torch.full((B, 4), -1, dtype=torch.int32, device="cuda")
    free, count = torch.randperm(20).to(torch.int32).cuda(), i32([20])
    held, one = i32([0, 0, 0]), i32([1, 1, 1])
    qkv = torch.empty((B, Hq + 2 * Hkv, D), dtype=torch.float16, device="cuda")
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]

    def step():
        slots, cu, lens, left = wql.kv_plan_pages(held, one, table, free, count, ps, B)
        wql.kv_append_i4(k, v, slots, cache)
        y = wql.attention_kv_i4(q, cache, table, lens)
        held.copy_(lens)
        count.copy_(left)
        return y

    warm = (held.clone(), count.clone(), table.clone())
    qkv.normal_()
    step()  # first calls outside the capture
    for x, y in zip((held, count, table), warm):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step()
    for x, z in zip((held, count, table), warm):
        x.copy_(z)
    for it in range(40):
        qkv.normal_()
        g.replay()
        assert held.tolist() == [it + 1] * B
        o, bound = ref.kv_i4(q[:, None], cache, table, [it + 1] * B)
        within(y[:, None], o, bound, it)
    assert int(count) == 20 - 3 * 3
    wql.device_status()


def test_empty_calls(wql):
    cache = wql.kv_cache_i4(2, 2, 64, 16)
    h = lambda *s: torch.empty(s, dtype=torch.float16, device="cuda")  # noqa: E731
    z = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    assert wql.kv_append_i4(h(0, 2, 64), h(0, 2, 64), z(0), cache) is cache
    k, v = wql.kv_read_i4(cache, z(0))
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)
    assert wql.attention_kv_i4(h(0, 4, 64), cache, z(0, 3), z(0)).shape == (0, 4, 64)
    assert wql.attention_kv_i4(h(3, 0, 4, 64), cache, z(3, 3), z(3)).shape == (3, 0, 4, 64)
    assert wql.attention_prompt(h(0, 4, 64), h(0, 2, 64), h(0, 2, 64), i32([0])).shape == (0, 4, 64)
    out = torch.full((5, 4, 64), 2.0, dtype=torch.float16, device="cuda")
    x = torch.randn((5, 4, 64), device="cuda").half()
    wql.attention_prompt(x, x, x, i32([0]), out=out)        # no sequence
    wql.attention_prompt(x, x, x, i32([3, 3, 3]), out=out)  # sequences without rows
    assert bool((out == 2.0).all())
    wql.device_status()


def test_binding_refusals_on_the_device(wql):
    cache = wql.kv_cache_i4(4, 2, 128, 16)
    x = torch.zeros((4, 2, 128), dtype=torch.float16, device="cuda")
    sl = i32([0, 1, 2, 3])
    for bad in (x.float(), x[:, :1], x[..., :64], x.transpose(1, 2).contiguous().transpose(1, 2), x.cpu(), x[0]):
        with pytest.raises((TypeError, ValueError)):
            wql.kv_append_i4(bad, x, sl, cache)
    with pytest.raises((TypeError, ValueError)):
        wql.kv_append_i4(x, x[:3], sl, cache)
    for bad in (sl.long(), sl[:3], sl.cpu()):
        with pytest.raises((TypeError, ValueError)):
            wql.kv_append_i4(x, x, bad, cache)
    with pytest.raises(wql.WQLError):  # a stride that is no multiple of 8
        odd = torch.zeros((4 * 260,), dtype=torch.float16, device="cuda").as_strided((4, 2, 128), (257, 128, 1))
        wql.kv_append_i4(odd, x, sl, cache)
    q, table, lens = torch.zeros((2, 4, 128), dtype=torch.float16, device="cuda"), i32([[0], [1]]), i32([3, 4])
    for kw in (dict(q=q[:, :3]), dict(table=table[:1]), dict(lens=lens.long()), dict(out=q[:1]),
               dict(workspace=torch.empty((1 << 20,), dtype=torch.int8, device="cuda"))):
        args = dict(q=q, table=table, lens=lens)
        extra = {k: v for k, v in kw.items() if k not in args}
        args.update({k: v for k, v in kw.items() if k in args})
        with pytest.raises((TypeError, ValueError, wql.WQLError)):
            wql.attention_kv_i4(args["q"], cache, args["table"], args["lens"], **extra)
    uneven = torch.zeros((2, 4, 4, 128), dtype=torch.float16, device="cuda")[:, :3]  # tokens not evenly strided
    with pytest.raises(ValueError):
        wql.attention_kv_i4(uneven, cache, table, lens)
    with pytest.raises(wql.WQLError):
        wql.attention_kv_i4(q, cache, table, lens, scale=math.nan)
    with pytest.raises((TypeError, ValueError)):
        wql.attention_prompt(x, x, x, i32([0, 4]).long())
    with pytest.raises(wql.WQLError):
        y = torch.zeros((4, 3, 128), dtype=torch.float16, device="cuda")
        wql.attention_prompt(y, x, x, i32([0, 4]))
    wql.device_status()


@pytest.mark.parametrize("seed", range(12))
def test_drawn_shapes(wql, seed):
    r = random.Random(seed)
    D, ps = r.choice([64, 128]), r.choice([16, 32, 48, 64, 128, 208])
    Hkv, G = r.choice([(1, 1), (1, 8), (2, 3), (3, 5), (2, 16), (4, 2), (1, 20)])
    B, Lq = r.randint(1, 9), r.choice([1, 1, 2, 3, 9])
    lens = [r.choice([0, r.randint(1, 70), r.randint(1, 2500)]) for _ in range(B)]
    q, cache, table, kv_lens = ref.paged_case(B, lens, Lq, Hkv * G, Hkv, D, ps, seed)
    o, bound = ref.kv_i4(q, cache, table, lens)
    within(wql.attention_kv_i4(q, cache, table, kv_lens), o, bound, ("kv", lens, Lq, Hkv, G, D, ps))
    lens = [r.choice([0, r.randint(1, 140), r.randint(1, 1100)]) for _ in range(r.randint(1, 7))] + [1]
    q, k, v, cu = _prompt(lens, Hkv * G, Hkv, D, seed)
    o, bound = ref.prompt(q, k, v, cu)
    within(wql.attention_prompt(q, k, v, i32(cu)), o, bound, ("prompt", lens, Hkv, G, D))
    wql.device_status()
