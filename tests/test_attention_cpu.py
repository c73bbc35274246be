"""CPU tests of the attention and 4-bit cache calls: what the C ABI and the binding refuse (before anything touches a
device), and the 64-bit restatements the GPU tests compare against, pinned to exact rational arithmetic."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import _attn_ref as ref  # noqa: E402

OK, EINVAL, EUNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p(1 << 20)      # never read: validation comes first
ODD = ctypes.c_void_p((1 << 20) + 2)
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib(wql_lib):
    return wql_lib.load()


def plan(lib, B=4, ps=16, cap=8, width=4, T=32, ctx=P, new=P, free=P, count=P, table=P, cu=P, lens=P, slots=P,
         left=ctypes.c_void_p(2 << 20)):
    return lib.wql_kv_plan_pages(ctx, new, B, ps, free, cap, count, table, width, T, cu, lens, slots, left, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(B=-1), EINVAL, b"B"), (dict(B=4097), EUNSUPPORTED, b"4096"), (dict(ps=0), EINVAL, b"page_size"),
    (dict(ps=24), EINVAL, b"page_size"), (dict(width=0), EINVAL, b"table_width"),
    (dict(width=1 << 20, ps=2048), EINVAL, b"2^31"), (dict(T=-1), EINVAL, b"T"), (dict(cap=-1), EINVAL, b"free_capacity"),
    (dict(slots=ODD), EINVAL, b"slots"), (dict(slots=None), EINVAL, b"slots"), (dict(ctx=None), EINVAL, b"ctx_lens"),
    (dict(table=ODD), EINVAL, b"block_table"), (dict(count=None), EINVAL, b"free_count"),
    (dict(left=P), EINVAL, b"free_count_out"), (dict(free=None), EINVAL, b"free_pages")])
def test_plan_refusals(lib, kw, status, word):
    assert plan(lib, **kw) == status
    assert word in lib.wql_last_error()


def test_cache_refusals(lib):
    def append(T=4, H=2, D=128, ks=256, vs=256, pages=3, ps=16, k=P, v=P, slots=P, cache=P):
        return lib.wql_kv_append_i4(k, v, ks, vs, T, H, D, slots, cache, pages, ps, None)

    assert append(D=96) == EUNSUPPORTED and b"64 or 128" in lib.wql_last_error()
    assert append(ks=255) == EINVAL and append(vs=250) == EINVAL and append(ks=260) == EINVAL  # too short, not 8-fold
    assert append(H=0) == EINVAL and append(T=-1) == EINVAL and append(pages=0) == EINVAL
    assert append(pages=1 << 28) == EINVAL and b"2^31" in lib.wql_last_error()
    assert append(ps=8) == EINVAL and append(k=ODD) == EINVAL and append(cache=ODD) == EINVAL and append(slots=ODD) == EINVAL
    assert append(T=1 << 30, H=2, pages=1) == EUNSUPPORTED
    assert append(T=0, k=None, v=None, slots=None, cache=None) == OK

    def read(T=4, H=2, D=64, pages=3, ps=16, cache=P, slots=P, k=P, v=P):
        return lib.wql_kv_read_i4(cache, pages, ps, H, D, slots, T, k, v, None)

    assert read(D=32) == EUNSUPPORTED and read(k=ODD) == EINVAL and read(v=None) == EINVAL and read(slots=None) == EINVAL
    assert read(T=0, cache=None, slots=None, k=None, v=None) == OK


def test_attention_refusals(lib):
    def kv(B=2, Lq=1, Hq=4, Hkv=2, D=128, qs=512, pages=3, ps=16, width=4, scale=0.1, q=P, cache=P, table=P, lens=P,
           out=P, ws=P, n=1 << 40):
        return lib.wql_attention_kv_i4(q, qs, B, Lq, Hq, Hkv, D, cache, pages, ps, table, width, lens, F(scale), out, ws, n, None)

    assert kv(Hq=5) == EINVAL and kv(Hkv=0) == EINVAL and kv(Hq=1) == EINVAL and b"multiple" in lib.wql_last_error()
    assert kv(D=256, qs=1024) == EUNSUPPORTED and kv(qs=511) == EINVAL and kv(qs=516) == EINVAL
    assert kv(scale=math.nan) == EINVAL and kv(scale=math.inf) == EINVAL and b"finite" in lib.wql_last_error()
    assert kv(width=0) == EINVAL and kv(ps=20) == EINVAL and kv(B=-1) == EINVAL and kv(Lq=-2) == EINVAL
    assert kv(ws=None) == EINVAL and kv(ws=ODD) == EINVAL and kv(n=64) == EINVAL and b"workspace" in lib.wql_last_error()
    assert kv(lens=None) == EINVAL and kv(table=ODD) == EINVAL and kv(out=ODD) == EINVAL
    assert kv(B=1 << 20, Hq=64, Hkv=64, qs=64 * 128, width=1 << 20) == EUNSUPPORTED
    assert kv(B=0, q=None, cache=None, table=None, lens=None, out=None, ws=None, n=0) == OK
    assert kv(Lq=0, q=None, cache=None, table=None, lens=None, out=None, ws=None, n=0) == OK
    assert lib.wql_attention_kv_i4_workspace_bytes(2, 1, 4, 2, 128) > 0
    assert lib.wql_attention_kv_i4_workspace_bytes(2, 1, 5, 2, 128) == 0

    def prompt(T=8, Hq=4, Hkv=2, D=128, qs=512, ks=256, vs=256, B=1, scale=0.1, q=P, k=P, v=P, cu=P, out=P):
        return lib.wql_attention_prompt(q, qs, k, ks, v, vs, T, Hq, Hkv, D, cu, B, F(scale), out, None)

    assert prompt(Hq=3) == EINVAL and prompt(D=80) == EUNSUPPORTED and prompt(qs=256) == EINVAL and prompt(ks=252) == EINVAL
    assert prompt(T=-1) == EINVAL and prompt(B=-1) == EINVAL and prompt(scale=-math.inf) == EINVAL
    assert prompt(cu=None) == EINVAL and prompt(v=ODD) == EINVAL and prompt(out=None) == EINVAL
    assert prompt(Hq=65536, Hkv=1, qs=65536 * 128) == EUNSUPPORTED
    assert prompt(T=0, q=None, k=None, v=None, cu=None, out=None) == OK
    assert prompt(B=0, q=None, k=None, v=None, cu=None, out=None) == OK


def test_binding_refuses_before_any_launch(wql_lib):
    w = wql_lib
    z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)  # noqa: E731
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    cache = z(2, 2, 1, 16 * 136, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        w.kv_plan_pages(z(2), z(2), z(2, 3), z(4), z(1), 16, 5)
    with pytest.raises(ValueError, match="CUDA"):
        w.kv_append_i4(h(3, 2, 128), h(3, 2, 128), z(3), cache)
    with pytest.raises(ValueError, match="kv_cache_i4"):
        w.kv_read_i4(z(2, 2, 5, dtype=torch.uint8), z(3))
    with pytest.raises(ValueError, match="CUDA"):
        w.attention_kv_i4(h(2, 4, 128), cache, z(2, 1), z(2))
    with pytest.raises(ValueError, match="CUDA"):
        w.attention_prompt(h(4, 2, 64), h(4, 2, 64), h(4, 2, 64), z(2))
    with pytest.raises(TypeError):
        w.attention_prompt(None, h(4, 2, 64), h(4, 2, 64), z(2))
    with pytest.raises(ValueError, match="head_dim"):
        w.kv_cache_i4(2, 2, 96, 16, device="cpu")
    with pytest.raises(ValueError, match="page_size"):
        w.kv_cache_i4(2, 2, 64, 20, device="cpu")
    assert tuple(w.kv_cache_i4(3, 2, 64, 48, device="cpu").shape) == (3, 2, 3, 16 * 72)


# ---- the restatements --------------------------------------------------------------------------

def _fp16(x: Fraction) -> Fraction:
    """The fp16 number nearest to x >= 0, ties to even, from the definition of the format."""
    if x == 0:
        return Fraction(0)
    e = max(math.floor(math.log2(float(x))), -14)
    while Fraction(2) ** e > x and e > -14:
        e -= 1
    while Fraction(2) ** (e + 1) <= x:
        e += 1
    ulp = Fraction(2) ** (e - 10)
    n, rest = divmod(x, ulp)
    if rest * 2 > ulp or (rest * 2 == ulp and n % 2):
        n += 1
    return n * ulp


def _round_even(x: Fraction) -> int:
    n, rest = divmod(x, 1)
    return int(n + (1 if rest * 2 > 1 or (rest * 2 == 1 and n % 2) else 0))


@pytest.mark.parametrize("seed", range(6))
def test_quantise_is_the_real_quotient_rounded_once(seed):
    g = torch.Generator().manual_seed(seed)
    if seed < 3:
        x = torch.randn((20, 64), generator=g) * 10.0 ** (2 * seed - 2) + seed
    else:  # few mantissa bits: ties abound
        x = torch.randint(-16, 17, (20, 64), generator=g) * 2.0 ** (seed - 14)
    x = x.half()
    x[0] = 3.5
    c, s, lo = ref.quantise(x)
    for r in range(x.shape[0]):
        v = [Fraction(float(t)) for t in x[r]]
        step = _fp16((max(v) - min(v)) / 15) or Fraction(1)
        assert Fraction(float(s[r])) == step and Fraction(float(lo[r])) == min(v)
        want = [min(max(_round_even((t - min(v)) / step), 0), 15) for t in v]
        assert c[r].tolist() == want


def test_write_and_read_round_trip_and_layout():
    cache = torch.zeros((3, 2, 2, 16 * 72), dtype=torch.uint8)
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn((70, 2, 64), generator=g).half() for _ in range(2))
    slots = torch.randperm(96, generator=g)[:70]
    ref.write(cache, slots, k, v)
    kk, vv = ref.read(cache, slots)
    for x, y in ((k, kk), (v, vv)):
        step = (x.double().amax(-1) - x.double().amin(-1))[..., None] / 15
        assert bool(((x.double() - y.double()).abs() <= step * 0.501 + y.double().abs() * 2.0 ** -11 + 2.0 ** -24).all())
    t = 5  # one row's bytes, by hand
    page, blk, row = int(slots[t]) // 32, int(slots[t]) % 32 // 16, int(slots[t]) % 16
    c, s, lo = ref.quantise(v[t, 1])
    b = cache[page, 1, blk]
    codes = b[512 + 32 * row:512 + 32 * (row + 1)]
    assert (codes & 15).tolist() == c[0::2].tolist() and (codes >> 4).tolist() == c[1::2].tolist()
    par = b[1024 + 64 + 4 * row:1024 + 64 + 4 * row + 4].contiguous().view(torch.float16)
    assert float(par[0]) == float(s) and float(par[1]) == float(lo)


def test_attention_restatement_against_direct_sums():
    q, cache, table, lens = ref.paged_case(2, [19, 3], 2, 4, 2, 64, 16, 1, device="cpu")
    o, bound = ref.kv_i4(q, cache, table, [19, 3])
    t = torch.arange(19)
    k, v = (x.double() for x in ref.read(cache, table[0].long()[t // 16] * 16 + t % 16))
    for r in range(2):
        for h in range(4):
            n = 19 - 2 + r + 1
            e = [math.exp(float(q[0, r, h].double() @ k[j, h // 2]) / 8) for j in range(n)]
            want = sum(x * v[j, h // 2] for j, x in enumerate(e)) / sum(e)
            # read() rounds k and v to fp16: that alone may move a score by 64 * 2^-11 of its terms
            assert bool(((o[0, r, h] - want).abs() < 0.05 * want.abs().max() + 1e-3).all())
            assert bool((bound[0, r, h] < 0.02).all())
    empty = ref.kv_i4(q[:, :2], cache, table, [1, 0])
    assert not empty[0][1].any() and not empty[0][0, 0].any() and empty[0][0, 1].any()


def test_plan_restatement_keeps_pages_apart():
    rng = np.random.default_rng(3)
    for _ in range(20):
        B, ps = int(rng.integers(1, 12)), 16
        ctx, new = rng.integers(0, 60, B), rng.integers(0, 40, B)
        held = -(-ctx // ps)
        pages = rng.permutation(400)
        table = np.full((B, 8), -1)
        at = 0
        for b in range(B):
            table[b, :held[b]] = pages[at:at + held[b]]
            at += held[b]
        free = pages[at:at + int(rng.integers(0, 30))]
        slots, cu, lens, left, after = ref.plan(ctx, new, table, free, len(free), ps, int(new.sum()))
        used = slots[slots >= 0]
        assert len(set(used.tolist())) == len(used)  # no slot twice
        taken = [int(x) for b in range(B) if lens[b] for x in after[b, held[b]:-(-int(lens[b]) // ps)]]
        assert sorted(taken) == sorted(int(x) for x in free[left:])
        for b in range(B):
            assert int(lens[b]) in (0, int(ctx[b] + new[b]))
