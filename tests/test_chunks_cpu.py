"""CPU tests of attention over chunks, of attention weights and of eviction: what the C ABI and the binding refuse (before
anything touches a device), and the 64-bit restatements that the GPU tests compare against, pinned to direct sums."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import _attn_ref as ref  # noqa: E402
import _chunks_ref as cref  # noqa: E402

OK, EINVAL, EUNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p(1 << 20)      # never read: validation comes first
ODD = ctypes.c_void_p((1 << 20) + 2)
ODD4 = ctypes.c_void_p((1 << 20) + 4)
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib(wql_lib):
    return wql_lib.load()


def chunks(lib, T=8, Hq=4, Hkv=2, D=128, qs=512, pages=3, ps=16, width=4, B=2, scale=0.1, q=P, cache=P, table=P, cu=P, lens=P,
           out=P, lse=P, ws=P, n=1 << 40):
    return lib.wql_attention_chunks_kv_i4(q, qs, T, Hq, Hkv, D, cache, pages, ps, table, width, cu, lens, B, F(scale), out, lse,
                                          ws, n, None)


def weights(lib, T=8, Hq=4, Hkv=2, D=128, qs=512, pages=3, ps=16, width=4, B=2, scale=0.1, q=P, cache=P, table=P, cu=P, lens=P,
            lse=P, w=P, ws=P, n=1 << 40):
    return lib.wql_kv_weights_i4(q, qs, T, Hq, Hkv, D, cache, pages, ps, table, width, cu, lens, B, F(scale), lse, w, ws, n,
                                 None)


def evict(lib, w=P, cache=P, pages=3, ps=16, H=2, D=128, table=P, width=4, lens=P, B=2, new=P, new_width=2, budget=20, recent=4,
          kept=P, nw=P, nl=P):
    return lib.wql_kv_evict_i4(w, cache, pages, ps, H, D, table, width, lens, B, new, new_width, budget, recent, kept, nw, nl,
                               None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(Hq=5), EINVAL, b"multiple"), (dict(Hkv=0), EINVAL, b"multiple"), (dict(Hq=1), EINVAL, b"multiple"),
    (dict(T=-1), EINVAL, b"T"), (dict(B=-1), EINVAL, b"B"), (dict(B=4097), EUNSUPPORTED, b"4096"),
    (dict(D=96), EUNSUPPORTED, b"64 or 128"), (dict(ps=24), EINVAL, b"page_size"), (dict(ps=0), EINVAL, b"page_size"),
    (dict(pages=0), EINVAL, b"pages"), (dict(pages=1 << 28), EINVAL, b"2^31"), (dict(width=0), EINVAL, b"table_width"),
    (dict(width=1 << 27, ps=16), EINVAL, b"2^31"), (dict(Hq=258, Hkv=2, qs=258 * 128), EUNSUPPORTED, b"128"),
    (dict(T=1 << 30), EUNSUPPORTED, b"2^31"), (dict(Hq=65536, Hkv=65536, qs=65536 * 128), EUNSUPPORTED, b"65535"), (dict(scale=math.nan), EINVAL, b"scale"),
    (dict(scale=-math.inf), EINVAL, b"scale"), (dict(scale=2.0 ** 65), EINVAL, b"scale"), (dict(qs=511), EINVAL, b"stride"),
    (dict(qs=516), EINVAL, b"stride"), (dict(q=None), EINVAL, b"q"), (dict(q=ODD4), EINVAL, b"q"),
    (dict(cache=ODD4), EINVAL, b"cache"), (dict(table=ODD), EINVAL, b"block_table"), (dict(cu=None), EINVAL, b"cu_new"),
    (dict(lens=ODD), EINVAL, b"kv_lens")])
@pytest.mark.parametrize("call", [chunks, weights])
def test_refusals_of_both(lib, call, kw, status, word):
    assert call(lib, **kw) == status
    assert word in lib.wql_last_error()


def test_own_refusals(lib):
    assert chunks(lib, out=None) == EINVAL and chunks(lib, out=ODD4) == EINVAL and chunks(lib, lse=ODD) == EINVAL
    assert chunks(lib, ws=None) == EINVAL and chunks(lib, ws=ODD4) == EINVAL
    assert chunks(lib, n=8) == EINVAL and b"workspace" in lib.wql_last_error()
    for kw in (dict(T=0), dict(B=0)):
        assert chunks(lib, q=None, cache=None, table=None, cu=None, lens=None, out=None, lse=None, ws=None, n=0, **kw) == OK
        assert weights(lib, q=None, cache=None, table=None, cu=None, lens=None, lse=None, w=None, ws=None, n=0, **kw) == OK
    f = lib.wql_attention_chunks_kv_i4_workspace_bytes
    assert f(8, 2, 4, 2, 128) > 0
    assert f(8, 2, 5, 2, 128) == f(0, 2, 4, 2, 128) == f(8, 0, 4, 2, 128) == f(8, 2, 4, 2, 80) == f(8, 2, 258, 2, 64) == 0
    assert weights(lib, lse=None) == EINVAL and weights(lib, lse=ODD) == EINVAL
    assert weights(lib, w=None) == EINVAL and weights(lib, w=ODD4) == EINVAL
    assert weights(lib, ws=None) == EINVAL and weights(lib, ws=ODD4) == EINVAL
    assert weights(lib, n=8) == EINVAL and b"workspace" in lib.wql_last_error()
    assert lib.wql_kv_weights_i4_workspace_bytes() > 0


@pytest.mark.parametrize("kw,status,word", [
    (dict(B=-1), EINVAL, b"B"), (dict(H=0), EINVAL, b"H"), (dict(B=4097), EUNSUPPORTED, b"4096"), (dict(D=80), EUNSUPPORTED, b"64 or 128"),
    (dict(ps=8), EINVAL, b"page_size"), (dict(pages=0), EINVAL, b"pages"), (dict(width=0), EINVAL, b"table_width"),
    (dict(new_width=0), EINVAL, b"new_width"), (dict(new_width=1 << 27), EINVAL, b"new_width"), (dict(budget=0), EINVAL, b"budget"),
    (dict(budget=33), EINVAL, b"budget"), (dict(recent=-1), EINVAL, b"recent"),
    (dict(B=4096, H=1024, budget=16 * 1024, new_width=1024), EUNSUPPORTED, b"2^31"), (dict(w=None), EINVAL, b"weights"),
    (dict(w=ODD4), EINVAL, b"weights"), (dict(cache=ODD), EINVAL, b"cache"), (dict(table=None), EINVAL, b"block_table"),
    (dict(lens=ODD), EINVAL, b"kv_lens"), (dict(new=ODD), EINVAL, b"new_table"), (dict(kept=None), EINVAL, b"kept"),
    (dict(nw=ODD4), EINVAL, b"new_weights"), (dict(nl=None), EINVAL, b"new_lens")])
def test_evict_refusals(lib, kw, status, word):
    assert evict(lib, **kw) == status
    assert word in lib.wql_last_error()


def test_evict_empty(lib):
    assert evict(lib, B=0, w=None, cache=None, table=None, lens=None, new=None, kept=None, nw=None, nl=None) == OK


def test_binding_refuses_before_any_launch(wql_lib):
    w = wql_lib
    z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)  # noqa: E731
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    f = lambda *s: torch.zeros(s, dtype=torch.float32)  # noqa: E731
    cache = z(2, 2, 1, 16 * 136, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        w.attention_chunks_kv_i4(h(5, 4, 128), cache, z(2, 1), z(3), z(2))
    with pytest.raises(ValueError, match="CUDA"):
        w.kv_weights_i4(h(5, 4, 128), cache, z(2, 1), z(3), z(2), f(5, 4), f(2, 2, 16))
    with pytest.raises(ValueError, match="CUDA"):
        w.kv_evict_i4(f(2, 2, 16), cache, z(2, 1), z(2), z(2, 1), 8)
    with pytest.raises(ValueError, match="kv_cache_i4"):
        w.kv_evict_i4(f(2, 2, 16), z(2, 2, 5, dtype=torch.uint8), z(2, 1), z(2), z(2, 1), 8)
    with pytest.raises(TypeError):
        w.attention_chunks_kv_i4(h(5, 4, 128), None, z(2, 1), z(3), z(2))


# ---- the restatements --------------------------------------------------------------------------

def test_restatements_against_direct_sums():
    lens, new = [37, 3, 0, 20], [5, 4, 2, 20]  # rows that see nothing, a refused request, a whole prompt
    q, cache, table, cu = cref.case(lens, new, 6, 2, 64, 16, 1, pad=2, device="cpu")
    o, ob, lse, lb = cref.chunks(q, cache, table, cu, lens)
    before = torch.rand((4, 2, table.shape[1] * 16))
    lse32 = torch.nan_to_num(lse, nan=0.0).float()
    w, wb = cref.weights(q, cache, table, cu, lens, lse32, before)
    want = before.double().clone()
    for b in range(4):
        for r in range(new[b]):
            n = lens[b] - new[b] + r + 1  # tokens that it sees
            for h in range(6):
                got, z = o[cu[b] + r, h], lse[cu[b] + r, h]
                if n <= 0:
                    assert not got.any() and z == -math.inf
                    continue
                t = torch.arange(n)
                k, v = (x[:, h // 3].double() for x in ref.read(cache, table[b].long()[t // 16] * 16 + t % 16))
                e = [math.exp(float(q[cu[b] + r, h].double() @ x) / 8) for x in k]
                mean = sum(x * y for x, y in zip(e, v)) / sum(e)
                assert float((got - mean).abs().max()) < 1e-9 and abs(float(z) - math.log(sum(e))) < 1e-9
                for j, x in enumerate(e):
                    want[b, h // 3, j] += x * math.exp(-float(lse32[cu[b] + r, h]))
    assert float((w - want).abs().max()) < 1e-9
    assert bool((ob[:cu[-1]] < 0.02).all()) and bool((lb[:cu[-1]] < 1e-3).all()) and bool((wb < 1e-3 * (1 + want)).all())
    assert bool(torch.isnan(o[cu[-1]:]).all())


def test_values_are_those_that_kv_read_gives_but_finite():
    cache = torch.zeros((2, 1, 1, 16 * 72), dtype=torch.uint8)
    k = torch.randn((3, 1, 64)).half()
    v = torch.zeros((3, 1, 64)).half()
    k[1, 0, 5] = math.nan
    v[2, 0, 7] = 65504.0  # s is rounded up: 15 s is beyond fp16
    ref.write(cache, torch.arange(3), k, v)
    kk, vv = cref.values(cache, torch.tensor([0]), 3, 16)
    a, b = ref.read(cache, torch.arange(3))
    assert bool(torch.isnan(kk[1]).all()) and torch.equal(kk[[0, 2]], a[[0, 2]].double())
    assert torch.isinf(b[2, 0, 7]) and vv[2, 0, 7] == 65504.0


def test_evict_restatement_by_hand():
    w = torch.tensor([[[3.0, 1.0, math.nan, 1.0, 0.0, 1.0, 9.0]]])
    assert cref.evict(w, [7], 4, 1) == [[[0, 1, 2, 6]]]
    assert cref.evict(w, [7], 5, 0) == [[[0, 1, 2, 3, 6]]]
    assert cref.evict(w, [6], 2, 5) == [[[4, 5]]]
    assert cref.evict(w, [3], 8, 1) == [[[0, 1, 2]]] and cref.evict(w, [0], 8, 1) == [[[]]]
    assert cref.evict(torch.tensor([[[-0.0, 0.0, -1.0]]]), [3], 1, 0) == [[[0]]]


def test_eviction_into_its_own_tensors_is_refused(lib):
    A = [ctypes.c_void_p((1 << 20) + 4096 * i) for i in range(1, 9)]
    kw = dict(w=A[0], cache=A[1], table=A[2], lens=A[3], new=A[4], kept=A[5], nw=A[6], nl=A[7])
    for own, other in (("new", "table"), ("nw", "w"), ("nl", "lens")):
        assert evict(lib, **dict(kw, **{own: kw[other]})) == EINVAL
        assert b"must not be" in lib.wql_last_error()
