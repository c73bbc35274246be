"""GPU tests of attention_prompt with more than 128 sequences, which it takes in their order, 32 at a time: empty, short and
long ones, several tiles and pairs per block, one that is invalid among them."""
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


def lengths(B, seed, empty_chunk):
    g = torch.Generator().manual_seed(seed)
    kind = torch.randint(0, 4, (B,), generator=g).tolist()
    n = [0 if k == 0 else int(torch.randint(1, 41, (1,), generator=g)) if k < 3 else int(torch.randint(130, 701, (1,), generator=g))
         for k in kind]
    if empty_chunk:
        n[32:64] = [0] * 32
    return n


@pytest.mark.parametrize("B,Hq,Hkv,D,empty_chunk", [(140, 8, 4, 128, False), (140, 5, 5, 128, True), (161, 6, 2, 64, False),
                                                    (200, 8, 1, 64, True), (129, 7, 1, 128, False)])
def test_many_sequences_of_mixed_length(wql, B, Hq, Hkv, D, empty_chunk):
    lens = lengths(B, B + Hq, empty_chunk)
    T = sum(lens) + 9
    g = torch.Generator().manual_seed(B)
    q, k, v = (torch.randn((T, h, D), generator=g).half().cuda() for h in (Hq, Hkv, Hkv))
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    # more pairs of tiles than two rounds of blocks take
    rows = 128 if (Hq // Hkv) % 2 == 0 else 256
    pairs = sum(-(-n // rows) for n in lens) * (Hq // 2 if rows == 128 else Hq)
    assert pairs > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    out = torch.full(q.shape, 3.0, dtype=torch.float16, device="cuda")
    wql.attention_prompt(q, k, v, i32(cu), out=out)
    wql.device_status()
    o, bound = ref.prompt(q, k, v, cu)
    within(out[:T - 9], o[:T - 9], bound[:T - 9])
    assert bool((out[T - 9:] == 3.0).all())
    # the same bits as in calls of up to 128 sequences, which sort them
    for a in range(0, B, 100):
        part = cu[a:a + 101]
        z = wql.attention_prompt(q, k, v, i32(part))
        assert torch.equal(out[part[0]:part[-1]].view(torch.int16), z[part[0]:part[-1]].view(torch.int16))


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 4, 128), (5, 5, 64)])
def test_an_invalid_sequence_in_a_later_chunk_is_left_out(wql, Hq, Hkv, D):
    B = 150
    lens = lengths(B, 7, False)
    lens[99], lens[100] = 300, 200
    T = sum(lens)
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn((T, h, D), generator=g).half().cuda() for h in (Hq, Hkv, Hkv))
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    good = wql.attention_prompt(q, k, v, i32(cu))
    wql.device_status()
    bad = list(cu)
    bad[100] = T + 5  # sequence 99 ends behind the rows, 100 before it begins
    out = torch.full(q.shape, 3.0, dtype=torch.float16, device="cuda")
    wql.attention_prompt(q, k, v, i32(bad), out=out)
    with pytest.raises(wql.WQLError) as e:
        wql.device_status()
    assert e.value.status == 1
    wql.device_status()
    assert torch.equal(out[:cu[99]], good[:cu[99]]) and torch.equal(out[cu[101]:], good[cu[101]:])
    assert bool((out[cu[99]:cu[101]] == 3.0).all())
