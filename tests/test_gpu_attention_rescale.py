"""GPU tests of attention_prompt where the running maximum moves again and again: both head sizes (which keep the weights in
different places), even and odd groups."""
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


def rescales(q, k, scale=None):
    """How often each row [T, Hq] of one sequence takes a new maximum behind its first 128 keys: a tile of 128 keys whose
    weights against the maximum so far, less 7, add up to more than 2^15 (base 2)."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    f = (D ** -0.5 if scale is None else scale) / math.log(2)
    late = torch.arange(T, device=q.device)[None] > torch.arange(T, device=q.device)[:, None]
    out = torch.zeros((T, Hq), dtype=torch.int32, device=q.device)
    for h in range(Hq):
        s = (q[:, h].double() @ k[:, h // G].double().T * f).masked_fill(late, -math.inf)
        m = s[:, :128].amax(-1) - 7
        for a in range(128, T, 128):
            t = s[:, a:a + 128]
            more = torch.exp2(t - m[:, None]).sum(-1) > 2 ** 15
            out[:, h] += more
            m = torch.where(more, torch.maximum(m, t.amax(-1) - 7), m)
    return out


def rising(T, Hq, Hkv, D, per_tile, seed):
    """Scores that rise by about per_tile (natural logarithm) from one tile of 128 keys to the next, with noise."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((T, Hq, D), generator=g)
    k = torch.randn((T, Hkv, D), generator=g)
    v = torch.randn((T, Hkv, D), generator=g)
    q[..., 0] = 8.0
    k[..., 0] = torch.arange(T)[:, None] * (per_tile / 128 * D ** 0.5 / 8)
    return [x.half().cuda() for x in (q, k, v)]


@pytest.mark.parametrize("per_tile", [5.0, 7.0, 30.0])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 1), (1, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_take_a_new_maximum_in_every_step(wql, D, Hq, Hkv, per_tile):
    T = 800
    q, k, v = rising(T, Hq, Hkv, D, per_tile, D + Hq)
    n = rescales(q, k)
    assert int(n[640:].min()) >= 3 and int(n.max()) >= 5  # by the input, not by the kernel
    y = wql.attention_prompt(q, k, v, i32([0, T]))
    wql.device_status()
    o, bound = ref.prompt(q, k, v, [0, T])
    within(y, o, bound)
    # what came before is in the sums: a rise of 5 per tile leaves e^-5 = 6.7e-3 of it, more than 2^-11 each for the output,
    # the weights and the scores (128 products of size 1 and one of up to 35 in fp32: below 1e-4 of a weight)
    err = (y.double() - o).norm(dim=-1) / o.norm(dim=-1)
    assert float(err.max()) < 3 * 2.0 ** -11


@pytest.mark.parametrize("D", [64, 128])
def test_only_some_rows_of_a_tile_take_a_new_maximum(wql, D):
    # every 37th row's scores rise, the others' fall: their neighbours' accumulators are multiplied by one
    T, Hq, Hkv = 900, 4, 2
    q, k, v = rising(T, Hq, Hkv, D, 9.0, 3)
    pick = torch.arange(T, device="cuda") % 37 == 5
    q[..., 0] = torch.where(pick[:, None], 8.0, -8.0).half()
    n = rescales(q, k)
    assert int(n[640:][pick[640:]].min()) >= 3 and not n[~pick].any()
    y = wql.attention_prompt(q, k, v, i32([0, T]))
    wql.device_status()
    o, bound = ref.prompt(q, k, v, [0, T])
    within(y, o, bound)
    # the others give the same bits without them
    q2 = q.clone()
    q2[pick, :, 0] = -8.0
    z = wql.attention_prompt(q2, k, v, i32([0, T]))
    assert torch.equal(y[~pick].view(torch.int16), z[~pick].view(torch.int16))


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (3, 3, 128), (4, 1, 64), (3, 3, 64)])
def test_scores_that_grow_by_thousands(wql, Hq, Hkv, D):
    T, n = 700, 300
    g = torch.Generator().manual_seed(11)
    q, k, v = (torch.randn((T, h, D), generator=g).half().cuda() for h in (Hq, Hkv, Hkv))
    q[n:] *= 64
    k[n:] *= torch.linspace(1, 64, T - n, device="cuda").half()[:, None, None]
    v[n:] *= -100
    assert bool((rescales(q, k)[n + 128:] > 0).any())
    y = wql.attention_prompt(q, k, v, i32([0, T]))
    wql.device_status()
    o, bound = ref.prompt(q, k, v, [0, T])
    within(y, o, bound)


@pytest.mark.parametrize("D", [64, 128])
def test_new_maxima_over_several_pairs_of_a_block(wql, D):
    # enough rows that every block takes several pairs of tiles, each with maxima that move
    lens, Hq, Hkv = [1500, 900, 1300, 40, 1700], 16, 4
    parts = [rising(n, Hq, Hkv, D, 6.0 + i, i) for i, n in enumerate(lens)]
    q, k, v = (torch.cat(x) for x in zip(*parts))
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    y = wql.attention_prompt(q, k, v, i32(cu))
    wql.device_status()
    o, bound = ref.prompt(q, k, v, cu)
    within(y, o, bound)
    for a, e in zip(cu[:-1], cu[1:]):
        alone = wql.attention_prompt(q[a:e], k[a:e], v[a:e], i32([0, e - a]))
        assert torch.equal(y[a:e].view(torch.int16), alone.view(torch.int16))
