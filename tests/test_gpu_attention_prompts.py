"""GPU tests of causal attention over packed prompts where keys are infinite: what has the weight zero counts for nothing,
wherever it stands."""
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


def packed(lens, Hq, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((sum(lens), Hq + 2 * Hkv, D), generator=g)
    qkv[:, :Hq] *= 0.5 + 2 * torch.rand((1, Hq, 1), generator=g)
    qkv = qkv.half().cuda()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], cu


@pytest.mark.parametrize("first", [1, 127, 128, 129, 200, 300])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (3, 1, 128), (4, 2, 64), (1, 1, 64)])
def test_keys_of_score_minus_infinity_count_for_nothing(wql, Hq, Hkv, D, first):
    # the first keys of the second sequence: a row that sees others too is what it would be without them, in the 64-bit
    # definition; one that sees no others has no softmax (NaN)
    lens = [40, 450, 30]
    q, k, v, cu = packed(lens, Hq, Hkv, D, first)
    q, k = q.clone(), k.clone()
    q[..., 3] = q[..., 3].abs() + 0.1
    k[40:40 + first, :, 3] = -math.inf
    y = wql.attention_prompt(q, k, v, i32(cu))
    wql.device_status()
    assert torch.isnan(y[40:40 + first]).all()
    o, bound = ref.prompt(q, k, v, [0, 40])
    within(y[:40], o[:40], bound[:40])
    o, bound = ref.prompt(q, k, v, [40 + first, 490, 520])
    within(y[40 + first:], o[40 + first:], bound[40 + first:])


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (3, 1, 64)])
def test_keys_of_score_minus_infinity_with_low_scores_behind(wql, Hq, Hkv, D):
    # scores of -300 and less behind them must not vanish against a maximum that nothing has set
    q, k, v, cu = packed([400], Hq, Hkv, D, 2)
    q, k = q.clone(), k.clone()
    q[..., 3], q[..., 5] = 8.0, 16.0
    k[:150, :, 3] = -math.inf
    k[150:, :, 5] = torch.linspace(-200, -150, 250, device="cuda").half()[:, None]
    y = wql.attention_prompt(q, k, v, i32(cu))
    wql.device_status()
    assert torch.isnan(y[:150]).all()
    o, bound = ref.prompt(q, k, v, [150, 400])
    within(y[150:], o[150:], bound[150:])
