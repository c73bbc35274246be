"""GPU test of eviction at the most tokens that a head may keep: indexes behind them pass 2^31."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


def test_places_behind_nearly_2_31_kept_tokens(wql):
    # all pages of the table are page 0 and all new ones page 1, which then holds some of its rows: the numbers are what is looked at
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB")
    ps, width = 16, 2 ** 27 - 1
    cap = ps * width  # 2^31 - 16
    n = cap - 5
    cache = wql.kv_cache_i4(2, 1, 64, ps)
    cache.fill_(1)
    table = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    new_table = torch.ones((1, width), dtype=torch.int32, device="cuda")
    w = torch.rand((1, 1, cap), device="cuda")
    kept = torch.full((cap + 64,), 7, dtype=torch.int32, device="cuda")
    nw = torch.full((cap + 64,), 7.0, device="cuda")
    new_lens = torch.zeros((1,), dtype=torch.int32, device="cuda")
    wql.kv_evict_i4(w, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), new_table, cap, 3,
                    kept=kept[32:32 + cap].view(1, 1, cap), new_weights=nw[32:32 + cap].view(1, 1, cap), new_lens=new_lens)
    wql.device_status()
    assert new_lens.tolist() == [n]
    for a in range(0, n, 1 << 28):
        e = min(a + (1 << 28), n)
        assert torch.equal(kept[32 + a:32 + e], torch.arange(a, e, dtype=torch.int32, device="cuda"))
        assert torch.equal(nw[32 + a:32 + e], w[0, 0, a:e])
    assert kept[32 + n:32 + cap].tolist() == [-1] * 5 and nw[32 + n:32 + cap].tolist() == [0.0] * 5
    for x, left in ((kept, 7), (nw, 7.0)):
        assert bool((x[:32] == left).all()) and bool((x[32 + cap:] == left).all())
    assert torch.equal(cache[0], torch.ones_like(cache[0]))
