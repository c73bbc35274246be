"""GPU tests of attention over chunks whose inputs were written by the kernels right in front of it: queries, cache, table, starts and
lengths change from call to call without a wait, in batches that have chunks of many rows and of a few."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import _chunks_ref as cref  # noqa: E402


@pytest.fixture(scope="module")
def wql(wql_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return wql_lib


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# (tokens, new ones) of variants of a batch with as many rows and pages: chunks among single and drafted tokens
SHAPES = [[([900, 33, 400, 700, 50, 1], [1, 1, 60, 4, 2, 1]), ([300, 500, 64, 9, 1000, 210], [60, 2, 1, 1, 4, 1]), ([70, 800, 0, 65, 640, 508], [1, 4, 1, 2, 1, 60])],
          [([3000, 40], [1, 3]), ([20, 3020], [2, 2]), ([1500, 1540], [3, 1])]]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 4, 4)])
@pytest.mark.parametrize("shapes", SHAPES)
def test_inputs_written_right_before_the_call(wql, shapes, D, Hq, Hkv, captured):
    ps, made = 16, []
    for seed, (lens, new) in enumerate(shapes):
        q, cache, table, cu = cref.case(lens, new, Hq, Hkv, D, ps, seed + 1)
        made.append([q, cache, table, i32(cu), i32(lens)])
    pages, width = max(m[1].shape[0] for m in made), max(m[2].shape[1] for m in made)
    for m in made:
        m[1] = torch.cat([m[1], torch.zeros((pages - m[1].shape[0],) + m[1].shape[1:], dtype=torch.uint8, device="cuda")])
        m[2] = torch.cat([m[2], torch.full((len(m[2]), width - m[2].shape[1]), -1, dtype=torch.int32, device="cuda")], 1)
    T = made[0][0].shape[0]
    assert all(m[0].shape[0] == T for m in made)
    ws = torch.empty((wql.attention_chunks_kv_i4_workspace_bytes(T, len(made[0][4]), Hq, Hkv, D),), dtype=torch.uint8, device="cuda")

    def call(m, out, lse):
        wql.attention_chunks_kv_i4(*m, out=out, lse=lse, workspace=ws)

    want = []
    for m, (lens, new) in zip(made, shapes):
        out, lse = torch.zeros((T, Hq, D), dtype=torch.float16, device="cuda"), torch.zeros((T, Hq), device="cuda")
        call(m, out, lse)
        torch.cuda.synchronize()
        o, ob, z, zb = cref.chunks(*m[:3], m[3].tolist(), lens)
        assert bool(((out.double() - o).abs() <= ob).all()) and bool((((lse.double() - z).abs() <= zb) | (lse.double() == z)).all())
        want.append((out, lse))
    live = [torch.zeros_like(x) for x in made[0]]
    out, lse = torch.zeros_like(want[0][0]), torch.zeros_like(want[0][1])
    graphs = []
    if captured:
        for m in made:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                for x, y in zip(live, m):
                    x.copy_(y)
                call(live, out, lse)
            graphs.append(g)
    got = []
    for i in range(120):
        k = (i * i + i // 7) % len(made)
        if captured:
            graphs[k].replay()
        else:
            order = range(5) if i % 2 else reversed(range(5))  # another one is written last
            for j in order:
                live[j].copy_(made[k][j])
            call(live, out, lse)
        got.append((k, out.clone(), lse.clone()))
    for k, y, z in got:
        assert torch.equal(y.view(torch.int16), want[k][0].view(torch.int16)) and torch.equal(z.view(torch.int32), want[k][1].view(torch.int32))
    wql.device_status()
