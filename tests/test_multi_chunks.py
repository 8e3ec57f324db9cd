"""Long chains in pa_decode_tree: a prompt's chunk, whose queries see what the cache holds before it and, of the chunk,
themselves and what lies before them."""
import numpy as np
import pytest
import torch

import multi_gpu_ref
from multi_ref import Batch

INF = float("inf")


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


def against(b, scale):
    out, spread, size, _ = multi_gpu_ref.batch(b, scale)
    return out, (multi_gpu_ref.bf16_bound if b.dtype == torch.bfloat16 else multi_gpu_ref.f32_bound)(
        out, spread, size, max(b.lens), b.q.shape[2])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,hd", [(2, 2, 128), (2, 2, 64), (8, 1, 128), (5, 1, 64), (80, 2, 128)])
def test_chunks_with_and_without_a_prefix(pa, dtype, Hq, Hkv, hd):
    """Row blocks that begin inside a query's heads, chunks that end inside a tile, and a chunk that is the whole sequence."""
    news = [2000, 1001, 130, 7] if Hq < 80 else [250, 41, 130, 7]
    lens = [2000, 1001 + 777, 130 + 64, 7 + 1]
    b = Batch("chain", lens, news, Hq, Hkv, hd, 16, dtype, hd + Hq, padding=2)
    out, bound = against(b, hd ** -0.5)
    got, flags = b.on_gpu(pa, hd ** -0.5)
    assert flags == 0
    assert ((got[:len(out)].double() - out).abs() <= bound).all() and (got[len(out):] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,most", [(2, 2, 900), (8, 1, 900), (4, 4, 12)])
def test_values_that_are_not_finite_reach_the_rows_behind_them(pa, dtype, Hq, Hkv, most):
    """At the borders of row blocks and tiles, in the context and in the chunk."""
    n = 900 + 130
    for at in (0, 129, 130, 131, 257, 258, 386, 640, 1028, 1029):
        b = Batch("chain", [n, 300], [most, min(most, 300)], Hq, Hkv, 64, 16, dtype, 7)
        clean, bound = against(b, 0.125)
        place = int(b.tables[0, at // 16]), slice(None), at % 16
        b.v[place][..., 3], b.v[place][..., 9] = -INF, float("nan")
        got = b.on_gpu(pa, 0.125)[0].double()
        hit = torch.zeros_like(clean, dtype=torch.bool)
        hit[max(0, at - (n - most)):most, :, 3] = True
        assert (got[hit] == -INF).all()
        hit[..., 9] = hit[..., 3]
        assert got[..., 9][hit[..., 9]].isnan().all()
        assert ((got - clean).abs() <= bound)[~hit].all()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(16, 16), (32, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_infinity_does_not_cost_more_than_the_chunk(pa, Hq, Hkv, dtype):
    """Rows are mended at the end of their item, of the tokens that some of them do not see (fp32: of the tiles that hold such
    values): not of the whole chunk."""
    b = Batch("chain", [4000], [4000], Hq, Hkv, 128, 16, dtype, 1)
    args = [torch.empty_like(b.q).cuda(), b.q.cuda(), b.k.cuda(), b.v.cuda(), torch.from_numpy(b.tables).cuda(),
            torch.tensor(b.lens, dtype=torch.int32).cuda(), torch.from_numpy(b.start).cuda(), 0.1]
    ws = torch.empty(pa.pa_decode_tree_workspace_size(4000, Hq, Hkv, 128), dtype=torch.uint8, device="cuda")

    def best():
        times = []
        for _ in range(6):
            a, z = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            pa.pa_decode_tree(*args, max_context_len=4000, workspace=ws)
            z.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(z))
        return min(times)

    plain = best()
    args[3][int(b.tables[0, 9]), :, 3, 1] = INF
    assert best() < 10 * plain
