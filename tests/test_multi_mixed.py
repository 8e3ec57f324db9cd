"""Batches of requests with one query and with many: max_query_len lets pa_decode_tree and pa_decode_cross run each as it
needs, and changes no result."""
import ctypes

import numpy as np
import pytest
import torch

import multi_gpu_ref
import multi_ref
from multi_ref import Batch

FAKE = 0x10000


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


# ------------------------------------------------------------- on the CPU ---

def test_negative_bounds_are_refused_on_the_host(pa):
    args = pa._DecodeArgs(2, 512, 8, 1, 0, 64, FAKE, 1 << 40, max_query_len=-1)
    assert pa._lib.pa_decode_cross(*[FAKE] * 7, 8, 2, 128, 16, 0.1, 5, ctypes.byref(args)) == -1
    assert pa._lib.pa_decode_tree(*[FAKE] * 7, None, 8, 2, 128, 16, 0.1, 5, 0, ctypes.byref(args)) == -1
    assert b"max_query_len" in pa._lib.pa_last_error_string()


# ------------------------------------------------------------- on the GPU ---

def close(b, got, scale):
    out, spread, size, _ = multi_gpu_ref.batch(b, scale)
    bound = (multi_gpu_ref.bf16_bound if b.dtype == torch.bfloat16 else multi_gpu_ref.f32_bound)(
        out, spread, size, max(b.lens), b.q.shape[2])
    assert ((got[:len(out)].double() - out).abs() <= bound).all()
    assert (got[len(out):] == 7).all()


def mixed(kind, Hq, Hkv, hd, dtype, seed, padding=0):
    rng = np.random.default_rng(seed)
    news = rng.integers(0, 3, 40).tolist() + [300, 7, 130, 1]
    lens = (np.array(news) + rng.integers(0, 200, 44)).tolist()
    lens[-4], lens[3] = 900, 700
    return wide(Batch(kind, lens, news, Hq, Hkv, hd, 16, dtype, seed, padding=padding))


# Tables with room for this many tokens, and a bound on the lengths to match: which kernels run goes by those.
ROOM = 2 ** 17


def wide(b):
    rest = np.random.default_rng(1).choice([-1, 2**31 - 1], size=(len(b.tables), ROOM // b.bs - b.tables.shape[1]))
    b.tables = np.concatenate([b.tables, rest.astype(np.int32)], axis=1)
    return b


@pytest.mark.gpu
@pytest.mark.parametrize("kind", multi_ref.KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,hd", [(2, 2, 128), (2, 2, 64), (8, 1, 64), (40, 1, 128)])
def test_short_and_long_ones_together(pa, kind, dtype, Hq, Hkv, hd):
    """Bounds that hold, one that does not, and none; rows behind the last sequence are left."""
    b = mixed(kind, Hq, Hkv, hd, dtype, 3, padding=500)
    for bound in (300, 301, 2**31 - 1, 20, 1, 0):
        got, flags = b.on_gpu(pa, hd ** -0.5, max_query_len=bound, max_context_len=ROOM)
        assert flags == 0
        close(b, got, hd ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bad_device_data_is_flagged_in_both_passes(pa, dtype):
    for i in (-4, 3):      # the long sequence, and one of few rows
        b = mixed("chain", 2, 2, 64, dtype, 5)
        used = {int(x) for j, n in enumerate(b.lens) for x in b.tables[j, :-(-n // 16)]}
        spare = min(set(range(b.k.shape[0])) - used)
        b.tables[i, 1] = 10**6
        got, flags = b.on_gpu(pa, 0.1, max_query_len=300, max_context_len=ROOM)
        assert flags == pa.STATUS_BAD_BLOCK_ID
        b.v[spare], b.k[spare] = 0.0, 0.0       # a bad block reads as zeros
        b.tables[i, 1] = spare
        close(b, got, 0.1)
        b.news[i], b.lens[i] = b.news[i] or 1, 0
        b.start = np.concatenate([[0], np.cumsum(b.news)]).astype(np.int32)
        b.q = torch.randn(int(b.start[-1]), *b.q.shape[1:]).to(dtype)
        got, flags = b.on_gpu(pa, 0.1, max_query_len=300, max_context_len=ROOM)
        assert flags == pa.STATUS_BAD_CONTEXT_LEN
        assert (got[int(b.start[i % 44]):int(b.start[i % 44 + 1])] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hd", [64, 128])
def test_a_step_kept_while_its_rows_change(pa, dtype, hd):
    """q as long as it ever gets, one step, captured once and replayed: query_start, lengths and q are rewritten in
    between, from a batch of single tokens to one that holds a long chunk.  In turn with another step on its workspace."""
    from paged_kv_cache_237_gb300.engine import CrossDecodeStep, TreeDecodeStep
    b = wide(Batch("chain", [600] * 6, [1] * 6, 4, 2, hd, 16, dtype, 8, padding=394))
    cap = b.q.shape[0]
    q, lens = b.q.cuda(), torch.tensor(b.lens, dtype=torch.int32).cuda()
    start = torch.from_numpy(b.start).cuda()
    caches = b.k.cuda(), b.v.cuda(), torch.from_numpy(b.tables).cuda()
    step = TreeDecodeStep(q, *caches, lens, start, 0.1, ROOM, max_query_len=390)
    other = CrossDecodeStep(q[:6].contiguous(), *caches, lens, torch.arange(7, dtype=torch.int32).cuda(), 0.1, ROOM,
                            workspace=step.workspace)
    step.decode()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.decode()
        other.decode()
    for news in ([1] * 6, [1, 1, 390, 1, 0, 1], [5, 0, 130, 0, 130, 2], [0] * 6, [2, 390, 0, 0, 0, 2]):
        b.news, b.start = news, np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        b.q = torch.randn(cap, 4, hd).to(dtype)
        b.lens = [max(c, 40 * i + 7) for i, c in enumerate(news)]
        q.copy_(b.q)
        start.copy_(torch.from_numpy(b.start))
        lens.copy_(torch.tensor(b.lens, dtype=torch.int32))
        first = None
        for _ in range(3):
            step.out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            close(b, step.out, 0.1)
            first = step.out.clone() if first is None else first
            assert torch.equal(step.out, first)
    assert step.status.read() == 0
    step.max_query_len = 0
    step.out.fill_(7.0)
    close(b, step.decode(), 0.1)
