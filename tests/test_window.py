"""pa_decode_window: decode attention with a sliding window and first tokens that
stay visible, against fp64 attention over the visible positions.  Tolerances
are the framework's own (helpers.py): fp32 1e-5, bf16 2e-3 + 1e-2 |ref|."""
import ctypes

import numpy as np
import pytest
import torch

import q4_ref
from helpers import assert_decode_close

FAKE = 0x10000


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


# ------------------------------------------------------------- on the CPU ---

@pytest.mark.parametrize("change,code", [
    (dict(window=0), -1), (dict(window=-5), -1), (dict(sinks=-1), -1), (dict(hd=96), -2), (dict(bs=8), -2),
    (dict(dtype=9), -1), (dict(P=24), -1), (dict(simt=1), -2), (dict(ctx=4096, P=512, window=600), -7),
    (dict(q=None), -1), (dict(q=FAKE + 4), -1), (dict(phase=9), -1), (dict(seqs=0), 0),
])
def test_bad_arguments_are_refused_on_the_host(pa, change, code):
    a = dict(q=FAKE, hd=128, bs=16, window=64, sinks=4, seqs=2, dtype=1, P=0, ctx=64, phase=0, simt=0)
    a.update(change)
    args = pa._DecodeArgs(a["seqs"], 512, 8, a["dtype"], a["P"], a["ctx"], None, 0, None, None, a["phase"], None,
                          None, None, a["simt"], 0)
    rc = pa._lib.pa_decode_window(FAKE, a["q"], FAKE, FAKE, FAKE, FAKE, 8, 2, a["hd"], a["bs"], 0.1, a["window"],
                                  a["sinks"], ctypes.byref(args))
    assert rc == code, pa._lib.pa_last_error_string()


def test_workspace_is_sized_by_what_is_visible(pa):
    size = lambda *a, **k: pa.pa_decode_window_workspace_size(4, 8, 2, 128, *a, **k)
    plain = lambda tokens, P: pa.pa_decode_workspace_size(4, 8, 128, tokens, P)
    assert size(10**6, 512, window=400, num_sinks=4) == 0
    assert size(10**6, 512, window=600, num_sinks=4) == plain(631, 512)
    assert size(700, 512, window=10**9, num_sinks=10**9) == plain(700, 512)
    assert size(700, 512, window=0) == 0 and size(700, 0, window=5, num_sinks=-1) == 0
    assert pa.pa_decode_window_workspace_size(4, 8, 3, 128, 700, 0, window=64) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_library_picks_equal_partitions(pa, dtype):
    """partition_size 0: few rows are cut finely, many short ones not at all, and
    the longest windows fit the largest partition."""
    size = lambda S, W: pa.pa_decode_window_workspace_size(S, 64, 8, 128, 10**6, 0, window=W, num_sinks=4, dtype=dtype)
    a256 = lambda x: (x + 255) // 256 * 256
    parts = lambda S, W: next(n for n in range(2, 10**5) if size(S, W) ==
                              256 + a256(S * n * 64 * 8) + a256(S * n * 64 * 128 * 4))
    assert parts(1, 512) >= 5
    if dtype == torch.bfloat16:
        assert size(32, 512) == 0 and size(64, 512) == 0
    assert 2 <= parts(64, 4096) <= 9
    assert parts(1, 10**6) >= 10**6 // 4096


def test_binding_and_step_refuse_bad_windows(pa):
    from paged_kv_cache_237_gb300.engine import DecodeStep
    q = torch.zeros(1, 2, 64)
    with pytest.raises(ValueError, match="window"):
        pa.pa_decode_window(q, q, q, q, q, q, 0.1, window=0, max_context_len=1)
    for kw in (dict(window=-1), dict(num_sinks=3), dict(window=4, simt=True), dict(window=4, num_sinks=-1)):
        with pytest.raises(ValueError):
            DecodeStep(q, q, q, q, q, 0.1, 1, **kw)


# ------------------------------------------------------------- on the GPU ---

def make(lens, Hq, Hkv, hd, bs, dtype, seed, window, sinks):
    """A batch whose pool holds NaN in every slot that is not visible and whose
    table entries of blocks without a visible slot are junk."""
    rng = np.random.default_rng(seed)
    per = [-(-n // bs) for n in lens]
    nb, width = sum(per) + 3, max(1, max(per))
    perm = rng.permutation(nb)
    tables = np.full((len(lens), width), -1, np.int32)
    live = np.zeros((nb, bs), bool)
    at = 0
    for i, n in enumerate(lens):
        tables[i, :per[i]] = perm[at:at + per[i]]
        at += per[i]
        for j in range(per[i]):
            t = np.arange(j * bs, j * bs + bs)
            seen = (t < n) & ((t >= n - window) | (t < sinks))
            live[tables[i, j]] = seen
            if not seen.any():
                tables[i, j] = rng.choice([-1, 2**31 - 1, nb, -2**31])
    g = torch.Generator().manual_seed(seed)
    caches = []
    for _ in range(2):
        c = torch.randn(nb, Hkv, bs, hd, generator=g).to(dtype)
        c.masked_fill_(~torch.from_numpy(live)[:, None, :, None], float("nan"))
        caches.append(c)
    q = torch.randn(len(lens), Hq, hd, generator=g).to(dtype)
    return q, *caches, tables, np.array(lens, np.int32)


def reference(case, scale, window, sinks):
    q, kc, vc, tables, lens = case
    return torch.from_numpy(q4_ref.attend(q.double().numpy(), kc.double().numpy(), vc.double().numpy(), tables, lens,
                                          scale, kc.shape[2], window, sinks))


def on_gpu(pa, case, scale, window, sinks, **kw):
    q, kc, vc, tables, lens = case
    status = pa.DeviceStatus()
    out = torch.full_like(q, float("nan")).cuda()
    pa.pa_decode_window(out, q.cuda(), kc.cuda(), vc.cuda(), torch.from_numpy(tables).cuda(),
                        torch.from_numpy(lens).cuda(), scale, window=window, num_sinks=sinks,
                        max_context_len=max(1, int(lens.max())), status=status, **kw)
    torch.cuda.synchronize()
    return out, status.read()


EDGES = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 511, 512, 513, 1025, 1500]
WINDOWS = [(1, 0), (1, 1), (5, 3), (16, 16), (17, 33), (32, 0), (33, 64), (100, 1), (512, 0), (500, 4), (3000, 4),
           (64, 2000), (2**31 - 1, 2**31 - 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("dtype,hd,bs", [(torch.bfloat16, 128, 16), (torch.bfloat16, 64, 32),
                                         (torch.float32, 128, 32), (torch.float32, 64, 16)])
def test_windows_at_edge_lengths(pa, window, sinks, dtype, hd, bs):
    for P in (0, 64):
        case = make(EDGES, 4, 2, hd, bs, dtype, 7, window, sinks)
        out, flags = on_gpu(pa, case, hd ** -0.5, window, sinks, partition_size=P)
        assert flags == 0
        assert_decode_close(out, reference(case, hd ** -0.5, window, sinks), dtype, what=f"P {P}")
        assert (out[0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 1), (9, 1), (16, 2), (40, 2), (6, 6)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_head_layouts(pa, Hq, Hkv, dtype):
    case = make([90, 700, 20], Hq, Hkv, 128, 16, dtype, Hq, 150, 5)
    out, flags = on_gpu(pa, case, 0.09, 150, 5)
    assert flags == 0
    assert_decode_close(out, reference(case, 0.09, 150, 5), dtype, what=f"{Hq}/{Hkv}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_window_that_covers_everything_is_pa_decode_bit_for_bit(pa, dtype):
    case = make([700, 33, 1200], 8, 2, 128, 16, dtype, 2, 2000, 0)
    q, kc, vc, tables, lens = case
    ref = torch.empty_like(q).cuda()
    pa.pa_decode(ref, q.cuda(), kc.cuda(), vc.cuda(), torch.from_numpy(tables).cuda(),
                 torch.from_numpy(lens).cuda(), 0.09, max_context_len=1200, partition_size=256)
    for window, sinks in ((1200, 0), (5000, 3), (1, 1200)):
        out, flags = on_gpu(pa, case, 0.09, window, sinks, partition_size=256)
        assert flags == 0 and torch.equal(out, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 4), (300, 17)])
def test_fused_write_puts_the_new_token_in_and_attends(pa, dtype, window, sinks):
    lens = [1, 16, 17, 333, 640, 33]
    case = make(lens, 8, 2, 128, 16, dtype, 3, window, sinks)
    q, kc, vc, tables, lens_a = case
    g = torch.Generator().manual_seed(8)
    kn, vn = (torch.randn(len(lens), 2, 128, generator=g).to(dtype) for _ in range(2))
    slots = np.array([tables[i, (n - 1) // 16] * 16 + (n - 1) % 16 for i, n in enumerate(lens)], np.int64)
    dk, dv, status = kc.cuda(), vc.cuda(), pa.DeviceStatus()
    out = torch.empty_like(q).cuda()
    pa.pa_decode_window(out, q.cuda(), dk, dv, torch.from_numpy(tables).cuda(), torch.from_numpy(lens_a).cuda(), 0.09,
                        window=window, num_sinks=sinks, max_context_len=640, partition_size=64, status=status,
                        k_new=kn.cuda(), v_new=vn.cuda(), slot_mapping=torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    assert status.read() == 0
    for c, n in ((kc, kn), (vc, vn)):
        c[slots // 16, :, slots % 16] = n
    assert torch.equal(torch.nan_to_num(dk.cpu()), torch.nan_to_num(kc))
    assert torch.equal(torch.nan_to_num(dv.cpu()), torch.nan_to_num(vc))
    assert_decode_close(out, reference(case, 0.09, window, sinks), dtype, what="fused")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bad_visible_blocks_are_flagged_and_hidden_ones_are_not(pa, dtype):
    case = make([500, 300], 4, 1, 128, 16, dtype, 5, 100, 4)
    q, kc, vc, tables, lens = case
    assert (tables[0] == tables[0].clip(0, kc.shape[0] - 1)).sum() < tables.shape[1]   # junk behind the window
    tables[0, 29] = kc.shape[0] + 5
    out, flags = on_gpu(pa, case, 0.09, 100, 4, partition_size=64)
    assert flags == pa.STATUS_BAD_BLOCK_ID
    assert_decode_close(out, reference(case, 0.09, 100, 4), dtype, what="bad id reads as zeros")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_steps_graphs_and_streams(pa, dtype):
    from paged_kv_cache_237_gb300.engine import DecodeStep
    case = make([900, 33, 2000, 0, 640], 16, 2, 128, 16, dtype, 11, 300, 4)
    q, kc, vc, tables, lens = case
    s = DecodeStep(q.cuda(), kc.cuda(), vc.cuda(), torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(),
                   0.09, 2000, partition_size=64, window=300, num_sinks=4)
    ref = reference(case, 0.09, 300, 4)
    first = s.decode().clone()
    assert_decode_close(first, ref, dtype)
    s.out.fill_(float("nan"))
    s.decode(phase=pa.PA_PHASE_PARTITIONS)
    assert torch.equal(s.decode(phase=pa.PA_PHASE_REDUCE), first)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        s.decode()
    s.out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s.out, first) and s.status.read() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q4", [False, True])
def test_a_bound_of_zero_tokens(pa, dtype, q4):
    """max_context_len 0: every row is empty, and any length is flagged."""
    q = torch.randn(3, 8, 128).to(dtype).cuda()
    tables = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    status = pa.DeviceStatus()
    for lens, flag in (([0, 0, 0], 0), ([0, 5, 0], pa.STATUS_BAD_CONTEXT_LEN)):
        out = torch.full_like(q, 3.0)
        ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if q4:
            c = torch.zeros(2, 2, pa.pa_q4_page_bytes(128, 16), dtype=torch.uint8, device="cuda")
            pa.pa_decode_q4(out, q, c, c, tables, ctx, 0.1, max_context_len=0, status=status, window=4)
        else:
            c = torch.zeros(2, 2, 16, 128, dtype=dtype, device="cuda")
            pa.pa_decode_window(out, q, c, c, tables, ctx, 0.1, max_context_len=0, status=status, window=4)
        assert (out == 0).all() and status.read() == flag


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_a_call_on_another_stream_makes_its_workspace_there(pa, raw):
    """No workspace given, and the current stream is busy: the zeroed workspace
    has to be made on the stream of the call."""
    case = make([3000, 700, 2500], 8, 2, 128, 16, torch.bfloat16, 4, 2000, 4)
    q, kc, vc, tables, lens = [x.cuda() if isinstance(x, torch.Tensor) else torch.from_numpy(x).cuda() for x in case]
    ref = reference(case, 0.09, 2000, 4)
    side = torch.cuda.Stream()
    outs = [torch.empty_like(q) for _ in range(3)]
    junk = torch.full((64 << 20,), 0xAB, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del junk
    for out in outs:
        torch.cuda._sleep(20_000_000)
        pa.pa_decode_window(out, q, kc, vc, tables, lens, 0.09, window=2000, num_sinks=4, max_context_len=3000,
                            partition_size=64, stream=side.cuda_stream if raw else side)
    side.synchronize()
    for out in outs:
        assert_decode_close(out, ref, torch.bfloat16)
    torch.cuda.synchronize()
