"""pa_decode_q4: decode attention over the 4-bit cache against fp64 attention over
the values the cache holds.

Tolerances.  fp32 outputs: the framework's 1e-5 for unit-sized values, times the
largest |v|.  bf16 outputs: half a step of the result (2^-8 |ref|), plus the
weights' rounding: a weight may enter its product as fp16 (relative 2^-11), the
weights sum to 1 and a value's code part s * c is at most twice the largest
|v|, so 2^-10 max|v|; a quarter of that again for the fp32 scores (a dot
product of 128 terms of size 1 is off by less than 2^-14 in the exponent, which
moves weighted values by less than 2^-12 max|v|)."""
import ctypes

import numpy as np
import pytest
import torch

import q4_ref

FAKE = 0x10000


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


# ------------------------------------------------------------- on the CPU ---

@pytest.mark.parametrize("change,code", [
    (dict(hd=96), -2), (dict(bs=8), -2), (dict(group=16), -2), (dict(hq=6, hkv=4), -1), (dict(hkv=0), -1),
    (dict(dtype=5), -1), (dict(P=16), -1), (dict(P=48), -1), (dict(P=2048), -1), (dict(phase=3), -1),
    (dict(window=-1), -1), (dict(sinks=-1), -1), (dict(ctx=4096, P=512), -7), (dict(ctx=4096, P=512, window=600), -7),
    (dict(q=None), -1), (dict(kc=FAKE + 8), -1), (dict(simt=1), -2), (dict(k_new=FAKE), -2), (dict(seqs=-1), -1),
    (dict(nb=0), -1), (dict(width=0), -1), (dict(ctx=-1), -1), (dict(seqs=0), 0),
])
def test_bad_arguments_are_refused_on_the_host(pa, change, code):
    a = dict(q=FAKE, kc=FAKE, hq=8, hkv=2, hd=128, bs=16, group=64, window=0, sinks=0, seqs=2, width=512, nb=8,
             dtype=1, P=0, ctx=64, phase=0, k_new=None, simt=0)
    a.update(change)
    args = pa._DecodeArgs(a["seqs"], a["width"], a["nb"], a["dtype"], a["P"], a["ctx"], None, 0, None, None,
                          a["phase"], a["k_new"], None, None, a["simt"], 0)
    rc = pa._lib.pa_decode_q4(FAKE, a["q"], a["kc"], FAKE, FAKE, FAKE, a["hq"], a["hkv"], a["hd"], a["bs"],
                              a["group"], 0.1, a["window"], a["sinks"], ctypes.byref(args))
    assert rc == code, pa._lib.pa_last_error_string()
    if code:
        assert b"pa_decode_q4" in pa._lib.pa_last_error_string()
    assert pa._lib.pa_decode_q4(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 8, 2, 128, 16, 64, 0.1, 0, 0, None) == -1


def test_workspace_sizes(pa):
    """A header and a word per sequence, then two rows of heads (4, 8 or 16 for
    groups of up to 4, up to 8 and above) for each stretch: at most 2432 of them, and at most one
    per partition_size tokens of what the batch can hold."""
    size = pa.pa_decode_q4_workspace_size
    assert size(4, 8, 2, 128, 512, 512) == 0 and size(4, 8, 2, 128, 0) == 0 and size(0, 8, 2, 128, 4096) == 0
    assert size(4, 9, 2, 128, 4096) == 0        # refused: 9 heads over 2
    a256 = lambda x: (x + 255) // 256 * 256

    def want(seqs, rows, tile, hd, tokens, P):
        n = min(2432, -(-(seqs * rows * -(-tokens // 32)) // (P // 32)))
        return 256 + a256(4 * seqs) + a256(n * 2 * tile * 8) + a256(n * 2 * tile * hd * 4)

    assert size(4, 8, 2, 128, 1025, 512) == want(4, 2, 4, 128, 1025, 512)
    assert size(4, 10, 2, 128, 1025, 512) == want(4, 2, 8, 128, 1025, 512)
    assert size(300, 64, 8, 64, 10**6, 512) == want(300, 8, 8, 64, 10**6, 512)
    assert size(4, 40, 2, 128, 1025, 512) == want(4, 4, 16, 128, 1025, 512)
    # a window bounds what is walked: 600 tokens, 5 sinks, and blocks of 32 at their edges
    assert size(4, 8, 2, 128, 10**6, 512, window=600, num_sinks=5) == want(4, 2, 4, 128, 32 + 600 + 31, 512)
    big = 2**31 - 1
    assert size(1, 1, 1, 64, big, 1024) == want(1, 1, 4, 64, big, 1024)
    assert size(1, 1, 1, 64, big, 1024, window=big, num_sinks=big) == size(1, 1, 1, 64, big, 1024)


def test_binding_refuses_cpu_tensors(pa):
    q = torch.zeros(1, 2, 64)
    with pytest.raises(ValueError):
        pa.pa_decode_q4(q, q, torch.zeros(1, 1, 640, dtype=torch.uint8), torch.zeros(1, 1, 640, dtype=torch.uint8),
                        torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32), 0.1,
                        max_context_len=1)


# ------------------------------------------------------------- on the GPU ---

def make(lens, Hq, Hkv, hd, bs, group, dtype, seed, window=0, sinks=0, spread=1.0):
    """A batch whose pool holds NaN wherever nothing may be read: behind each
    sequence's end, in blocks of nobody, and (windowed) in given-back blocks'
    table entries, which hold junk."""
    rng = np.random.default_rng(seed)
    per = [-(-n // bs) for n in lens]
    nb, width = sum(per) + 3, max(1, max(per))
    perm = rng.permutation(nb)
    tables = np.full((len(lens), width), -1, np.int32)
    shape = (nb, Hkv, bs, hd // group)
    cut = bs * hd // 2
    caches = []
    live = np.zeros((nb, bs), bool)
    at = 0
    for i, n in enumerate(lens):
        tables[i, :per[i]] = perm[at:at + per[i]]
        at += per[i]
        for j in range(per[i]):
            t = np.arange(j * bs, j * bs + bs)
            seen = (t < n) & ((t >= n - window) | (t < sinks) if window else True)
            live[tables[i, j]] = seen
            if not seen.any():
                tables[i, j] = rng.choice([-1, 2**31 - 1, nb, -2**31])
    for _ in range(2):
        cache = np.empty((nb, Hkv, q4_ref.page_bytes(hd, bs, group)), np.uint8)
        cache[..., :cut] = rng.integers(0, 256, (nb, Hkv, cut), dtype=np.uint8)
        s = rng.uniform(0.02, 0.4, shape) * spread
        m = rng.uniform(-3.5, -1.0, shape) * spread
        dead = ~live[:, None, :, None] & np.ones(shape, bool)
        s[dead], m[dead] = np.inf, np.nan
        par = np.stack([q4_ref.bf16_bits(s), q4_ref.bf16_bits(m)], -1)
        cache[..., cut:] = np.ascontiguousarray(par).view(np.uint8).reshape(nb, Hkv, -1)
        caches.append(cache)
    q = torch.from_numpy(rng.standard_normal((len(lens), Hq, hd))).to(dtype)
    return q, caches[0], caches[1], tables, np.array(lens, np.int32)


def on_gpu(pa, case, scale, group, dtype, **kw):
    q, kc, vc, tables, lens = case
    status = pa.DeviceStatus()
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    pa.pa_decode_q4(out, q.cuda(), torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(),
                    torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), scale,
                    max_context_len=max(1, int(lens.max())), group_size=group, status=status, **kw)
    torch.cuda.synchronize()
    return out, status.read()


def check(out, case, scale, bs, group, window=0, sinks=0, what=""):
    q, kc, vc, tables, lens = case
    hd = q.shape[-1]
    with np.errstate(invalid="ignore"):      # inf * 0 in dead slots
        k, v = q4_ref.values(kc, bs, hd, group), q4_ref.values(vc, bs, hd, group)
    ref = q4_ref.attend(q.double().numpy(), k, v, tables, lens, scale, bs, window, sinks)
    o = out.double().cpu().numpy()
    assert np.isfinite(o).all(), f"{what}: not finite"
    vmax = np.abs(v[np.isfinite(v)]).max()
    tol = 1e-5 * vmax + 0 * ref if out.dtype == torch.float32 else 2.0 ** -8 * np.abs(ref) + 1.25 * 2.0 ** -10 * vmax
    worst = (np.abs(o - ref) / tol).max() if o.size else 0
    assert worst <= 1, f"{what}: error {worst:.2f} of the tolerance, at {np.unravel_index((np.abs(o - ref) / tol).argmax(), o.shape)}"


FORMATS = [(128, 16, 64), (128, 32, 32), (128, 32, 64), (64, 16, 32), (64, 32, 64), (64, 32, 32)]
EDGES = [0, 1, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 127, 511, 512, 513, 1025, 1100]


@pytest.mark.gpu
@pytest.mark.parametrize("hd,bs,group", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("P", [0, 64, 512])
def test_edge_lengths(pa, hd, bs, group, dtype, P):
    case = make(EDGES, 8, 2, hd, bs, group, dtype, seed=hd + bs)
    out, flags = on_gpu(pa, case, hd ** -0.5, group, dtype, partition_size=P)
    assert flags == 0
    check(out, case, hd ** -0.5, bs, group, what=f"P {P}")
    assert (out[0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (3, 1), (4, 1), (5, 1), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1),
                                    (24, 2), (40, 1), (64, 8), (6, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_head_layouts(pa, Hq, Hkv, dtype):
    for hd, bs, group in ((128, 16, 32), (64, 32, 64)):
        case = make([100, 3, 700], Hq, Hkv, hd, bs, group, dtype, seed=Hq)
        out, flags = on_gpu(pa, case, hd ** -0.5, group, dtype, partition_size=256)
        assert flags == 0
        check(out, case, hd ** -0.5, bs, group, what=f"heads {Hq}/{Hkv} hd {hd}")


WINDOWS = [(1, 0), (1, 1), (5, 3), (16, 16), (17, 33), (32, 0), (33, 64), (100, 1), (500, 4), (3000, 4), (64, 2000)]


@pytest.mark.gpu
@pytest.mark.parametrize("hd,bs,group", [(128, 16, 64), (128, 32, 32), (64, 16, 32), (64, 32, 64)])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_windows(pa, hd, bs, group, window, sinks):
    for dtype, P in ((torch.bfloat16, 0), (torch.float32, 64)):
        case = make(EDGES, 4, 2, hd, bs, group, dtype, window + sinks, window, sinks)
        out, flags = on_gpu(pa, case, hd ** -0.5, group, dtype, partition_size=P, window=window, num_sinks=sinks)
        assert flags == 0
        check(out, case, hd ** -0.5, bs, group, window, sinks, what=f"{dtype}")


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [1e-6, 1e-20, 1e6, 1e20])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_values_far_from_one(pa, spread, dtype):
    """Steps and minima of any size bf16 holds; q is scaled back so that scores stay ordinary."""
    case = list(make([600, 77], 8, 1, 128, 16, 64, dtype, 5, spread=spread))
    case[0] = (case[0].double() / spread).to(dtype)
    out, flags = on_gpu(pa, case, 128 ** -0.5, 64, dtype, partition_size=256)
    assert flags == 0
    check(out, case, 128 ** -0.5, 16, 64, what=f"spread {spread}")


@pytest.mark.gpu
def test_mixed_sizes_of_steps_in_one_sequence(pa):
    """Tokens whose steps differ by up to 2^30, small ones first and large ones first."""
    for order in (1, -1):
        q, kc, vc, tables, lens = make([400], 8, 1, 128, 16, 64, torch.bfloat16, 6)
        cut = 16 * 64
        par = np.ascontiguousarray(vc[..., cut:]).view(np.uint16).reshape(-1, 16, 2, 2).copy()
        for j, b in enumerate(tables[0]):
            e = 2.0 ** ((j - 12) * order)
            p = torch.from_numpy(par[b].view(np.int16)).view(torch.bfloat16).double() * e
            par[b] = q4_ref.bf16_bits(p.numpy())
        vc[..., cut:] = par.view(np.uint8).reshape(vc.shape[0], 1, -1)
        case = (q, kc, vc, tables, lens)
        out, flags = on_gpu(pa, case, 128 ** -0.5, 64, torch.bfloat16)
        assert flags == 0
        check(out, case, 128 ** -0.5, 16, 64, what=f"order {order}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_peaked_and_flat_scores(pa, dtype):
    for scale in (0.0, 3.0, 40.0, -1.0):
        case = make([1, 300, 1000], 8, 2, 64, 16, 32, dtype, 9)
        out, flags = on_gpu(pa, case, scale, 32, dtype, partition_size=128)
        assert flags == 0
        if abs(scale) < 2 or dtype == torch.bfloat16 and scale == 3.0:
            check(out, case, scale, 16, 32, what=f"scale {scale}")
        else:
            # fp32 scores of size 40 * 30 are off by more than a softmax forgives; the result stays a mean of values
            k, v = q4_ref.values(case[2], 16, 64, 32), None
            assert torch.isfinite(out).all() and float(out.abs().max()) <= np.nanmax(np.where(np.isfinite(k), k, 0)) + 4


@pytest.mark.gpu
@pytest.mark.parametrize("hd,group", [(128, 64), (64, 32)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_long_flat_sums_keep_their_precision(pa, dtype, hd, group):
    """20000 tokens of nearly equal weight and values of mean zero: the output is a
    hundredth of the values, so an error of the sums' size rather than the
    output's shows.  In the 2-norm, weights' errors are independent of each
    other: fp32 parts of a few 2^-23 each (the exponential, the weight's two
    fp16 parts) stay below 2^-19 relative; for bf16, half a step of the result
    spread evenly is 2^-8 / sqrt(3), the fp16 weights' 2^-11 / sqrt(3) times the
    code part's size against the value's (3), and as much again for the sums."""
    rng = np.random.default_rng(12)
    case = list(make([20000, 9000], 8, 1, hd, 16, group, dtype, 12))
    cut = 16 * hd // 2
    par = case[2][..., cut:].copy().view(np.uint16).reshape(case[2].shape[0], 1, 16, -1, 2)
    s = torch.from_numpy(par[..., 0].view(np.int16).copy()).view(torch.bfloat16).double().numpy()
    par[..., 1] = q4_ref.bf16_bits(np.where(np.isfinite(s), -7.5 * s, np.nan))    # ranges about zero
    case[2] = case[2].copy()
    case[2][..., cut:] = par.view(np.uint8).reshape(case[2].shape[0], 1, -1)
    scale = 0.02 * hd ** -0.5
    out, flags = on_gpu(pa, case, scale, group, dtype)
    assert flags == 0
    q, kc, vc, tables, lens = case
    with np.errstate(invalid="ignore"):
        k, v = q4_ref.values(kc, 16, hd, group), q4_ref.values(vc, 16, hd, group)
    ref = q4_ref.attend(q.double().numpy(), k, v, tables, lens, scale, 16)
    rel = np.linalg.norm(out.double().cpu().numpy() - ref) / np.linalg.norm(ref)
    assert rel <= (2.0 ** -19 if dtype == torch.float32 else (2.0 ** -8 + 6 * 2.0 ** -11) / 3 ** 0.5), rel


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_in_a_visible_group_shows_in_its_columns_only(pa, dtype):
    """A NaN value group poisons its 32 columns, a NaN key group its whole rows, as an unquantised cache would."""
    q, kc, vc, tables, lens = make([90, 70], 4, 1, 128, 16, 32, dtype, 4)
    cut = 16 * 64
    bad = q4_ref.bf16_bits([0.0, np.nan]).view(np.uint8)
    b = tables[0][2]
    vc2 = vc.copy()
    vc2[b, 0, cut + 3 * 16 + 4:cut + 3 * 16 + 8] = bad          # row 3, group 1
    out, _ = on_gpu(pa, (q, kc, vc2, tables, lens), 0.09, 32, dtype)
    nan = torch.isnan(out.cpu())
    assert nan[0, :, 32:64].all() and int(nan.sum()) == 4 * 32
    kc2 = kc.copy()
    kc2[b, 0, cut + 3 * 16 + 4:cut + 3 * 16 + 8] = bad
    out, _ = on_gpu(pa, (q, kc2, vc, tables, lens), 0.09, 32, dtype)
    assert torch.isnan(out.cpu()[0]).all() and torch.isfinite(out.cpu()[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bs,group", [(16, 64), (32, 32)])
def test_bad_blocks_and_lengths_are_flagged(pa, bs, group):
    case = list(make([200, 150, 90], 8, 2, 128, bs, group, torch.bfloat16, 8))
    case[3] = case[3].copy()
    case[3][0, 1], case[3][1, 2] = -1, case[1].shape[0]
    out, flags = on_gpu(pa, case, 0.09, group, torch.bfloat16, partition_size=64)
    assert flags == pa.STATUS_BAD_BLOCK_ID
    check(out, case, 0.09, bs, group, what="bad ids read as zeros")
    case = list(make([200, 150, 90], 8, 2, 128, bs, group, torch.bfloat16, 8))
    longer = case[4].copy()
    longer[0], longer[1] = 2**31 - 1, -3
    case[4] = longer
    status = pa.DeviceStatus()
    q, kc, vc, tables, lens = case
    width = tables.shape[1]
    out = torch.empty_like(q).cuda()
    pa.pa_decode_q4(out, q.cuda(), torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(),
                    torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), 0.09, max_context_len=200,
                    group_size=group, status=status)
    assert status.read() == pa.STATUS_BAD_CONTEXT_LEN and (out[1] == 0).all()
    case[4] = np.array([200, 0, 90], np.int32)
    assert width * bs >= 200
    check(out, case, 0.09, bs, group, what="clamped length")


@pytest.mark.gpu
def test_batches_of_nothing_and_of_many_short_rows(pa):
    """No token anywhere; and more rows than the GPU has warps, most of them empty or short, split and unsplit."""
    for dtype in (torch.bfloat16, torch.float32):
        case = make([0, 0, 0], 8, 2, 128, 16, 64, dtype, 1)
        for ctx in (1, 5000):
            q, kc, vc, tables, lens = case
            out = torch.full(q.shape, 5.0, dtype=dtype, device="cuda")
            pa.pa_decode_q4(out, q.cuda(), torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(),
                            torch.from_numpy(np.repeat(tables, 320, 1)).cuda(), torch.from_numpy(lens).cuda(), 0.09,
                            max_context_len=ctx, group_size=64)
            assert (out == 0).all()
        lens = np.random.default_rng(2).choice([0, 1, 2, 16, 31, 33, 64, 70, 130], size=700).tolist()
        case = make(lens, 8, 8, 64, 16, 32, dtype, 2)
        for P in (0, 32, 256):
            out, flags = on_gpu(pa, case, 0.125, 32, dtype, partition_size=P)
            assert flags == 0
            check(out, case, 0.125, 16, 32, what=f"{dtype} P {P}")


def step(pa, case, group, **kw):
    from paged_kv_cache_237_gb300.engine import Q4DecodeStep
    q, kc, vc, tables, lens = case
    return Q4DecodeStep(q.cuda(), torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(),
                        torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(), 0.09, int(lens.max()),
                        group_size=group, **kw)


@pytest.mark.gpu
def test_repeats_phases_and_graphs_give_the_same_bits(pa):
    case = make([900, 33, 2000, 0, 640], 16, 2, 128, 16, 64, torch.bfloat16, 11)
    s = step(pa, case, 64, partition_size=128)
    first = s.decode().clone()
    check(first, case, 0.09, 16, 64)
    for _ in range(5):
        s.out.fill_(float("nan"))
        assert torch.equal(s.decode(), first)
    s.out.fill_(float("nan"))
    s.decode(phase=pa.PA_PHASE_PARTITIONS)
    assert torch.equal(s.decode(phase=pa.PA_PHASE_REDUCE), first)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        s.decode()
        s.decode()
    s.q.mul_(2)
    s.out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    doubled = (s.q.cpu(), *case[1:])
    check(s.out, doubled, 0.09, 16, 64)
    assert s.status.read() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("word", [-1, 0, 1, 1 << 30, -(1 << 31)])
def test_a_join_without_its_pass_stays_inside_the_workspace(pa, word):
    """Places left unwritten (as by a pass that gave up on a wait) are whatever
    the workspace held: rows that they put past its end are left out."""
    case = make([900, 33, 2000, 0, 640], 16, 2, 128, 16, 64, torch.bfloat16, 11)
    s = step(pa, case, 64, partition_size=128)
    s.workspace.view(torch.int32).fill_(word)
    s.decode(phase=pa.PA_PHASE_REDUCE)
    torch.cuda.synchronize()
    s.out.fill_(float("nan"))
    check(s.decode(), case, 0.09, 16, 64)
    assert s.status.read() == 0


@pytest.mark.gpu
def test_two_calls_at_once_on_streams_of_their_own(pa):
    cases = [make([3000, 500], 8, 1, 128, 16, 64, torch.bfloat16, 20 + i) for i in range(2)]
    steps = [step(pa, c, 64, partition_size=64) for c in cases]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st in zip(steps, streams):
            s.decode(stream=st)
    torch.cuda.synchronize()
    for s, c in zip(steps, cases):
        check(s.out, c, 0.09, 16, 64)
        assert s.status.read() == 0


@pytest.mark.gpu
def test_pages_past_four_gigabytes(pa):
    hd, bs, group, H = 128, 32, 32, 32
    page = q4_ref.page_bytes(hd, bs, group)
    nb = (1 << 32) // (H * page) + 4
    case = make([70, 5], H, H, hd, bs, group, torch.bfloat16, 3)
    q, kc, vc, tables, lens = case
    n = kc.shape[0]
    far_k = torch.zeros(nb, H, page, dtype=torch.uint8, device="cuda")
    far_v = torch.zeros_like(far_k)
    far_k[nb - n:], far_v[nb - n:] = torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda()
    moved = np.where(tables >= 0, tables + nb - n, -1).astype(np.int32)
    out = torch.empty_like(q).cuda()
    pa.pa_decode_q4(out, q.cuda(), far_k, far_v, torch.from_numpy(moved).cuda(), torch.from_numpy(lens).cuda(), 0.09,
                    max_context_len=70, group_size=group)
    check(out, case, 0.09, bs, group)
