"""pa_decode_tree and pa_decode_cross: several queries per sequence over the
paged cache, against fp64 attention over what each query sees.  Tolerances are
the framework's own (helpers.py): fp32 1e-5, bf16 2e-3 + 1e-2 |ref|."""
import ctypes

import numpy as np
import pytest
import torch

import multi_ref
from helpers import assert_decode_close
from multi_ref import Batch

FAKE = 0x10000
TYPES = [(torch.bfloat16, 128, 16), (torch.bfloat16, 64, 32), (torch.float32, 128, 32), (torch.float32, 64, 16)]


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


# ------------------------------------------------------------- on the CPU ---

@pytest.mark.parametrize("change,code", [
    (dict(hd=96), -2), (dict(bs=8), -2), (dict(dtype=9), -1), (dict(hq=6, hkv=4), -1), (dict(hkv=0), -1),
    (dict(T=-1), -1), (dict(seqs=-1), -1), (dict(q=None), -1), (dict(q=FAKE + 8), -1), (dict(start=None), -1),
    (dict(start=FAKE + 2), -1), (dict(phase=1), -2), (dict(simt=1), -2), (dict(P=64), -2), (dict(k_new=FAKE), -2),
    (dict(nb=0), -1), (dict(nb=2**31 - 1), -2), (dict(ctx=-1), -1), (dict(ws=None), -7), (dict(ws_bytes=100), -7),
    (dict(ws=FAKE + 8), -7), (dict(T=2**30), -2), (dict(seqs=0), 0), (dict(T=0), 0),
])
def test_bad_arguments_are_refused_on_the_host(pa, change, code):
    a = dict(q=FAKE, hd=128, bs=16, hq=8, hkv=2, seqs=2, dtype=1, P=0, ctx=64, phase=0, simt=0, T=5, start=FAKE,
             nb=8, ws=FAKE, ws_bytes=1 << 40, k_new=None)
    a.update(change)
    args = pa._DecodeArgs(a["seqs"], 512, a["nb"], a["dtype"], a["P"], a["ctx"], a["ws"], a["ws_bytes"], None, None,
                          a["phase"], a["k_new"], None, None, a["simt"], 0)
    tail = [a["hq"], a["hkv"], a["hd"], a["bs"], 0.1, a["T"]]
    head = [FAKE, a["q"], FAKE, FAKE, FAKE, FAKE, a["start"]]
    assert pa._lib.pa_decode_cross(*head, *tail, ctypes.byref(args)) == code, pa._lib.pa_last_error_string()
    assert pa._lib.pa_decode_tree(*head, None, *tail, 0, ctypes.byref(args)) == code


@pytest.mark.parametrize("mask,words", [(None, 1), (FAKE, 0), (FAKE, 17), (FAKE + 4, 1), (FAKE, -1)])
def test_bad_masks_are_refused_on_the_host(pa, mask, words):
    args = pa._DecodeArgs(2, 512, 8, 1, 0, 64, FAKE, 1 << 40)
    assert pa._lib.pa_decode_tree(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, mask, 8, 2, 128, 16, 0.1, 5, words,
                                  ctypes.byref(args)) == -1
    assert pa._lib.pa_decode_tree(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 8, 2, 128, 16, 0.1, 5, 0, None) == -1


def test_workspace_does_not_grow_with_contexts_and_stops_growing_with_rows(pa):
    size = pa.pa_decode_tree_workspace_size
    assert 0 < size(1, 8, 8, 64) < size(2, 8, 8, 64) < size(2, 16, 8, 64)
    assert size(10**5, 64, 8, 128) == size(10**6, 64, 8, 128)
    assert size(0, 8, 8, 64) == 0 and size(5, 8, 3, 64) == 0 and size(5, 0, 0, 64) == 0


def test_binding_refuses_wrong_tensors(pa):
    q = torch.zeros(1, 2, 64)
    for call in (pa.pa_decode_tree, pa.pa_decode_cross):
        with pytest.raises(ValueError, match="CUDA"):
            call(q, q, q, q, q, q, q, 0.1, max_context_len=1)


# ------------------------------------------------------------- on the GPU ---

def check(pa, b, scale, **kw):
    out, flags = b.on_gpu(pa, scale, **kw)
    assert flags == 0
    tokens = int(b.start[-1])
    assert_decode_close(out[:tokens], b.reference(scale), b.dtype, what=b.kind)
    assert (out[tokens:] == 7).all()
    return out


# Head counts that put a test's batch into items of few rows (4 query heads a KV head at most) or many (16).
WIDTHS = [2, 16]
LENS = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 400]


def counts(kind, lens, most, seed):
    rng = np.random.default_rng(seed)
    c = [int(rng.integers(0, most + 1)) for _ in lens]
    return c if kind == "cross" else [min(a, n) for a, n in zip(c, lens)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", multi_ref.KINDS)
@pytest.mark.parametrize("dtype,hd,bs", TYPES)
@pytest.mark.parametrize("most,Hq,Hkv", [(1, 4, 2), (9, 4, 2), (40, 2, 2), (70, 6, 2), (150, 4, 1), (30, 32, 2),
                                          (120, 16, 2), (8, 32, 1)])
def test_edge_lengths(pa, kind, dtype, hd, bs, most, Hq, Hkv):
    b = Batch(kind, LENS, counts(kind, LENS, most, most), Hq, Hkv, hd, bs, dtype, most + hd, padding=3)
    check(pa, b, hd ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", multi_ref.KINDS)
@pytest.mark.parametrize("group", [1, 3, 5, 7, 8, 12, 16, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_head_groups(pa, kind, group, dtype):
    lens = [100, 3, 300]
    b = Batch(kind, lens, [30, 3, 11], 2 * group, 2, 64, 16, dtype, group)
    check(pa, b, 0.11)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", multi_ref.KINDS)
@pytest.mark.parametrize("dtype,hd,bs", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_one_long_sequence_and_many_short_ones(pa, kind, dtype, hd, bs, width):
    """The axis is cut inside the long one and between the short ones."""
    lens = [9000] + [int(x) for x in np.random.default_rng(1).integers(1, 40, size=300)]
    b = Batch(kind, lens, counts(kind, lens, 3, 2), width, 1, hd, bs, dtype, 3)
    check(pa, b, hd ** -0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,hd,bs", TYPES)
@pytest.mark.parametrize("width", [1, *WIDTHS])
def test_arbitrary_masks_and_empty_rows(pa, dtype, hd, bs, width):
    """Bits in any pattern (later tokens, not itself); rows that see nothing at all are zero."""
    rng = np.random.default_rng(4)
    news = [130, 64, 65, 5, 1]
    lens = [130, 200, 65, 5, 1]
    see = [rng.random((c, c)) < 0.3 for c in news]
    see[0][7] = see[2][64] = see[3][:] = False
    see[4][:] = False
    b = Batch("mask", lens, news, 2 * width, 2, hd, bs, dtype, 5, see=see)
    out = check(pa, b, 0.2)
    at = b.start
    for row in (at[0] + 7, at[2] + 64, *range(at[3], at[5])):
        assert (out[row] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["mask", "chain"])
@pytest.mark.parametrize("dtype,hd,bs", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("width", WIDTHS)
def test_hidden_tokens_may_hold_anything(pa, kind, dtype, hd, bs, bad, width):
    """A drafted token whose values or keys are not finite spoils the rows that see it and no other."""
    c, n = 20, 150
    for side in ("v", "k"):
        b = Batch(kind, [n, n], [c, c], 2 * width, 2, hd, bs, dtype, 6)
        if kind == "mask":
            b.see[0][:, 11] = False
            b.see[0][[12, 14], 11] = True
            b.mask = torch.from_numpy(np.concatenate([multi_ref.mask_words(s, 1) for s in b.see]))
        clean = b.reference(0.1)
        pos = n - c + 11
        where = (int(b.tables[0, pos // bs]), 1, pos % bs)
        cols = slice(0, 5) if side == "v" else slice(None)
        getattr(b, side)[where][cols] = bad
        out, flags = b.on_gpu(pa, 0.1)
        assert flags == 0
        sees = b.visible(0)[:, pos]
        rows = torch.from_numpy(np.flatnonzero(sees))
        hit = torch.zeros_like(clean, dtype=torch.bool)
        hit[rows, width:] = True          # the query heads of KV head 1
        if side == "v":
            hit[:, :, 5:] = False
        got = out.double().cpu()
        assert_decode_close(torch.where(hit, 0, got), torch.where(hit, 0, clean), dtype)
        if side == "v":
            if bad != bad:
                assert got[hit].isnan().all()
            else:
                assert (got[hit] == bad).all()
        elif bad != bad and len(rows):
            assert got[hit].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", multi_ref.KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", WIDTHS)
def test_bad_device_data_is_flagged_and_harmless(pa, kind, dtype, width):
    b = Batch(kind, [100, 50, 300], [4, 3, 20], 2 * width, 2, 64, 16, dtype, 8)
    ref = b.reference(0.1)
    # a block id out of range reads as zeros
    b.tables[0, 2] = 10**6
    out, flags = b.on_gpu(pa, 0.1)
    assert flags == pa.STATUS_BAD_BLOCK_ID
    assert_decode_close(out, b.reference(0.1), dtype)
    assert_decode_close(out[4:], ref[4:], dtype)
    b.tables[0, 2] = 0
    # lengths beyond the bound are clamped to it, negative ones are empty
    b.lens[0] = -5
    out, flags = b.on_gpu(pa, 0.1)
    assert flags == pa.STATUS_BAD_CONTEXT_LEN
    assert (out[:4] == 0).all()
    assert_decode_close(out[4:], ref[4:], dtype)
    b.lens[0] = 100
    b.lens[2] = 10**9
    _, flags = b.on_gpu(pa, 0.1, max_context_len=300)
    assert flags == pa.STATUS_BAD_CONTEXT_LEN
    b.lens[2] = 300
    # query rows that run backwards or leave q: no queries, their rows are left
    for start in ([0, 4, 7, 28], [0, 4, 2, 27], [-1, 4, 7, 27], [0, -7, 7, 27]):
        b.start = np.array(start, np.int32)
        _, flags = b.on_gpu(pa, 0.1)
        assert flags & pa.STATUS_BAD_TREE
    if kind != "cross":
        # more queries than tokens: zero rows
        b.start = np.array([0, 4, 7, 27], np.int32)
        b.lens[1] = 2
        out, flags = b.on_gpu(pa, 0.1)
        assert flags == pa.STATUS_BAD_CONTEXT_LEN
        assert (out[4:7] == 0).all()
        assert_decode_close(out[7:], ref[7:], dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_mask_shorter_than_the_tree_hides_the_rest(pa, dtype):
    b = Batch("mask", [300], [100], 4, 2, 64, 16, dtype, 9)
    b.mask = b.mask[:, :1].contiguous()
    b.see[0][:, 64:] = False
    check(pa, b, 0.1)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", WIDTHS)
def test_scales(pa, scale, dtype, width):
    """Flat, reversed and peaked scores."""
    b = Batch("cross", [700, 40], [9, 30], 2 * width, 2, 128, 16, dtype, 10)
    out, _ = b.on_gpu(pa, scale)
    ref = b.reference(scale)
    if dtype == torch.float32 and scale == 3.0:
        # a score is off by at most (hd + 2) 2^-24 scale |q| |k|, a weight by e to twice that
        e = 130 * 2.0 ** -24 * 3.0 * float(b.q.norm(dim=-1).max()) * 20
        assert ((out.double().cpu() - ref).abs() <= 2.2 * e * 5 + 1e-5).all()
    else:
        assert_decode_close(out, ref, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_query_is_a_decode_step(pa, dtype):
    """A chain of one token, and a cross step of one query, are pa_decode."""
    lens = [1, 17, 700, 1300]
    b = Batch("chain", lens, [1] * 4, 8, 2, 128, 16, dtype, 11)
    plain = torch.empty_like(b.q).cuda()
    pa.pa_decode(plain, b.q.cuda(), b.k.cuda(), b.v.cuda(), torch.from_numpy(b.tables).cuda(),
                 torch.tensor(lens, dtype=torch.int32).cuda(), 0.09, max_context_len=1300)
    for kind in ("chain", "cross"):
        b.kind = kind
        out, _ = b.on_gpu(pa, 0.09)
        assert_decode_close(out, plain.double().cpu(), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", WIDTHS)
def test_repeatable_on_other_streams_and_in_graphs(pa, dtype, width):
    """Bit-identical results from call to call, on a side stream without a workspace, and replayed."""
    from paged_kv_cache_237_gb300.engine import TreeDecodeStep
    b = Batch("mask", [3100, 40, 900], [20, 5, 33], 2 * width, 2, 128, 16, dtype, 12)
    first, _ = b.on_gpu(pa, 0.1)
    args = [b.q.cuda(), b.k.cuda(), b.v.cuda(), torch.from_numpy(b.tables).cuda(),
            torch.tensor(b.lens, dtype=torch.int32).cuda(), torch.from_numpy(b.start).cuda(), 0.1]
    side, out = torch.cuda.Stream(), torch.empty_like(first)
    torch.cuda.synchronize()
    for _ in range(3):
        pa.pa_decode_tree(out.fill_(0), *args, max_context_len=3100, tree_mask=b.mask.cuda())
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    mask = b.mask.cuda()
    out.zero_()
    torch.cuda.synchronize()
    pa.pa_decode_tree(out, *args, max_context_len=3100, tree_mask=mask, stream=side)
    side.synchronize()
    assert torch.equal(out, first)
    step = TreeDecodeStep(*args, 3100, tree_mask=mask)
    step.decode()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.decode()
    for _ in range(2):
        step.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.out, first)
    # a replay follows its inputs (other lengths cut the work elsewhere, so the other rows' bits may differ)
    step.context_lens[0] = b.lens[0] = 3000
    graph.replay()
    assert_decode_close(step.out, b.reference(0.1), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("width", WIDTHS)
def test_large_offsets(pa, width):
    """A cache whose element offsets pass 2^31."""
    bs, hd, Hkv = 32, 128, 4
    nb = 2**31 // (bs * hd * Hkv) + 40
    k = torch.zeros(nb, Hkv, bs, hd, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    ids = torch.tensor([nb - 1, 3, nb - 20, nb - 7, 2], dtype=torch.int32)
    g = torch.Generator().manual_seed(0)
    small = Batch("chain", [150], [30], Hkv * width, Hkv, hd, bs, torch.bfloat16, 13)
    small.tables = np.arange(5, dtype=np.int32)[None]
    small.k, small.v = (torch.randn(5, Hkv, bs, hd, generator=g).bfloat16() for _ in range(2))
    k[ids.long().cuda()], v[ids.long().cuda()] = small.k.cuda(), small.v.cuda()
    out = torch.empty_like(small.q).cuda()
    pa.pa_decode_tree(out, small.q.cuda(), k, v, ids[None].cuda(), torch.tensor([150], dtype=torch.int32).cuda(),
                      torch.from_numpy(small.start).cuda(), 0.1, max_context_len=150)
    assert_decode_close(out, small.reference(0.1), torch.bfloat16)


@pytest.mark.gpu
def test_binding_checks_shapes_and_types(pa):
    b = Batch("mask", [40, 20], [4, 3], 4, 2, 64, 16, torch.bfloat16, 14)
    good = dict(out=b.q.cuda(), q=b.q.cuda(), k_cache=b.k.cuda(), v_cache=b.v.cuda(),
                block_tables=torch.from_numpy(b.tables).cuda(), context_lens=torch.tensor(b.lens).int().cuda(),
                query_start=torch.from_numpy(b.start).cuda(), scale=0.1, max_context_len=40, tree_mask=b.mask.cuda())
    pa.pa_decode_tree(**good)
    for name, bad, error in [
            ("q", b.q.cuda().half(), TypeError), ("q", b.q.cuda()[:, :, ::2], ValueError),
            ("out", b.q.cuda()[:-1], ValueError), ("query_start", good["query_start"][:-1], ValueError),
            ("query_start", good["query_start"].long(), TypeError), ("tree_mask", b.mask.cuda().int(), TypeError),
            ("tree_mask", b.mask.cuda()[:-1], ValueError), ("context_lens", good["context_lens"][:1], ValueError),
            ("v_cache", b.v.cuda()[:-1], ValueError),
            ("workspace", torch.zeros(64, dtype=torch.uint8, device="cuda"), pa.PAError)]:
        with pytest.raises(error):
            pa.pa_decode_tree(**{**good, name: bad})


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,hd", [(torch.bfloat16, 128), (torch.float32, 64)])
@pytest.mark.parametrize("width", WIDTHS)
def test_peaked_and_rising_scores(pa, dtype, hd, width):
    """Scores that rise along the context by much more than fp32's exponent holds, and one token that outweighs all:
    running maxima move at almost every step."""
    b = Batch("cross", [1500, 300], [10, 7], width, 1, hd, 16, dtype, 15)
    b.q[:] = b.q.abs()
    t = torch.arange(1500)
    blocks = torch.from_numpy(b.tables[0]).long()[t // 16]
    b.k[blocks, 0, t % 16] = (t[:, None] * 0.02).expand(-1, hd).to(dtype)
    t = torch.arange(300)
    blocks = torch.from_numpy(b.tables[1]).long()[t // 16]
    b.k[blocks, 0, t % 16] *= 0.01
    b.k[int(b.tables[1, 11]), 0, 3] = 5.0
    out, flags = b.on_gpu(pa, hd ** -0.5)
    assert flags == 0
    ref = b.reference(hd ** -0.5)
    # a score is off by at most (hd + 2) 2^-21 of the sum of |scale q k|, here up to 30 x 0.8 hd / sqrt(hd); a weight by e
    # to twice that, and the result by so much of the values (below 5)
    e = 2 * (hd + 2) * 2.0 ** -21 * 24 * hd ** 0.5
    tol = 2.0 ** -8 * ref.abs() + 2e-3 if dtype == torch.bfloat16 else 5 * e + 1e-5
    assert ((out.double().cpu() - ref).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", WIDTHS)
def test_visible_infinities_show(pa, dtype, width):
    """An infinite value that every row sees leaves every row's column without a finite result, and no other column.
    (In bf16 not always an infinity: a weight enters as two parts, hi + lo, and lo is zero for a weight that one part
    holds, and of either sign; infinity times zero, and infinities of two signs, are not numbers.)"""
    b = Batch("cross", [400, 90], [12, 3], width, 1, 64, 16, dtype, 16)
    at = lambda i, u: (int(b.tables[i, u // 16]), 0, u % 16)
    b.v[at(0, 7)][0] = float("inf")
    b.v[at(0, 300)][1] = -float("inf")
    b.v[at(0, 200)][2], b.v[at(0, 201)][2] = float("inf"), -float("inf")
    out = b.on_gpu(pa, 0.125)[0].double().cpu()
    assert not out[:12, :, :3].isfinite().any() and out[:12, :, 2].isnan().all()
    if dtype == torch.float32:
        assert (out[:12, :, 0] == float("inf")).all() and (out[:12, :, 1] == -float("inf")).all()
    ref = b.reference(0.125)
    assert_decode_close(out[:12, :, 3:], ref[:12, :, 3:], dtype)
    assert_decode_close(out[12:], ref[12:], dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_streams_with_workspaces_of_their_own(pa, dtype):
    batches = [Batch("mask", [2000, 70], [20, 9], 16, 2, 64, 16, dtype, 17), Batch("cross", [900] * 8, [60] * 8, 2, 2, 128,
                                                                                  16, dtype, 18)]
    calls = []
    for b in batches:
        args = [torch.zeros_like(b.q).cuda(), b.q.cuda(), b.k.cuda(), b.v.cuda(), torch.from_numpy(b.tables).cuda(),
                torch.tensor(b.lens, dtype=torch.int32).cuda(), torch.from_numpy(b.start).cuda(), 0.1]
        T, Hq, hd = b.q.shape
        ws = torch.empty(pa.pa_decode_tree_workspace_size(T, Hq, b.k.shape[1], hd), dtype=torch.uint8, device="cuda")
        kw = dict(max_context_len=max(b.lens), workspace=ws, stream=torch.cuda.Stream())
        if b.kind == "mask":
            kw["tree_mask"] = b.mask.cuda()
        calls.append((pa.pa_decode_tree if b.kind == "mask" else pa.pa_decode_cross, args, kw))
    torch.cuda.synchronize()
    for _ in range(20):
        for call, args, kw in calls:
            call(*args, **kw)
    torch.cuda.synchronize()
    for b, (_, args, _) in zip(batches, calls):
        assert_decode_close(args[0], b.reference(0.1), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("hd", [64, 128])
def test_many_short_items_in_a_row(pa, hd):
    """Items of one tile each, one behind the other in every CTA: whatever a stream of rows
    leaves for the other one must last until it is read.  Bit-equal from call to call."""
    rng = np.random.default_rng(hd)
    lens = rng.integers(1, 129, 3000).tolist()
    b = Batch("cross", lens, [20] * 3000, 2, 2, hd, 16, torch.bfloat16, 5)
    out = check(pa, b, hd ** -0.5)
    for _ in range(20):
        assert torch.equal(b.on_gpu(pa, hd ** -0.5)[0], out)


@pytest.mark.gpu
@pytest.mark.parametrize("hd", [64, 128])
def test_weights_that_are_alike(pa, hd):
    """One token above 4095 equal ones, whose weight e^-s is as far from a bf16 value as can be:
    a row is off by its weights' rounding (2^-8 of itself) and its own (2^-8), no more."""
    n = 4096
    grid = torch.arange(128, 256, dtype=torch.float64) / 256                       # bf16 values of [0.5, 1)
    s = grid[:, None] * (grid + 0.5)[None, :].to(torch.bfloat16).double()          # products are exact in fp32
    w = torch.exp(-s)
    off = ((w.to(torch.bfloat16).double() - w).abs() / w).flatten()
    i, j = divmod(int(off.argmax()), 128)
    assert off.max() > 0.95 * 2 ** -8
    b = Batch("cross", [n], [300], 2, 2, hd, 16, torch.bfloat16, 9)
    b.q.zero_()
    b.q[..., 0] = grid[i].to(torch.bfloat16)
    b.k.masked_fill_(~b.k.isnan(), 0.0)
    b.k[int(b.tables[0, 0]), :, 0, 0] = (grid[j] + 0.5).to(torch.bfloat16)
    v0 = float(b.v[int(b.tables[0, 0]), :, 0].abs().max())
    out = b.on_gpu(pa, 1.0)[0].double().cpu()
    q, first = b.q[:1].clone(), b.start.copy()
    b.q, b.start, b.news = q, np.array([0, 1], np.int32), [1]                      # all rows are the same
    want = b.reference(1.0)
    # fp32: the sum of 4096 weights is off by 4096 * 2^-24 at most; a product's sums by 2^-22 of the largest partial sum at
    # each of 256 steps, in two parts of p; the first token's weight is one of 4095 * 0.5 and off by 2^-8 itself.
    t = torch.arange(n)
    v = b.v[torch.from_numpy(b.tables[0]).long()[t // 16], :, t % 16].double()
    slack = 2 * 2 ** -8 + 2 ** -16 + 4096 * 2 ** -24
    floor = 512 * 2 ** -22 * 2 * float(v.cumsum(0).abs().max()) / 4095 + 2 ** -8 * v0 / 2000
    assert ((out - want).abs() <= slack * want.abs() + floor).all()
