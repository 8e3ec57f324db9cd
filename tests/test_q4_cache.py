"""pa_reshape_and_cache_q4 and pa_gather_q4: the 4-bit cache's bytes and the
values they stand for, against the numpy implementation of the format.

Both are exact: the format fixes every rounding, so bytes must be equal, and a
value s * c + m (exact in fp64) is rounded once, so gathered values must equal
the fp64 value rounded to the output type.  (The sign of a zero minimum is not
fixed by the format; the inputs below hold no negative zeros.)"""
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

def test_the_reference_covers_its_inputs():
    """|s c + m - x| <= s / 2 up to the fp32 roundings of (x - m) * (1 / s):
    three roundings of a quotient of at most 15 (1 + 2^-23), 15 * 3 * 2^-24 steps."""
    rng = np.random.default_rng(0)
    for scale in (1e-30, 1e-3, 1.0, 1e4, 1e30):
        x = q4_ref.f32(rng.standard_normal((50, 2, 128)) * scale + scale * 3)
        c, s, m = q4_ref.quantise(x, 32)
        y = c * np.repeat(s, 32, -1) + np.repeat(m, 32, -1)
        assert (np.abs(y - x) <= np.repeat(s, 32, -1) * (0.5 + 45 * 2.0 ** -24)).all()


def test_pack_and_unpack_are_inverse():
    rng = np.random.default_rng(1)
    for hd, bs, g in ((64, 16, 32), (64, 32, 64), (128, 32, 32), (128, 16, 64)):
        x = q4_ref.f32(rng.standard_normal((7, 3, hd)))
        cache = np.zeros((2, 3, q4_ref.page_bytes(hd, bs, g)), np.uint8)
        slots = rng.permutation(2 * bs)[:7]
        q4_ref.write(cache, x, slots, bs, g)
        c, s, m = q4_ref.quantise(x, g)
        got = q4_ref.values(cache, bs, hd, g)[slots // bs, :, slots % bs]
        assert np.array_equal(got, c * np.repeat(s, g, -1) + np.repeat(m, g, -1))


def test_page_bytes(pa):
    for hd in (64, 128):
        for bs in (16, 32):
            for g in (32, 64):
                assert pa.pa_q4_page_bytes(hd, bs, g) == q4_ref.page_bytes(hd, bs, g)
                assert pa.pa_q4_page_bytes(hd, bs, g) % 16 == 0
    for bad in ((96, 16, 32), (128, 8, 32), (128, 16, 128), (128, 16, 0)):
        assert pa._lib.pa_q4_page_bytes(*bad) == 0
        with pytest.raises(pa.PAError):
            pa.pa_q4_page_bytes(*bad)


@pytest.mark.parametrize("name", ["pa_reshape_and_cache_q4", "pa_gather_q4"])
@pytest.mark.parametrize("change,code", [
    (dict(dtype=7), -1), (dict(tokens=-1), -1), (dict(heads=0), -1), (dict(blocks=0), -1),
    (dict(hd=96), -2), (dict(bs=8), -2), (dict(group=128), -2), (dict(k=None), -1), (dict(slots=None), -1),
    (dict(k=FAKE + 8), -1), (dict(slots=FAKE + 4), -1), (dict(tokens=2**31 - 1, heads=64), -2), (dict(tokens=0), 0),
])
def test_bad_arguments_are_refused_on_the_host(pa, name, change, code):
    a = dict(k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, slots=FAKE, tokens=3, heads=2, hd=128, bs=16, group=64, blocks=4,
             dtype=1, status=None, stream=None)
    a.update(change)
    fn = getattr(pa._lib, name)
    assert fn(*a.values()) == code
    if code:
        assert name.encode() in pa._lib.pa_last_error_string()


def test_binding_refuses_cpu_tensors_and_block_rows_shares_memory(pa):
    k = torch.zeros(2, 3, 64)
    cache = torch.zeros(4, 3, pa.pa_q4_page_bytes(64, 16, 32), dtype=torch.uint8)
    with pytest.raises(ValueError):
        pa.pa_reshape_and_cache_q4(k, k, cache, cache, torch.zeros(2, dtype=torch.int64), group_size=32)
    rows = pa.q4_block_rows(cache, 16)
    assert rows.data_ptr() == cache.data_ptr() and rows.shape[:3] == (4, 3, 16) and rows.dtype == torch.bfloat16
    assert rows.numel() * 2 == cache.numel()


# ------------------------------------------------------------- on the GPU ---

def rows(T, H, hd, dtype, seed):
    """Rows whose groups cover the format's corners, besides normals."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, hd, generator=g)
    x[0] = 0.0                                              # step 0
    x[1 % T] = 2.5                                          # constant, exact in bf16
    if T > 8:
        x[2] = 1.0009765625                                 # constant, not exact in bf16
        x[3] *= 1e-30
        x[4] = x[4] * 1e30
        x[5] = torch.linspace(-3, 4.5, hd)                  # ties: 15 equal steps of 1/2 per 64, and halves
        x[6] = x[6].abs() * 1e-39                           # subnormal
        x[7] = torch.randint(0, 16, (H, hd), generator=g).float() * 0.25 - 1.0
        x[7, :, 0::32], x[7, :, 1::32] = -1.0, 2.75         # an exact grid: codes and values are exact
        x[8] = x[8] + 300.0                                 # minimum far from zero
    return (x + 0.0).to(dtype)


CASES = [(hd, bs, group, dtype, T, H)
         for hd, bs, group in ((128, 16, 64), (128, 32, 32), (64, 16, 32), (64, 32, 64))
         for dtype in (torch.bfloat16, torch.float32) for T, H in ((1, 1), (2, 5), (61, 3))]


def run_write(pa, x, y, kc, vc, slots, group):
    status = pa.DeviceStatus()
    dk, dv = torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda()
    sm = torch.from_numpy(slots).cuda()
    pa.pa_reshape_and_cache_q4(x.cuda(), y.cuda(), dk, dv, sm, group_size=group, status=status)
    return dk, dv, sm, status


@pytest.mark.gpu
@pytest.mark.parametrize("hd,bs,group,dtype,T,H", CASES)
def test_write_and_gather_are_exact(pa, hd, bs, group, dtype, T, H):
    rng = np.random.default_rng(T)
    nb = 1 + (T + bs - 1) // bs * 2
    x, y = rows(T, H, hd, dtype, 1), rows(T, H, hd, dtype, 2)
    kc = rng.integers(0, 256, (nb, H, q4_ref.page_bytes(hd, bs, group)), dtype=np.uint8)
    vc = rng.integers(0, 256, kc.shape, dtype=np.uint8)
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    if T > 8:
        slots[T // 2] = -1
    dk, dv, sm, status = run_write(pa, x, y, kc, vc, slots, group)
    k = torch.full_like(x, 7.0).cuda()
    v = torch.full_like(x, 7.0).cuda()
    pa.pa_gather_q4(k, v, dk, dv, sm, group_size=group, status=status)
    torch.cuda.synchronize()
    assert status.read() == 0
    for src, cache, dev, got in ((x, kc, dk, k), (y, vc, dv, v)):
        q4_ref.write(cache, src.double().numpy(), slots, bs, group)
        assert np.array_equal(dev.cpu().numpy(), cache)             # every byte of the pool
        ref = torch.from_numpy(q4_ref.values(cache, bs, hd, group)[slots // bs, :, slots % bs]).to(dtype)
        keep = torch.from_numpy(slots >= 0)
        assert torch.equal(got.cpu()[keep], ref[keep])
        assert (got.cpu()[~keep] == 7.0).all()                      # padding rows left as they were


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), 2.0 ** 126, -3e38])
def test_a_group_with_something_not_finite_stands_for_nan(pa, dtype, bad):
    x = torch.randn(3, 2, 128, generator=torch.Generator().manual_seed(0)).to(dtype)
    x[1, 1, 40] = bad
    kc = np.zeros((1, 2, q4_ref.page_bytes(128, 16, 32)), np.uint8)
    dk, dv, sm, status = run_write(pa, x, x, kc, kc.copy(), np.array([0, 1, 2]), 32)
    k, v = torch.empty_like(x).cuda(), torch.empty_like(x).cuda()
    pa.pa_gather_q4(k, v, dk, dv, sm, group_size=32)
    nan = torch.isnan(k.cpu())
    assert nan[1, 1, 32:64].all() and int(nan.sum()) == 32 and torch.equal(nan, torch.isnan(v.cpu()))
    q4_ref.write(kc, x.double().numpy(), [0, 1, 2], 16, 32)
    assert np.array_equal(dk.cpu().numpy(), kc)


@pytest.mark.gpu
def test_bad_slots_are_flagged_and_nothing_else_is_touched(pa):
    x = torch.randn(4, 2, 64, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    kc = np.full((2, 2, q4_ref.page_bytes(64, 16, 32)), 0xAB, np.uint8)
    slots = np.array([31, 32, 2**40, -5], np.int64)
    dk, dv, sm, status = run_write(pa, x, x, kc, kc.copy(), slots, 32)
    assert status.read() == pa.STATUS_BAD_SLOT
    q4_ref.write(kc, x.double().numpy(), [31, -1, -1, -1], 16, 32)
    assert np.array_equal(dk.cpu().numpy(), kc) and np.array_equal(dv.cpu().numpy(), kc)
    k = torch.full_like(x, 3.0).cuda()
    v = k.clone()
    pa.pa_gather_q4(k, v, dk, dv, sm, group_size=32, status=status)
    assert status.read() == pa.STATUS_BAD_SLOT
    assert (k[1:].cpu() == 3.0).all() and not (k[0].cpu() == 3.0).all()


@pytest.mark.gpu
def test_pages_past_four_gigabytes(pa):
    """Offsets of the last page pass 32 bits."""
    hd, bs, group, H = 128, 32, 32, 32
    page = q4_ref.page_bytes(hd, bs, group)
    nb = (1 << 32) // (H * page) + 3
    dk = torch.zeros(nb, H, page, dtype=torch.uint8, device="cuda")
    dv = torch.zeros_like(dk)
    x = torch.randn(2, H, hd, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    slots = torch.tensor([nb * bs - 1, 0])
    pa.pa_reshape_and_cache_q4(x.cuda(), x.cuda(), dk, dv, slots.cuda(), group_size=group)
    ref = np.zeros((2, H, page), np.uint8)
    q4_ref.write(ref, x.double().numpy(), [2 * bs - 1, 0], bs, group)
    for d in (dk, dv):
        assert np.array_equal(d[-1].cpu().numpy(), ref[1]) and np.array_equal(d[0].cpu().numpy(), ref[0])
        assert int(d[1:-1].max()) == 0
    k = torch.empty_like(x).cuda()
    v = torch.empty_like(x).cuda()
    pa.pa_gather_q4(k, v, dk, dv, slots.cuda(), group_size=group)
    want = torch.from_numpy(q4_ref.values(ref, bs, hd, group)[[1, 0], :, [bs - 1, 0]]).to(x.dtype)
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)


@pytest.mark.gpu
def test_whole_blocks_copy_and_swap_as_bytes(pa):
    """Copy-on-write copies and swaps move 4-bit blocks through q4_block_rows."""
    rng = np.random.default_rng(3)
    kc = torch.from_numpy(rng.integers(0, 256, (6, 2, q4_ref.page_bytes(128, 16, 64)), dtype=np.uint8)).cuda()
    vc = kc.flip(0).contiguous()
    k0, v0 = kc.cpu(), vc.cpu()
    pa.pa_copy_blocks(pa.q4_block_rows(kc, 16), pa.q4_block_rows(vc, 16), torch.tensor([[1, 5], [2, 4]]).cuda())
    for c, was in ((kc, k0), (vc, v0)):
        assert torch.equal(c.cpu()[[5, 4]], was[[1, 2]]) and torch.equal(c.cpu()[:4], was[:4])
    hk, hv = torch.zeros_like(k0).pin_memory(), torch.zeros_like(k0).pin_memory()
    pa.pa_swap_blocks(pa.q4_block_rows(kc, 16), pa.q4_block_rows(vc, 16), pa.q4_block_rows(hk, 16),
                      pa.q4_block_rows(hv, 16), torch.tensor([[0, 3]]).cuda())
    torch.cuda.synchronize()
    assert torch.equal(hk[3], k0[0]) and torch.equal(hv[3], v0[0]) and int(hk[:3].max()) == 0


@pytest.mark.gpu
def test_write_on_another_stream_and_in_a_graph(pa):
    x = torch.randn(40, 2, 128, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    src = torch.zeros_like(x).cuda()
    kc = torch.zeros(5, 2, q4_ref.page_bytes(128, 16, 64), dtype=torch.uint8, device="cuda")
    vc, k, v = torch.zeros_like(kc), torch.zeros_like(src), torch.zeros_like(src)
    sm = torch.randperm(80, generator=torch.Generator().manual_seed(1))[:40].cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        pa.pa_reshape_and_cache_q4(src, src, kc, vc, sm)
        with torch.cuda.graph(graph, stream=side):
            pa.pa_reshape_and_cache_q4(src, src, kc, vc, sm)
            pa.pa_gather_q4(k, v, kc, vc, sm)
    torch.cuda.synchronize()
    src.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    ref = np.zeros(tuple(kc.shape), np.uint8)
    q4_ref.write(ref, x.double().numpy(), sm.cpu().numpy(), 16, 64)
    assert np.array_equal(kc.cpu().numpy(), ref) and np.array_equal(vc.cpu().numpy(), ref)
    s = sm.cpu().numpy()
    want = torch.from_numpy(q4_ref.values(ref, 16, 128, 64)[s // 16, :, s % 16]).to(x.dtype)
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("wrong,error", [
    (dict(k=torch.zeros(4, 2, 64, dtype=torch.float16)), TypeError), (dict(v=torch.zeros(4, 2, 64)), TypeError),
    (dict(v=torch.zeros(4, 2, 128, dtype=torch.bfloat16)), ValueError),
    (dict(slot_mapping=torch.zeros(4, dtype=torch.int32)), TypeError),
    (dict(slot_mapping=torch.zeros(3, dtype=torch.int64)), ValueError),
    (dict(k_cache=torch.zeros(3, 2, 640)), TypeError), (dict(v_cache=torch.zeros(2, 2, 640, dtype=torch.uint8)), ValueError),
    (dict(k=torch.zeros(4, 64, 2, dtype=torch.bfloat16).transpose(1, 2)), ValueError),
    (dict(k_cache=torch.zeros(3, 2, 641, dtype=torch.uint8), v_cache=torch.zeros(3, 2, 641, dtype=torch.uint8)), ValueError),
    (dict(k_cache=torch.zeros(3, 1, 640, dtype=torch.uint8), v_cache=torch.zeros(3, 1, 640, dtype=torch.uint8)), ValueError),
])
def test_binding_refuses_wrong_tensors(pa, wrong, error):
    a = dict(k=torch.zeros(4, 2, 64, dtype=torch.bfloat16), v=torch.zeros(4, 2, 64, dtype=torch.bfloat16),
             k_cache=torch.zeros(3, 2, 640, dtype=torch.uint8), v_cache=torch.zeros(3, 2, 640, dtype=torch.uint8),
             slot_mapping=torch.arange(4))
    a = {k: v.cuda() for k, v in a.items()}
    for fn in (pa.pa_reshape_and_cache_q4, pa.pa_gather_q4):
        fn(**a, group_size=32)
        with pytest.raises(error):
            fn(**{**a, **{k: v.cuda() for k, v in wrong.items()}}, group_size=32)
        with pytest.raises(ValueError):
            fn(**{**a, "v": a["v"].cpu()}, group_size=32)
        with pytest.raises(ValueError):
            fn(**a, group_size=48)
        with pytest.raises(TypeError):
            fn(**{**a, "k": None}, group_size=32)
    torch.cuda.synchronize()
