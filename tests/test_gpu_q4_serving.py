"""The 4-bit cache, the batch tables and the windowed decode as a serving loop uses
them together: prompts prefilled in chunks and decoded on, tables and slots
laid out on the GPU from the block manager's flat lists, forks with
copy-on-write, requests ending and arriving.  The numpy format and fp64
attention (q4_ref.py) follow step by step: caches must be equal byte for byte,
outputs within the tolerances of test_q4_decode.py and helpers.py."""
import numpy as np
import pytest
import torch

import q4_ref
from helpers import assert_decode_close

pytestmark = pytest.mark.gpu

NB, BS, HQ, HKV, HD, G = 120, 16, 8, 2, 128, 64
SCALE = HD ** -0.5


class Batch:
    """Tables and slots of a list of sequences, laid out on the GPU."""

    def __init__(self, pa, bm, seqs, new, width=16, pad=3):
        flat, lens = bm.flat_blocks(seqs)
        T = sum(new) + pad
        self.tables = torch.empty(len(seqs), width, dtype=torch.int32, device="cuda")
        self.slots = torch.empty(T, dtype=torch.int64, device="cuda")
        self.positions = torch.empty(T, dtype=torch.int32, device="cuda")
        self.starts = torch.empty(len(seqs) + 1, dtype=torch.int32, device="cuda")
        self.lens_h, self.lens = lens, lens.cuda()
        pa.pa_build_tables(self.tables, self.slots, self.positions, self.starts, flat.cuda(), self.lens,
                           torch.tensor(new, dtype=torch.int32).cuda(), block_size=BS, num_blocks=NB)
        want, _ = bm.build_tables(seqs, width)
        assert torch.equal(self.tables.cpu(), want)


def rows(gen, T, dtype):
    return torch.randn(T, HKV, HD, generator=gen).to(dtype)


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_serving_loop_over_a_four_bit_cache(dtype, window, sinks):
    from paged_kv_cache_237_gb300 import binding as pa
    from paged_kv_cache_237_gb300.engine import Q4DecodeStep
    gen = torch.Generator().manual_seed(3)
    rng = np.random.default_rng(3)
    page = q4_ref.page_bytes(HD, BS, G)
    kc_h, vc_h = (rng.integers(0, 256, (NB, HKV, page), dtype=np.uint8) for _ in range(2))
    kc, vc = torch.from_numpy(kc_h).cuda(), torch.from_numpy(vc_h).cuda()
    bm, status = pa.BlockManager(NB, BS), pa.DeviceStatus()
    live, nxt = [], 0

    def write(k, v, slots):
        for cache, x in ((kc_h, k), (vc_h, v)):
            q4_ref.write(cache, x.double().numpy(), slots.cpu().numpy(), BS, G)

    def admit(n):
        """A prompt of n tokens, prefilled in one padded chunk."""
        nonlocal nxt
        bm.add_seq(nxt, n)
        b = Batch(pa, bm, [nxt], [n])
        k, v = rows(gen, n + 3, dtype), rows(gen, n + 3, dtype)
        pa.pa_reshape_and_cache_q4(k.cuda(), v.cuda(), kc, vc, b.slots, group_size=G, status=status)
        write(k, v, b.slots)
        back = torch.empty(n + 3, HKV, HD, device="cuda")
        pa.pa_gather_q4(back, torch.empty_like(back), kc, vc, b.slots, group_size=G, status=status)
        held = q4_ref.values(kc_h, BS, HD, G)
        s = b.slots.cpu().numpy()[:n]
        assert torch.equal(back.cpu()[:n], torch.from_numpy(held[s // BS, :, s % BS]).float())
        assert b.positions.cpu().tolist() == list(range(n)) + [0] * 3
        live.append(nxt)
        nxt += 1

    for n in (1, 16, 37, 200):
        admit(n)
    for step in range(5):
        if step == 1:                       # parallel samples share their last, partial block
            bm.fork(live[2], nxt)
            live.append(nxt)
            nxt += 1
        if step == 3:
            bm.free_seq(live.pop(0))
            admit(65)
        slots_h, pairs = bm.append_slots(live)
        b = Batch(pa, bm, live, [1] * len(live))
        n = len(live)
        assert torch.equal(b.slots.cpu()[:n], slots_h) and (b.slots.cpu()[n:] == -1).all()
        assert (step == 1) == (pairs.numel() > 0)
        q = torch.randn(n, HQ, HD, generator=gen).to(dtype)
        k, v = rows(gen, n + 3, dtype), rows(gen, n + 3, dtype)
        d = Q4DecodeStep(q.cuda(), kc, vc, b.tables, b.lens, SCALE, int(b.lens_h.max()), 64 if step % 2 else 0,
                         group_size=G, window=window, num_sinks=sinks, status=status)
        out = d.run(k.cuda(), v.cuda(), b.slots, pairs.cuda())
        torch.cuda.synchronize()
        assert status.read() == 0
        for src, dst in pairs.tolist():
            kc_h[dst], vc_h[dst] = kc_h[src], vc_h[src]
        write(k, v, b.slots)
        assert np.array_equal(kc.cpu().numpy(), kc_h) and np.array_equal(vc.cpu().numpy(), vc_h)
        with np.errstate(invalid="ignore"):
            kv, vv = q4_ref.values(kc_h, BS, HD, G), q4_ref.values(vc_h, BS, HD, G)
        used = np.unique(np.concatenate([bm.block_table(s) for s in live]))
        mine = np.zeros(NB, bool)
        mine[used] = True                   # the rest of the pool holds arbitrary bytes
        ref = torch.from_numpy(q4_ref.attend(q.double().numpy(), kv, vv, b.tables.cpu().numpy(), b.lens_h.numpy(),
                                             SCALE, BS, window, sinks))
        assert torch.isfinite(ref).all()
        assert_decode_close(out, ref, dtype, what=f"step {step}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_windowed_loop_gives_blocks_back(dtype):
    """A decode loop with a window over an unquantised cache: blocks that the
    window has left are dropped from the flat list's table and their memory is
    overwritten with NaN, and every step still matches fp64 attention."""
    from paged_kv_cache_237_gb300 import binding as pa
    from paged_kv_cache_237_gb300.engine import DecodeStep
    gen = torch.Generator().manual_seed(5)
    window, sinks, lens = 40, 5, [30, 100, 61]
    kc = torch.randn(NB, HKV, BS, HD, generator=gen).to(dtype)
    vc = torch.randn(NB, HKV, BS, HD, generator=gen).to(dtype)
    bm = pa.BlockManager(NB, BS)
    for i, n in enumerate(lens):
        bm.add_seq(i, n)
    kd, vd, status = kc.cuda(), vc.cuda(), pa.DeviceStatus()
    for step in range(20):
        bm.append_slots([0, 1, 2])
        b = Batch(pa, bm, [0, 1, 2], [1, 1, 1], width=10, pad=0)
        tables = b.tables.cpu()
        for i, n in enumerate(b.lens_h.tolist()):
            for j in range(-(-n // BS)):
                if j * BS >= sinks and j * BS + BS <= n - window:      # nothing of it is visible any more
                    kc[tables[i, j]] = vc[tables[i, j]] = float("nan")
                    kd[tables[i, j]] = vd[tables[i, j]] = float("nan")
                    tables[i, j] = -1
        q = torch.randn(3, HQ, HD, generator=gen).to(dtype)
        k, v = rows(gen, 3, dtype), rows(gen, 3, dtype)
        d = DecodeStep(q.cuda(), kd, vd, tables.cuda(), b.lens, SCALE, int(b.lens_h.max()), window=window,
                       num_sinks=sinks, status=status, partition_size=16 if step % 2 else 0)
        out = d.run_fused(k.cuda(), v.cuda(), b.slots)
        torch.cuda.synchronize()
        assert status.read() == 0
        s = b.slots.cpu()
        kc[s // BS, :, s % BS], vc[s // BS, :, s % BS] = k, v
        ref = torch.from_numpy(q4_ref.attend(q.double().numpy(), kc.double().numpy(), vc.double().numpy(),
                                             tables.numpy(), b.lens_h.numpy(), SCALE, BS, window, sinks))
        assert_decode_close(out, ref, dtype, what=f"step {step}")
    assert (tables == -1).any()
