"""Drafted steps as a serving loop runs them: trees planned, written, attended
to, accepted, moved and trimmed, step after step, with cross attention beside;
and the block manager's trim."""
import numpy as np
import pytest
import torch

import multi_ref
from helpers import assert_decode_close


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


# ------------------------------------------------------------- on the CPU ---

def test_trim_releases_the_blocks_past_the_end(pa):
    bm = pa.BlockManager(10, 16)
    bm.add_seq(0, 40)
    bm.append_slots([0] * 30)
    assert bm.num_tokens(0) == 70 and len(bm.block_table(0)) == 5
    blocks = bm.block_table(0)
    bm.trim_seq(0, 49)
    assert bm.block_table(0) == blocks[:4] and bm.num_free() == 6 and bm.num_tokens(0) == 49
    bm.trim_seq(0, 48)
    assert bm.block_table(0) == blocks[:3]
    slots, pairs = bm.append_slots([0])
    assert len(pairs) == 0 and int(slots[0]) == blocks[3] * 16     # the block released last comes back
    bm.trim_seq(0, 0)
    assert bm.block_table(0) == [] and bm.num_free() == 10
    bm.trim_seq(0, 0)


def test_trim_refuses_bad_requests(pa):
    bm = pa.BlockManager(4, 16)
    bm.add_seq(3, 20)
    for seq, n, code in ((3, 21, -1), (3, -1, -1), (4, 0, -6)):
        with pytest.raises(pa.PAError) as e:
            bm.trim_seq(seq, n)
        assert e.value.code == code
    assert bm.num_tokens(3) == 20


def test_trim_of_shared_and_keyed_blocks(pa):
    bm = pa.BlockManager(10, 4)
    tokens = list(range(12))
    bm.add_seq_cached(0, tokens)
    bm.fork(0, 1)
    bm.trim_seq(1, 6)                       # inside a block that sequence 0 holds too
    assert bm.refcount(bm.block_table(0)[1]) == 2 and bm.refcount(bm.block_table(0)[2]) == 1
    _, pairs = bm.append_slots([1])
    assert pairs.tolist() == [[bm.block_table(0)[1], bm.block_table(1)[1]]]
    bm.free_seq(1)
    # alone: the key goes when the block is written into, not before
    bm.trim_seq(0, 6)
    assert bm.add_seq_cached(2, tokens) == 12
    bm.free_seq(2)
    bm.append_slots([0, 0])
    assert bm.add_seq_cached(3, tokens) == 4
    bm.free_seq(0)
    bm.free_seq(3)
    assert bm.num_free() == 10


# ------------------------------------------------------------- on the GPU ---

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("chain", [False, True])
def test_drafted_steps_follow_a_plain_cache(pa, dtype, chain):
    """Every step's attention against fp64 over plain per-sequence lists of K/V rows,
    which keep the accepted rows only; the sequences grow through block edges."""
    from paged_kv_cache_237_gb300.engine import CrossDecodeStep, TreeDecodeStep
    rng = np.random.default_rng(5)
    g = torch.Generator().manual_seed(5)
    nb, bs, Hq, Hkv, hd, scale, most = 200, 16, 8, 2, 64, 0.12, 5
    kc, vc = (torch.full((nb, Hkv, bs, hd), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    enc = multi_ref.Batch("cross", [50, 1, 200], [1, 1, 1], Hq, Hkv, hd, bs, dtype, 6)
    enc_k, enc_v, enc_tables = enc.k.cuda(), enc.v.cuda(), torch.from_numpy(enc.tables).cuda()
    enc_lens = torch.tensor(enc.lens, dtype=torch.int32).cuda()
    bm, status = pa.BlockManager(nb, bs), pa.DeviceStatus()
    i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int64)).to(torch.int32).cuda()
    rows = {}
    for s, n in enumerate([14, 0, 95]):
        bm.add_seq(s, n)
        rows[s] = [torch.randn(n, Hkv, hd, generator=g).to(dtype) for _ in range(2)]
        ids = np.array(bm.block_table(s), np.int64)
        if n:
            slots = torch.from_numpy(ids[np.arange(n) // bs] * bs + np.arange(n) % bs).cuda()
            pa.pa_reshape_and_cache(rows[s][0].cuda(), rows[s][1].cuda(), kc, vc, slots, status=status)
    for step_no in range(6):
        news = [int(rng.integers(1, 20)) for _ in range(3)]
        if step_no == 3:
            news[0] = 0
        trees = [np.arange(-1, c - 1) if chain else multi_ref.random_tree(rng, c) for c in news]
        for s, c in enumerate(news):
            bm.append_slots([s] * c)
        ids, lens = bm.flat_blocks(range(3))
        T = sum(news)
        tables = torch.empty(3, 16, dtype=torch.int32, device="cuda")
        slots, start = torch.empty(T, dtype=torch.int64, device="cuda"), i32([0] * 4)
        positions, mask = torch.empty(T, dtype=torch.int32, device="cuda"), None
        pa.pa_build_tables(tables, slots, positions, start, ids.cuda(), lens.cuda(), i32(news), block_size=bs,
                           num_blocks=nb, status=status)
        parents = i32(np.concatenate(trees))
        if not chain:
            mask = torch.empty(T, 1, dtype=torch.int64, device="cuda")
            pa.pa_build_tree(mask, positions, parents, start, lens.cuda(), status=status)
        q, kn, vn = (torch.randn(T, h, hd, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
        max_len = int(lens.max())
        step = TreeDecodeStep(q.cuda(), kc, vc, tables, lens.cuda(), start, scale, max_len, tree_mask=mask,
                              status=status)
        out = step.run(kn.cuda(), vn.cuda(), slots).double().cpu()
        cross = CrossDecodeStep(q.cuda(), enc_k, enc_v, enc_tables, enc_lens, start, scale, 200, status=status).decode()
        draft, target = rng.integers(0, 3, size=T), rng.integers(0, 3, size=T)
        new = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
        taken, nodes, following, new_lens = new(3), new(3, most), new(3), new(3)
        pairs = torch.empty(3, most, 2, dtype=torch.int64, device="cuda")
        pa.pa_accept_tree(taken, nodes, following, new_lens, pairs, i32(draft), i32(target),
                          None if chain else parents, start, lens.cuda(), tables, block_size=bs, num_blocks=nb,
                          status=status)
        step.commit(pairs)
        assert status.read() == 0
        at = 0
        for s, c in enumerate(news):
            see = multi_ref.ancestors(trees[s])
            depth = see.sum(1) - 1
            have = len(rows[s][0])
            assert positions[at:at + c].tolist() == (have + depth).tolist()
            k = torch.cat([rows[s][0], kn[at:at + c]]).double().numpy()
            v = torch.cat([rows[s][1], vn[at:at + c]]).double().numpy()
            for r in range(c):
                w = np.concatenate([np.ones(have, bool), see[r]])
                ref = np.zeros((Hq, hd))
                for h in range(Hq):
                    x = scale * (k[w, h // 4] @ q[at + r, h].double().numpy())
                    e = np.exp(x - x.max())
                    ref[h] = e @ v[w, h // 4] / e.sum()
                assert_decode_close(out[at + r], torch.from_numpy(ref), dtype, what=f"step {step_no}")
            path = [r for r in nodes[s].tolist() if r >= 0]
            assert len(path) == taken[s].item() and new_lens[s].item() == have + len(path)
            rows[s] = [torch.cat([x, y[at:at + c][path]]) for x, y in zip(rows[s], (kn, vn))]
            bm.trim_seq(s, have + len(path))
            ids_s = np.array(bm.block_table(s) or [0], np.int64)
            p = np.arange(have + len(path))
            for cache, want in ((kc, rows[s][0]), (vc, rows[s][1])):
                assert torch.equal(cache[ids_s[p // bs], :, p % bs].cpu(), want)
            at += c
        enc.q, enc.news, enc.start = q, news, np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        assert_decode_close(cross, enc.reference(scale), dtype)


@pytest.mark.gpu
def test_steps_share_a_workspace_and_follow_their_attributes(pa):
    from paged_kv_cache_237_gb300.engine import CrossDecodeStep, TreeDecodeStep
    tree = multi_ref.Batch("mask", [900, 30], [30, 4], 8, 2, 128, 16, torch.bfloat16, 1)
    cross = multi_ref.Batch("cross", [500, 2000], [7, 50], 8, 2, 128, 16, torch.bfloat16, 2)
    ws = torch.empty(pa.pa_decode_tree_workspace_size(57, 8, 2, 128), dtype=torch.uint8, device="cuda")
    args = lambda b: (b.q.cuda(), b.k.cuda(), b.v.cuda(), torch.from_numpy(b.tables).cuda(),
                      torch.tensor(b.lens, dtype=torch.int32).cuda(), torch.from_numpy(b.start).cuda(), 0.1,
                      max(b.lens))
    a = TreeDecodeStep(*args(tree), tree_mask=tree.mask.cuda(), workspace=ws)
    c = CrossDecodeStep(*args(cross), workspace=ws)
    for _ in range(3):
        a.decode()
        c.decode()
    assert_decode_close(a.out, tree.reference(0.1), torch.bfloat16)
    assert_decode_close(c.out, cross.reference(0.1), torch.bfloat16)
    tree.kind = "chain"
    a.tree_mask = None
    assert_decode_close(a.decode(), tree.reference(0.1), torch.bfloat16)
    c.scale = 0.02
    assert_decode_close(c.decode(), cross.reference(0.02), torch.bfloat16)
    with pytest.raises(ValueError, match="workspace"):
        CrossDecodeStep(*args(cross), workspace=ws[:1000])


@pytest.mark.gpu
@pytest.mark.parametrize("width", [4, 30, 90])
def test_a_workspace_serves_decode_steps_too(pa, width):
    """pa_decode counts on the first bytes of its workspace from call to call."""
    from paged_kv_cache_237_gb300.engine import DecodeStep, TreeDecodeStep
    b = multi_ref.Batch("mask", [4000, 900, 30], [width, 30, 4], 8, 2, 128, 16, torch.bfloat16, 3)
    T = int(b.start[-1])
    q, k, v, tables = b.q.cuda(), b.k.cuda(), b.v.cuda(), torch.from_numpy(b.tables).cuda()
    lens = torch.tensor(b.lens, dtype=torch.int32).cuda()
    plain = DecodeStep(q[:3].contiguous(), k, v, tables, lens, 0.1, 4000)
    want = plain.decode().clone()
    need = max(pa.pa_decode_tree_workspace_size(T, 8, 2, 128), plain.workspace.numel())
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    ws[:256] = torch.arange(256, dtype=torch.uint8)
    tree = TreeDecodeStep(q, k, v, tables, lens, torch.from_numpy(b.start).cuda(), 0.1, 4000,
                          tree_mask=b.mask.cuda(), workspace=ws)
    tree.decode()
    assert torch.equal(ws[:256].cpu(), torch.arange(256, dtype=torch.uint8))
    ws[:256] = 0
    one = DecodeStep(q[:3].contiguous(), k, v, tables, lens, 0.1, 4000, workspace=ws)
    for _ in range(3):
        tree.decode()
        one.out.zero_()
        assert torch.equal(one.decode(), want)
    assert_decode_close(tree.decode(), b.reference(0.1), torch.bfloat16)
