"""pa_build_tables and pa_bm_flat_blocks against a plain loop and the host block
manager; everything is integers and must be equal."""
import numpy as np
import pytest
import torch

FAKE = 0x10000


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


def plain(ids, lens, news, bs, width, T, num_blocks):
    """The header's formulas, one element at a time; returns the outputs and the expected flags."""
    S = len(lens)
    tables = np.full((S, width), -1, np.int32)
    slots, pos, qs = np.full(T, -1, np.int64), np.zeros(T, np.int32), np.zeros(S + 1, np.int32)
    flags, first, start = 0, 0, 0

    def block(at):
        nonlocal flags
        if at >= len(ids):
            flags |= 32
            return -1
        if not 0 <= ids[at] < num_blocks:
            flags |= 1
            return -1
        return int(ids[at])

    for i in range(S):
        n = min(max(int(lens[i]), 0), width * bs)
        c = min(max(int(news[i]), 0), n)
        if n != lens[i] or c != news[i]:
            flags |= 2
        nb = -(-n // bs)
        for j in range(nb):
            tables[i, j] = block(first + j)
        qs[i] = start
        for r in range(c):
            if start + r >= T:
                flags |= 32
                break
            p = n - c + r
            b = block(first + p // bs)
            slots[start + r] = -1 if b < 0 else b * bs + p % bs
            pos[start + r] = p
        first += nb
        start += c
    qs[S] = start
    return tables, slots, pos, qs, flags


# ------------------------------------------------------------- on the CPU ---

@pytest.mark.parametrize("change,code", [
    (dict(S=-1), -1), (dict(width=0), -1), (dict(T=-1), -1), (dict(N=-1), -1), (dict(bs=0), -1), (dict(nb=0), -1),
    (dict(tables=None), -1), (dict(slots=None), -1), (dict(ids=None), -1), (dict(lens=None), -1),
    (dict(news=None), -1), (dict(slots=FAKE + 4), -1), (dict(pos=FAKE + 2), -1), (dict(ids=FAKE + 1), -1),
])
def test_bad_arguments_are_refused_on_the_host(pa, change, code):
    a = dict(tables=FAKE, slots=FAKE, pos=FAKE, qs=FAKE, ids=FAKE, lens=FAKE, news=FAKE, S=2, width=4, T=5, N=6,
             bs=16, nb=8, status=None, stream=None)
    a.update(change)
    assert pa._lib.pa_build_tables(*a.values()) == code
    assert b"pa_build_tables" in pa._lib.pa_last_error_string()


def test_binding_refuses_cpu_tensors(pa):
    i32, i64 = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        pa.pa_build_tables(torch.zeros(2, 3, dtype=torch.int32), i64, None, None, i32, i32, i32, block_size=16,
                           num_blocks=4)
    with pytest.raises(TypeError):
        pa.pa_build_tables(None, i64, None, None, i32, i32, i32, block_size=16, num_blocks=4)


@pytest.mark.gpu
@pytest.mark.parametrize("wrong,error", [
    (dict(block_tables=torch.zeros(2, 3)), TypeError), (dict(slot_mapping=torch.zeros(4, dtype=torch.int32)), TypeError),
    (dict(positions=torch.zeros(4)), TypeError), (dict(block_ids=torch.zeros(2, 2, dtype=torch.int32)), ValueError),
    (dict(context_lens=torch.zeros(3, dtype=torch.int32)), ValueError), (dict(new_lens=torch.zeros(2, 1, dtype=torch.int32)), ValueError),
    (dict(query_start=torch.zeros(2, dtype=torch.int32)), ValueError), (dict(positions=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(block_tables=torch.zeros(6, dtype=torch.int32)), ValueError),
    (dict(slot_mapping=torch.zeros(4, 1, dtype=torch.int64)), ValueError),
    (dict(block_tables=torch.zeros(3, 2, dtype=torch.int32).t()), ValueError),
])
def test_binding_refuses_wrong_tensors(pa, wrong, error):
    a = dict(block_tables=torch.zeros(2, 3, dtype=torch.int32), slot_mapping=torch.zeros(4, dtype=torch.int64),
             positions=torch.zeros(4, dtype=torch.int32), query_start=torch.zeros(3, dtype=torch.int32),
             block_ids=torch.zeros(2, dtype=torch.int32), context_lens=torch.zeros(2, dtype=torch.int32),
             new_lens=torch.zeros(2, dtype=torch.int32))
    a = {k: v.cuda() for k, v in a.items()}
    pa.pa_build_tables(**a, block_size=16, num_blocks=4)
    a.update({k: v.cuda() for k, v in wrong.items()})
    with pytest.raises(error):
        pa.pa_build_tables(**a, block_size=16, num_blocks=4)
    a["context_lens"] = torch.zeros(2, dtype=torch.int32)          # on the CPU
    with pytest.raises((ValueError, TypeError)):
        pa.pa_build_tables(**a, block_size=16, num_blocks=4)
    torch.cuda.synchronize()


def test_flat_blocks_lists_every_sequence_in_order(pa):
    bm = pa.BlockManager(40, 16)
    for s, n in ((5, 33), (2, 16), (9, 1)):
        bm.add_seq(s, n)
    bm.fork(5, 6)
    ids, lens = bm.flat_blocks([9, 5, 6, 2])
    assert lens.tolist() == [1, 33, 33, 16]
    assert ids.tolist() == bm.block_table(9) + bm.block_table(5) + bm.block_table(6) + bm.block_table(2)
    none, zero = bm.flat_blocks([])
    assert none.numel() == 0 and zero.numel() == 0
    with pytest.raises(pa.PAError):
        bm.flat_blocks([77])
    assert pa._lib.pa_bm_flat_blocks(bm._h, torch.tensor([5], dtype=torch.int32).data_ptr(), 1,
                                     ids.data_ptr(), 2, None) == -1     # out holds 2, 3 are needed


# ------------------------------------------------------------- on the GPU ---

def run(pa, ids, lens, news, bs, width, T, num_blocks, optional=True):
    i32 = lambda a: torch.tensor(np.asarray(a, np.int32)).cuda()
    S = len(lens)
    tables = torch.full((S, width), 99, dtype=torch.int32, device="cuda")
    slots = torch.full((T,), 99, dtype=torch.int64, device="cuda")
    pos = torch.full((T,), 99, dtype=torch.int32, device="cuda") if optional else None
    qs = torch.full((S + 1,), 99, dtype=torch.int32, device="cuda") if optional else None
    status = pa.DeviceStatus()
    pa.pa_build_tables(tables, slots, pos, qs, i32(ids), i32(lens), i32(news), block_size=bs, num_blocks=num_blocks,
                       status=status)
    torch.cuda.synchronize()
    back = [x.cpu().numpy() if x is not None else None for x in (tables, slots, pos, qs)]
    return (*back, status.read())


def same(got, want):
    for g, w in zip(got, want):
        if g is not None:
            assert np.array_equal(g, w)


def batch(S, max_len, max_new, bs, seed):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, max_len + 1, size=S)
    news = np.minimum(lens, rng.integers(0, max_new + 1, size=S))
    blocks = int((-(-lens // bs)).sum())
    return rng.permutation(blocks + 5)[:blocks], lens, news, blocks + 5


@pytest.mark.gpu
@pytest.mark.parametrize("S,max_len,max_new,bs,pad", [
    (1, 1, 1, 16, 0), (1, 40000, 40000, 16, 3), (7, 100, 1, 32, 0), (64, 2048, 1, 16, 17), (257, 300, 300, 16, 1000),
    (1500, 90, 90, 16, 5), (3, 50, 50, 1, 2), (5, 70, 70, 24, 0), (2500, 3, 1, 32, 1),
])
def test_tables_equal_the_plain_loop(pa, S, max_len, max_new, bs, pad):
    ids, lens, news, nb = batch(S, max_len, max_new, bs, S)
    width = max(1, -(-int(lens.max()) // bs)) + pad % 4
    T = int(news.sum()) + pad
    want = plain(ids, lens, news, bs, width, T, nb)
    got = run(pa, ids, lens, news, bs, width, T, nb)
    same(got[:4], want[:4])
    assert got[4] == 0 and want[4] == 0
    same(run(pa, ids, lens, news, bs, width, T, nb, optional=False)[:2], want[:2])


@pytest.mark.gpu
def test_empty_batches_and_rows(pa):
    got = run(pa, [], [], [], 16, 4, 5, 3)
    assert got[0].shape == (0, 4) and (got[1] == -1).all() and (got[2] == 0).all() and got[3].tolist() == [0]
    got = run(pa, [], [0, 0, 0], [0, 0, 0], 16, 2, 3, 3)
    assert (got[0] == -1).all() and (got[1] == -1).all() and got[3].tolist() == [0, 0, 0, 0] and got[4] == 0
    got = run(pa, [2, 1], [0, 17, 0], [0, 2, 0], 16, 2, 0 + 2, 3)
    assert got[0].tolist() == [[-1, -1], [2, 1], [-1, -1]] and got[1].tolist() == [47, 16] and got[4] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("what,flag", [("long", 2), ("negative", 2), ("new", 2), ("minus", 2), ("id", 1),
                                       ("idneg", 1), ("short", 32), ("rows", 32)])
def test_bad_data_is_flagged_and_stays_inside_the_buffers(pa, what, flag):
    bs, width = 16, 4
    lens, news = np.array([20, 64, 5, 33]), np.array([3, 1, 5, 33])
    ids = np.arange(3 * 4)[: 2 + 4 + 1 + 3][::-1].copy()
    T, nb = int(news.sum()) + 4, 12
    if what == "long":
        lens[1] = 2**31 - 1
    elif what == "negative":
        lens[1] = -7
    elif what == "new":
        news[2] = 2**31 - 1
    elif what == "minus":
        news[2] = -2**31
    elif what == "id":
        ids[3] = nb
    elif what == "idneg":
        ids[-1] = -1
    elif what == "short":
        ids = ids[:-2]
    elif what == "rows":
        T = 30
    want = plain(ids, lens, news, bs, width, T, nb)
    got = run(pa, ids, lens, news, bs, width, T, nb)
    assert want[4] == flag and got[4] == flag
    same(got[:4], want[:4])


@pytest.mark.gpu
def test_tables_equal_the_host_block_manager(pa):
    """A serving loop's batch: the device tables equal pa_bm_build_tables, and the
    slots those of append_slots, step after step, replayed from one graph."""
    bm = pa.BlockManager(300, 16)
    rng = np.random.default_rng(5)
    seqs = list(range(12))
    for s in seqs:
        bm.add_seq(s, int(rng.integers(1, 200)))
    width, cap = 20, 240
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, lens, news = torch.zeros(cap, **i32), torch.zeros(12, **i32), torch.ones(12, **i32)
    tables, pos, qs = torch.zeros(12, width, **i32), torch.zeros(16, **i32), torch.zeros(13, **i32)
    slots = torch.zeros(16, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    call = lambda: pa.pa_build_tables(tables, slots, pos, qs, ids, lens, news, block_size=16, num_blocks=300)
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for _ in range(20):
        want_slots, pairs = bm.append_slots(seqs)
        assert pairs.numel() == 0
        want, want_lens = bm.build_tables(seqs, width)
        flat, flat_lens = bm.flat_blocks(seqs)
        assert torch.equal(flat_lens, want_lens)
        ids[:len(flat)] = flat.cuda()
        lens.copy_(flat_lens)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tables.cpu(), want)
        assert torch.equal(slots.cpu()[:12], want_slots) and (slots.cpu()[12:] == -1).all()
        assert torch.equal(pos.cpu()[:12], want_lens - 1) and qs.cpu().tolist() == list(range(13))
