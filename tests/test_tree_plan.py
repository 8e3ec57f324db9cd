"""pa_build_tree, pa_accept_tree and pa_move_rows against plain Python."""
import numpy as np
import pytest
import torch

import multi_ref

FAKE = 0x10000


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int64)).to(torch.int32).cuda()


# ------------------------------------------------------------- on the CPU ---

def test_bad_arguments_are_refused_on_the_host(pa):
    L, F = pa._lib, FAKE
    assert L.pa_build_tree(F, F, F, F, F, -1, 4, 1, None, None) == -1
    assert L.pa_build_tree(F, F, F, F, F, 1, 4, 0, None, None) == -1
    assert L.pa_build_tree(F, F, F, F, F, 1, 4, 17, None, None) == -1
    assert L.pa_build_tree(None, F, F, F, F, 1, 4, 1, None, None) == -1
    assert L.pa_build_tree(F, F, None, F, F, 1, 4, 1, None, None) == -1
    assert L.pa_build_tree(F + 4, F, F, F, F, 1, 4, 1, None, None) == -1
    assert L.pa_build_tree(F, F + 1, F, F, F, 1, 4, 1, None, None) == -1
    assert L.pa_build_tree(None, None, None, None, None, 0, 4, 1, None, None) == 0
    assert L.pa_build_tree(None, None, None, None, None, 3, 0, 1, None, None) == 0

    def accept(ptrs=None, S=1, T=4, M=4, width=2, bs=16, nb=8):
        return L.pa_accept_tree(*(ptrs or [F] * 11), S, T, M, width, bs, nb, None, None)
    for kw in (dict(S=-1), dict(T=-1), dict(M=0), dict(M=1025), dict(width=0), dict(bs=0), dict(nb=0)):
        assert accept(**kw) == -1
    for k in range(11):
        if k == 7:      # parents may be NULL
            continue
        assert accept([None if j == k else F for j in range(11)]) == -1
        assert accept([F + 2 if j == k else F for j in range(11)]) == -1
    assert accept([F + 4 if j == 4 else F for j in range(11)]) == -1
    assert accept([None] * 11, S=0) == 0

    def move(k=F, v=F, pairs=F, groups=1, per=4, heads=2, hd=128, bs=16, nb=8, dtype=1):
        return L.pa_move_rows(k, v, pairs, groups, per, heads, hd, bs, nb, dtype, None, None)
    for kw in (dict(k=None), dict(v=None), dict(pairs=None), dict(k=F + 8), dict(pairs=F + 4), dict(groups=-1),
               dict(per=-1), dict(heads=0), dict(hd=0), dict(bs=0), dict(nb=0), dict(dtype=5)):
        assert move(**kw) == -1
    for kw in (dict(hd=4), dict(per=193), dict(per=97, dtype=0), dict(heads=65536)):
        assert move(**kw) == -2
    assert move(groups=0) == 0 and move(per=0) == 0


def test_masks_past_32_bits_are_refused(pa):
    L, F = pa._lib, FAKE
    assert L.pa_build_tree(F, F, F, F, F, 1, 2**26, 16, None, None) == -2
    assert L.pa_build_tree(F, F, F, F, F, 1, 2**31 - 1, 1, None, None) == -2


# ------------------------------------------------------------- on the GPU ---

def layout(news, padding=0):
    return np.concatenate([[0], np.cumsum(news)]), int(sum(news)) + padding


@pytest.mark.gpu
@pytest.mark.parametrize("news,words", [([1], 1), ([5, 0, 64, 1], 1), ([65, 3, 128], 2), ([300, 1, 0, 17], 5),
                                        ([1024, 1000], 16), ([7] * 700, 1)])
def test_masks_and_positions(pa, news, words):
    rng = np.random.default_rng(len(news))
    start, T = layout(news, padding=4)
    trees = [multi_ref.random_tree(rng, c) for c in news]
    if news[0] > 3:
        trees[0][3] = -1           # a forest
        trees[0][1:3] = [0, 1]
    lens = [c + int(rng.integers(0, 50)) for c in news]
    parents = np.concatenate([*trees, np.full(4, 77)])
    mask = torch.full((T, words), 9, dtype=torch.int64, device="cuda")
    pos = torch.full((T,), 9, dtype=torch.int32, device="cuda")
    status = pa.DeviceStatus()
    pa.pa_build_tree(mask, pos, i32(parents), i32(start), i32(lens), status=status)
    see = [multi_ref.ancestors(t) for t in trees]
    want = np.concatenate([multi_ref.mask_words(s, words) for s in see])
    depth = np.concatenate([n - c + s.sum(1) - 1 for n, c, s in zip(lens, news, see)])
    assert status.read() == 0
    assert np.array_equal(mask.cpu().numpy()[:-4], want) and (mask[-4:] == 9).all()
    assert np.array_equal(pos.cpu().numpy()[:-4], depth) and (pos[-4:] == 9).all()
    again = torch.zeros_like(mask)
    pa.pa_build_tree(again, None, i32(parents), i32(start), i32(lens))
    assert torch.equal(again[:-4], mask[:-4])


@pytest.mark.gpu
def test_bad_trees_are_flagged(pa):
    def run(parents, start, lens, words=1):
        T = len(parents)
        mask, pos = torch.zeros(T, words, dtype=torch.int64, device="cuda"), torch.zeros(T, dtype=torch.int32).cuda()
        status = pa.DeviceStatus()
        pa.pa_build_tree(mask, pos, i32(parents), i32(start), i32(lens), status=status)
        return mask.cpu(), pos.cpu(), status.read()
    for p in (1, 2, -2, 2**31 - 1, -2**31):        # not an earlier node: none
        mask, pos, flags = run([-1, p, 0], [0, 3], [10])
        assert flags == pa.STATUS_BAD_TREE
        assert mask[:, 0].tolist() == [1, 2, 5] and pos.tolist() == [7, 7, 8]
    mask, pos, flags = run([-1] + list(range(69)), [0, 70], [70])       # more nodes than the mask holds
    assert flags == pa.STATUS_BAD_TREE
    assert mask[63].item() == -1 and (mask[64:] == 0).all() and pos[63].item() == 63
    mask, _, flags = run([-1, 0, 1], [0, 4], [9])                          # rows outside the batch
    assert flags == pa.STATUS_BAD_TREE and (mask == 0).all()
    mask, _, flags = run([-1, 0, 1], [0, 3], [2])                          # more nodes than tokens
    assert flags == pa.STATUS_BAD_CONTEXT_LEN and (mask == 0).all()


def accept_batch(pa, news, lens, parents, draft, target, most, bs, tables, nb, chain=False):
    start, T = layout(news)
    S = len(news)
    new = lambda *s: torch.full(s, 99, dtype=torch.int32, device="cuda")
    outs = [new(S), new(S, most), new(S), new(S), torch.full((S, most, 2), 99, dtype=torch.int64, device="cuda")]
    status = pa.DeviceStatus()
    pa.pa_accept_tree(*outs, i32(draft), i32(target), None if chain else i32(parents), i32(start), i32(lens),
                      i32(tables), block_size=bs, num_blocks=nb, status=status)
    return [o.cpu().tolist() for o in outs], status.read()


@pytest.mark.gpu
@pytest.mark.parametrize("news,most,bs", [([1], 1, 16), ([9, 0, 30, 1], 8, 16), ([200, 64, 3], 40, 32),
                                          ([1024, 5], 1024, 16), ([12] * 500, 6, 16)])
@pytest.mark.parametrize("chain", [False, True])
def test_accepted_paths(pa, news, most, bs, chain):
    rng = np.random.default_rng(most + len(news))
    start, T = layout(news)
    trees = [np.arange(-1, c - 1) if chain else multi_ref.random_tree(rng, c) for c in news]
    lens = [c + int(rng.integers(0, 3 * bs)) for c in news]
    width = max(1, -(-max(lens) // bs))
    nb = len(news) * width + 1
    tables = rng.permutation(nb)[:len(news) * width].reshape(len(news), width)
    # few tokens, so that siblings share them and several children agree
    draft, target = rng.integers(0, 3, size=T), rng.integers(0, 3, size=T)
    if chain:
        target[:-1] = np.where(rng.random(T - 1) < 0.9, draft[1:], target[:-1])
    outs, flags = accept_batch(pa, news, lens, np.concatenate(trees), draft, target, most, bs, tables, nb, chain)
    assert flags == 0
    for i, c in enumerate(news):
        a = slice(start[i], start[i + 1])
        want = multi_ref.accept(lens[i], c, draft[a], target[a], trees[i], most,
                                lambda p: int(tables[i, p // bs]) * bs + p % bs)
        got = tuple(o[i] for o in outs)
        assert (got[0], got[1], got[2], got[3], [tuple(x) for x in got[4]]) == want


@pytest.mark.gpu
def test_bad_acceptances_are_flagged(pa):
    tables = [[0, 1], [2, 3]]
    base = dict(news=[4, 4], lens=[20, 20], parents=[-1, 0, 0, 2] * 2, draft=[5, 6, 7, 8] * 2, target=[7, 1, 8, 2] * 2,
                most=4, bs=16, tables=tables, nb=4)
    outs, flags = accept_batch(pa, **base)
    assert flags == 0 and outs[0] == [3, 3] and outs[1][0] == [0, 2, 3, -1] and outs[2] == [2, 2]
    assert outs[3] == [19, 19] and outs[4][1] == [[-1, -1], [50, 49], [51, 50], [-1, -1]]
    good = [o[1] for o in outs]
    for change, flag in ((dict(lens=[3, 20]), pa.STATUS_BAD_CONTEXT_LEN), (dict(lens=[33, 20]),
                                                                           pa.STATUS_BAD_CONTEXT_LEN)):
        outs, flags = accept_batch(pa, **{**base, **change})
        assert flags == flag and [o[0] for o in outs][:4] == [0, [-1] * 4, -1, change["lens"][0]]
        assert [o[1] for o in outs] == good
    outs, flags = accept_batch(pa, **{**base, "tables": [[0, 9], [2, 3]]})
    assert flags == pa.STATUS_BAD_BLOCK_ID and outs[0] == [3, 3] and outs[4][0] == [[-1, -1]] * 4
    outs, flags = accept_batch(pa, **{**base, "parents": [-1, 0, 2, 2] + [-1, 0, 0, 2]})
    assert flags == pa.STATUS_BAD_TREE and outs[0] == [1, 3]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,hd,Hkv,bs", [(torch.bfloat16, 128, 8, 16), (torch.float32, 64, 3, 32),
                                             (torch.bfloat16, 8, 1, 16)])
@pytest.mark.parametrize("groups,per", [(1, 1), (3, 7), (200, 12), (1, 96)])
def test_rows_move_as_if_at_once(pa, dtype, hd, Hkv, bs, groups, per):
    rng = np.random.default_rng(per)
    nb = -(-groups * per * 2 // bs) + 2
    g = torch.Generator().manual_seed(per)
    k, v = (torch.randn(nb, Hkv, bs, hd, generator=g).to(dtype) for _ in range(2))
    slots = rng.permutation(nb * bs)[:groups * per * 2].reshape(groups, 2 * per)
    pairs = np.full((groups, per, 2), -1, np.int64)
    for i in range(groups):
        own = slots[i]
        pairs[i, :, 1] = own[:per]
        pairs[i, :, 0] = rng.choice(own, size=per)      # sources that are destinations too, and repeats
        skip = rng.random(per) < 0.2
        pairs[i, skip, rng.integers(0, 2)] = -1
    want = [k.clone(), v.clone()]
    for x, y in zip((k, v), want):
        for s, d in pairs.reshape(-1, 2).tolist():
            if s >= 0 and d >= 0:
                y[d // bs, :, d % bs] = x[s // bs, :, s % bs]
    kc, vc = k.cuda(), v.cuda()
    status = pa.DeviceStatus()
    pa.pa_move_rows(kc, vc, torch.from_numpy(pairs).cuda(), status=status)
    assert status.read() == 0
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


@pytest.mark.gpu
def test_bad_slots_are_flagged_and_skipped(pa):
    k = torch.arange(4 * 16 * 8, dtype=torch.float32).view(4, 1, 16, 8).cuda()
    kc, vc = k.clone(), k.clone()
    pairs = torch.tensor([[[3, 64], [2**62, 5], [7, 8]]], dtype=torch.int64).cuda()
    status = pa.DeviceStatus()
    pa.pa_move_rows(kc, vc, pairs, status=status)
    assert status.read() == pa.STATUS_BAD_SLOT
    want = k.clone()
    want[0, :, 8] = k[0, :, 7]
    assert torch.equal(kc, want) and torch.equal(vc, want)
    with pytest.raises(ValueError):
        pa.pa_move_rows(kc, vc, pairs[0])
    with pytest.raises(TypeError):
        pa.pa_move_rows(kc, vc, pairs.int())
