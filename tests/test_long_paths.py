"""Accepted paths of more rows than one group of pa_move_rows holds."""
import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int64)).to(torch.int32).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,hd,limit", [(torch.float32, 128, 96), (torch.bfloat16, 128, 192), (torch.float32, 64, 192)])
@pytest.mark.parametrize("on", ["current", "side", "handle", "graph"])
def test_a_step_commits_every_path_that_can_be_accepted(pa, dtype, hd, limit, on):
    from paged_kv_cache_237_gb300.engine import TreeDecodeStep
    rng = np.random.default_rng(3)
    bs, Hkv, most, news, lens = 16, 2, 1024, [1000, 5, 700, 0], [1010, 5, 1500, 7]
    per = [-(-n // bs) for n in lens]
    nb = sum(per) + 1
    perm, tables, at = rng.permutation(nb), np.full((4, max(per)), -1, np.int64), 0
    for i, p in enumerate(per):
        tables[i, :p] = perm[at:at + p]
        at += p
    parents, target, draft = [], [], []
    for c in news:
        # a path that leaves out a node here and there, and with it everything that the nodes before did not skip
        kept = [0] if c else []
        for r in range(1, c):
            if rng.random() < 0.7:
                kept.append(r)
        par, tgt, drf = [-1] * c, list(rng.integers(0, 9, c)), [9] * c
        for a, b in zip(kept, kept[1:]):
            par[b], drf[b] = a, tgt[a]
        parents, target, draft = parents + par, target + tgt, draft + drf
    T = sum(news)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(nb, Hkv, bs, hd, generator=g).to(dtype) for _ in range(2))
    kc, vc = k.cuda(), v.cuda()
    start, ctx, tab = i32(np.concatenate([[0], np.cumsum(news)])), i32(lens), i32(tables)
    step = TreeDecodeStep(torch.zeros(T, 2, hd, dtype=dtype).cuda(), kc, vc, tab, ctx, start, 0.1, 1500)
    new = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    taken, nodes, following, new_lens = new(4), new(4, most), new(4), new(4)
    pairs = torch.empty(4, most, 2, dtype=torch.int64, device="cuda")
    pa.pa_accept_tree(taken, nodes, following, new_lens, pairs, i32(draft), i32(target), i32(parents), start, ctx, tab,
                      block_size=bs, num_blocks=nb, status=step.status)
    assert taken[0].item() > 2 * limit and taken[2].item() > limit
    torch.cuda.synchronize()
    with pytest.raises(pa.PAError):
        pa.pa_move_rows(kc, vc, pairs)
    if on == "graph":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step.commit(pairs)
        graph.replay()
    else:
        side = torch.cuda.Stream()
        step.commit(pairs, stream={"current": None, "side": side, "handle": side.cuda_stream}[on])
    torch.cuda.synchronize()
    assert step.status.read() == 0
    want = [k.clone(), v.clone()]
    for i, (n, c) in enumerate(zip(lens, news)):
        for j, r in enumerate(x for x in nodes[i].tolist() if x >= 0):
            s, d = n - c + r, n - c + j
            for x, y in zip((k, v), want):
                y[tables[i, d // bs], :, d % bs] = x[tables[i, s // bs], :, s % bs]
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


@pytest.mark.gpu
def test_wrong_pairs_are_refused(pa):
    from paged_kv_cache_237_gb300.engine import TreeDecodeStep
    k = torch.zeros(4, 1, 16, 128, device="cuda")
    step = TreeDecodeStep(torch.zeros(2, 1, 128, device="cuda"), k, k.clone(), i32([[0]]), i32([2]), i32([0, 2]), 0.1, 16)
    pairs = torch.full((1, 500, 2), -1, dtype=torch.int64, device="cuda")
    step.commit(pairs)
    for bad, error in ((pairs.int(), TypeError), (pairs[:, :, 0], ValueError), (pairs.cpu(), ValueError),
                       (pairs[:, ::2], ValueError), (pairs[:, :, :1].contiguous(), ValueError)):
        with pytest.raises(error):
            step.commit(bad)
