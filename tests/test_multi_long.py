"""Long contexts in every pass of pa_decode_tree and pa_decode_cross: CTAs that walk a hundred tiles of an item, past several
windows of looked-up pages, with shuffled tables, so that a page from the wrong place shows."""
import numpy as np
import pytest
import torch

import multi_gpu_ref
import multi_ref


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


@pytest.mark.gpu
@pytest.mark.parametrize("kind", multi_ref.KINDS)
@pytest.mark.parametrize("dtype,hd,bs", [(torch.bfloat16, 128, 16), (torch.bfloat16, 64, 32), (torch.float32, 128, 32),
                                         (torch.float32, 64, 16)])
@pytest.mark.parametrize("most,group", [(2, 1), (3, 4), (20, 2), (70, 4)])
def test_many_tiles_per_cta(pa, kind, dtype, hd, bs, most, group):
    """Six contexts of up to 60,000 tokens, 8 KV heads: 32,000 tiles of 64 tokens for at most 608 CTAs.  Rows within the bound
    of their type, bit-equal from call to call."""
    rng = np.random.default_rng(most + hd)
    Hkv, scale = 8, 2.0 * hd ** -0.5
    lens = [59_999, 60_000, 41_007, 128 * 300, 57_345, 33]
    news = [most, 1, most, most // 2, most, min(most, 33)]
    per = [-(-n // bs) for n in lens]
    nb = sum(per) + 5
    gen = torch.Generator(device="cuda").manual_seed(most)
    perm = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
    tables = torch.full((len(lens), max(per) + 1), 2**31 - 1, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(nb, Hkv, bs, hd, generator=gen, device="cuda").to(dtype) for _ in range(2))
    at = 0
    for i, p in enumerate(per):
        tables[i, :p] = perm[at:at + p]
        at += p
        last = tables[i, p - 1].long()
        for cache in (k, v):
            cache[last, :, (lens[i] - 1) % bs + 1:] = float("nan")
    k[perm[at:].long()] = v[perm[at:].long()] = float("nan")
    T = sum(news)
    q = torch.randn(T, Hkv * group, hd, generator=gen, device="cuda").to(dtype)
    start = np.concatenate([[0], np.cumsum(news)])
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    trees = [multi_ref.ancestors(multi_ref.random_tree(rng, c)) for c in news]
    mask = None
    if kind == "mask":
        words = -(-most // 64)
        mask = torch.from_numpy(np.concatenate([multi_ref.mask_words(s, words) for s in trees])).cuda()
    status = pa.DeviceStatus()
    args = q, k, v, tables, ctx, torch.from_numpy(start).to(torch.int32).cuda(), scale
    kw = dict(max_context_len=60_000, status=status)
    outs = []
    for _ in range(2):
        out = torch.empty_like(q)
        if kind == "cross":
            pa.pa_decode_cross(out, *args, **kw)
        else:
            pa.pa_decode_tree(out, *args, tree_mask=mask, **kw)
        outs.append(out)
    assert status.read() == 0 and torch.equal(*outs)
    for i, (n, c) in enumerate(zip(lens, news)):
        pages = tables[i, :per[i]].long()
        ki, vi = (x[pages].transpose(1, 2).reshape(-1, Hkv, hd)[:n] for x in (k, v))
        see = None
        if kind != "cross":
            see = torch.ones(c, n, dtype=torch.bool, device="cuda")
            see[:, n - c:] = torch.from_numpy(trees[i] if kind == "mask" else np.tri(c, dtype=bool)).cuda()
        rows = slice(int(start[i]), int(start[i + 1]))
        ref, spread, size, _ = multi_gpu_ref.attend(q[rows], ki, vi, scale, see)
        bound = (multi_gpu_ref.bf16_bound if dtype == torch.bfloat16 else multi_gpu_ref.f32_bound)(ref, spread, size, n, hd)
        assert ((outs[0][rows].double() - ref).abs() <= bound).all(), f"sequence {i}"
