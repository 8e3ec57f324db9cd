"""The weights of pa_decode_tree and pa_decode_cross over bf16 caches have two bf16 parts in every pass: beyond the
rounding of its result a row is off by 2^-16 or so of its values, whatever its weights and whatever shares its batch."""
import numpy as np
import pytest
import torch

import multi_gpu_ref
import multi_ref
from multi_ref import Batch


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


# (most queries, query heads, KV heads, copies): few rows per sequence, up to 128, more than that.  With the copies a CTA
# walks some twenty tiles: what a weight is held in may not depend on what its row has seen before.
ROWS = [(2, 4, 2, 60), (40, 2, 2, 60), (60, 16, 2, 12)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", multi_ref.KINDS)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("most,Hq,Hkv,times", ROWS)
def test_results_are_off_by_their_rounding_and_little_more(pa, kind, hd, most, Hq, Hkv, times):
    lens = [3000, 1, 129, 2000, 600]
    b = Batch(kind, lens, [most, 1, most, most // 2, most], Hq, Hkv, hd, 16, torch.bfloat16, most + hd)
    scale = hd ** -0.5
    out, spread, size, _ = multi_gpu_ref.batch(b, scale)
    bound = multi_gpu_ref.bf16_bound(out, spread, size, max(lens), hd)
    got, flags = multi_gpu_ref.repeated(b, times).on_gpu(pa, scale)
    assert flags == 0
    assert ((got.double().unflatten(0, (times, -1)) - out).abs() <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("most,Hq,Hkv,times", ROWS)
def test_weights_that_are_alike_give_their_values_mean(pa, hd, most, Hq, Hkv, times):
    """Every 64th token above the others, whose weight e^-s is as far from a bf16 value as can be; every value is
    255 / 128, and so is the result: 2^-16 of it is less than half a step."""
    n = 4096
    grid = torch.arange(128, 256, dtype=torch.float64) / 256                       # bf16 values of [0.5, 1)
    s = grid[:, None] * (grid + 0.5)[None, :].to(torch.bfloat16).double()          # products are exact in fp32
    w = torch.exp(-s)
    off = (w.to(torch.bfloat16).double() - w) / w
    i, j = divmod(int(off.abs().argmax()), 128)
    assert off.abs().max() > 0.95 * 2 ** -8
    b = Batch("cross", [n], [most], Hq, Hkv, hd, 16, torch.bfloat16, 9)
    b.q.zero_()
    b.q[..., 0] = grid[i].to(torch.bfloat16)
    b.k.masked_fill_(~b.k.isnan(), 0.0)
    b.k[torch.from_numpy(b.tables[0, ::4]).long(), :, 0, 0] = (grid[j] + 0.5).to(torch.bfloat16)
    b.v.masked_fill_(~b.v.isnan(), 255 / 128)
    out = multi_gpu_ref.repeated(b, times).on_gpu(pa, 1.0)[0]
    assert (out == 255 / 128).all()
