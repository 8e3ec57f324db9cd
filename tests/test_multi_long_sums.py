"""Sums over long contexts in pa_decode_tree and pa_decode_cross: a tensor core cuts its sums off where additions round, and
thousands of such steps lean towards zero.  They stay few in every pass, however many tiles a CTA walks."""
import pytest
import torch

import multi_gpu_ref
from multi_ref import Batch


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


@pytest.mark.gpu
@pytest.mark.parametrize("hd", [64, 128])
# few rows per sequence, up to 128, more than that; thousands of results, since each that moves counts
@pytest.mark.parametrize("most,Hq,Hkv,times", [(2, 16, 16, 13), (100, 1, 1, 200), (33, 8, 1, 200)])
def test_results_do_not_lean_towards_zero(pa, hd, most, Hq, Hkv, times):
    """How often a result is another bf16 value than the nearest, and to which side, where a CTA walks hundreds of tiles.

    An error is 1.44 * 2^7 times as many steps (of 2^-7 to 2^-8 of the value) on average.  A tensor core takes 16 tokens at a
    time, in each part of the weights, and cuts off half of 2^-24 each time on average: 1024 times in a run of 64 tiles,
    2^-15, 0.0056 steps to one side: below 2^-7.  Weights are off by 2^-17.3 in the root mean square, independently, as the
    values are; over the normal distribution of the results (many are small, and so are their steps) that moves 0.005
    of them: together below 2^-6."""
    b = Batch("cross", [60_000], [most], Hq, Hkv, hd, 16, torch.bfloat16, 4)
    scale = hd ** -0.5
    out = multi_gpu_ref.batch(b, scale)[0]
    near = out.float().bfloat16()
    got = multi_gpu_ref.repeated(b, times).on_gpu(pa, scale)[0].unflatten(0, (times, -1))
    step = torch.exp2(torch.floor(torch.log2(near.double().abs().clamp_min(1e-30)))) * 2.0 ** -7
    off = (got.double() - near.double()) * near.double().sign() / step
    assert (off != 0).double().mean() < 2.0 ** -6
    assert off.mean().abs() < 2.0 ** -7
