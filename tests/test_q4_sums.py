"""pa_decode_q4's sums over long rows that one warp holds whole: flat scores over
values of mean zero, where the output is a small difference of large sums, and
values that are all alike, where the same error is made in every term."""
import numpy as np
import pytest
import torch

import q4_ref
from q4_shared import Shared


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


@pytest.mark.gpu
@pytest.mark.parametrize("n", [8192, 131072])
@pytest.mark.parametrize("hd,group,heads", [(64, 64, 1), (128, 32, 1), (128, 64, 8), (64, 32, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("alike", [False, True])
def test_flat_scores_over_values_of_mean_zero(pa, dtype, hd, group, heads, n, alike):
    """In the 2-norm, relative to the output.  bf16: half a step of the result, spread evenly, is 2^-8 / sqrt(3).  A
    weight's error is 2^-11 of it at most and meets the code part, which counts from 0 for one half of the
    tokens and from 15 for the other: twice the value in root mean square (3 allowed, which covers the unequal
    steps), and for weights that are all alike the sum of the code parts is a random walk like the output.  As
    much again for the sums.  fp32: codes count from 7.5 and minima from the middle of a range, so both parts are
    random walks as the output is (the middles are what bf16 rounds off -7.5 steps, 2^-9 of it).  An accumulator adds
    256 times in 4096 tokens, to a sum of 4.6 * 64 steps at the end: 16 * 0.3 * 0.6 * 295 * 2^-24, 2^-14.3 steps,
    sqrt(32) of that at 131072 tokens, and the second sums' 32 additions of up to 1665 steps, 2^-13.3: 2^-22 of
    the output.  The exponential and a weight's two parts are 2^-22 each and independent, and products cut off at
    2^-24 of the largest, of either sign alike, less.  2^-18 allows for four times their sum."""
    rng = np.random.default_rng(n + hd)
    scores = np.zeros(n) if alike else q4_ref.bf16_toward(rng.uniform(-0.05, 0.05, n), True)
    codes = rng.integers(0, 16, (n, hd))
    step = np.full((n, hd // group), 0.3125) if alike else rng.uniform(0.1, 0.4, (n, hd // group))
    batch = Shared(scores, codes, step, -7.5 * step, group, heads=[1.0 - i / 32 for i in range(heads)])
    ref = batch.reference()
    out = batch.run(pa, dtype)
    rel = np.sqrt(((out - ref) ** 2).sum((1, 2)) / (ref ** 2).sum())
    assert rel.max() <= (2.0 ** -18 if dtype == torch.float32 else (2.0 ** -8 + 6 * 2.0 ** -11) / 3 ** 0.5), rel


@pytest.mark.gpu
@pytest.mark.parametrize("n", [8192, 131072])
@pytest.mark.parametrize("code", [0, 7, 15])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_same_value_all_along(pa, dtype, code, n):
    """Every term is the same, so nothing averages out; the minimum is -code steps, and the output zero, so that
    all of an error shows.  Weights: equal ones of 2^-11 at most (bf16) or 2^-22, times a code part of at most 15
    steps counted from 0 or from 15.  Sums of 4096 equal terms: fp32 additions of half a step, 512 to a lane of
    a sum that grows evenly: 512 * 2^-25; on tensor cores, cut off rather than rounded, 16 products at a time: 256
    times 2^-24 of a sum that grows evenly, for each of up to 17 terms that are brought to the sum's exponent,
    256 * 17 * 2^-25 = 2^-12.9 of the code part (bf16).  A bf16 result adds no rounding to a zero."""
    hd, group = 64, 64
    codes = np.full((n, hd), code)
    codes[:, 1::2] = 15 - code
    step, low = np.full((n, 1), 0.3125), np.full((n, 1), -0.3125 * code)
    batch = Shared(np.zeros(n), codes, step, low, group)
    ref = batch.reference()
    out = batch.run(pa, dtype)
    off = np.abs(out - ref)
    steps = 2.0 ** -11 + 2.0 ** -12.9 if dtype == torch.bfloat16 else 2.0 ** -22 + 2 * 2.0 ** -16
    tol = steps * 15 * 0.3125 + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0)
    assert (off <= tol).all(), (off / tol).max()


@pytest.mark.gpu
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("window,sinks", [(9000, 5), (12345, 4500), (4096, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_long_window_in_one_warp(pa, dtype, window, sinks, bs):
    """Sums put by on both sides of what the window leaves out: the tolerances of the flat scores above, with
    scores and values of ordinary spread (the output is larger against its parts, so they hold all the more)."""
    rng = np.random.default_rng(window)
    n, hd, group = 20011, 128, 64
    scores = q4_ref.bf16_toward(rng.uniform(-2, 2, n), True)
    step = rng.uniform(0.1, 0.4, (n, hd // group))
    batch = Shared(scores, rng.integers(0, 16, (n, hd)), step, -7.5 * step, group, bs, heads=(1.0, 0.5, -1.0))
    ref = batch.reference(window, sinks)
    out = batch.run(pa, dtype, window=window, num_sinks=sinks)
    rel = np.sqrt(((out - ref) ** 2).sum((1, 2)) / (ref ** 2).sum())
    assert rel.max() <= (2.0 ** -18 if dtype == torch.float32 else (2.0 ** -8 + 6 * 2.0 ** -11) / 3 ** 0.5), rel
