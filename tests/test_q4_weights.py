"""pa_decode_q4's weights over long rows that one warp holds whole: a token that
outweighs a long tail, and steps of very different sizes.

Rounding (include/pa.h): a weight times its value's step is held relative to
the largest such product of its group of values so far, M.  bf16: as one fp16
number, 2^-11 relative, but no finer than 2^-32 M (products are scaled to
[2^7, 2^8) and fp16 steps by 2^-24, so half a step is 2^-25 / 2^7).  fp32: as
two, 2^-22 relative, but no finer than 2^-43 M (the second counts 2^-11).
Scores in these tests are one product of K's minimum and a sum of q: fp32
keeps it to 2^-22 or so, bf16 to 2^-17 (q's sum in two bf16 parts)."""
import numpy as np
import pytest
import torch

import q4_ref
import test_q4_decode
from q4_shared import Shared


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


def relative(dtype, score):
    """Relative error of an output that is a sum of terms of one sign: the
    result's rounding, the weights', exp of a score off by its share, and for
    fp32 the sums': up to 4096 tokens are added up by themselves, 512 to a lane,
    and 512 additions of half a step, 2^-24, of a sum that grows evenly are 2^-16 at
    worst; for the numerator and the sum of weights together (4 tokens at a
    time) 1.25 times that."""
    off = abs(score) * 1.4427 * 2.0 ** (-22 if dtype == torch.float32 else -17) * np.log(2)
    return off + (1.25 * 2.0 ** -16 if dtype == torch.float32 else 2.0 ** -8 + 2.0 ** -11)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [8192, 65536])
@pytest.mark.parametrize("hd,group", [(64, 64), (128, 32)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["no step", "a step"])
def test_a_long_tail_under_one_dominant_token(pa, dtype, hd, group, n, kind):
    """The first token weighs 1 and has the value 0; the tail's tokens weigh e^-17 each, with every code
    the same, so that all their errors add up.  Without a step of its own ("no step") the first token
    has no product for the tail's to be small against, and the tail is held to its relative precision.
    With one ("a step"), each tail token may be off by the floor, times a code of at most 15; and fp32 sums
    round next to the first token's two parts of 7.5 steps, which only cancel in the end: 256 additions of
    codes and, in its lane, 512 of minima before the sums start anew, each off by half a step of 2^-24."""
    score = -17.0
    scores = np.full(n, score)
    scores[0] = 0.0
    codes = np.full((n, hd), 15)
    codes[0] = 0
    step, low = np.full((n, hd // group), 0.25), np.zeros((n, hd // group))
    if kind == "no step":
        step[0] = 0.0
    batch = Shared(scores, codes, step, low, group)
    ref = batch.reference()
    tol = relative(dtype, score) * np.abs(ref)
    if kind == "a step":
        tol = tol + n * 2.0 ** (-43 if dtype == torch.float32 else -32) * 0.25 * 15
        if dtype == torch.float32:
            tol = tol + (256 + 512) * 2.0 ** -25 * 7.5 * 0.25
    worst = (np.abs(batch.run(pa, dtype) - ref) / tol).max()
    assert worst <= 1, f"error {worst:.2f} of the tolerance"


@pytest.mark.gpu
@pytest.mark.parametrize("exponent", [20, 26, 40, 100])
@pytest.mark.parametrize("hd,group", [(64, 64), (128, 32)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("at", [0, 5, 3000])
def test_a_large_step_without_weight(pa, dtype, hd, group, exponent, at):
    """One visible token's step is 2^exponent times the others', and its weight e^-130 = 2^-187: its part of the
    output is below 2^-80 even so.  Tolerance relative to the others' values: fp32 the framework's 1e-5, bf16 the result's rounding and the weights',
    2^-11 each times a code part of at most twice the largest value."""
    rng = np.random.default_rng(exponent + at)
    n = 8000
    scores = q4_ref.bf16_toward(rng.uniform(-1, 1, n), True)
    scores[at] = -130.0
    codes = rng.integers(0, 16, (n, hd))
    step, low = rng.uniform(0.1, 0.4, (n, hd // group)), rng.uniform(-3.5, -1.0, (n, hd // group))
    step[at] = 0.25 * 2.0 ** exponent
    low[at] = 0.0
    batch = Shared(scores, codes, step, low, group)
    ref = batch.reference()
    others = np.abs(np.delete(batch.values, at, 0)).max()
    tol = 1e-5 * others + 0 * ref if dtype == torch.float32 else 2.0 ** -8 * np.abs(ref) + 1.25 * 2.0 ** -10 * others
    worst = (np.abs(batch.run(pa, dtype) - ref) / tol).max()
    assert worst <= 1, f"error {worst:.2f} of the tolerance"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_steps_that_start_at_nothing(pa, dtype):
    """No step at all in a row's first tokens (or steps near the smallest bf16), then ordinary and very large
    ones, some of them on tokens without weight."""
    rng = np.random.default_rng(3)
    for first, later in ((0.0, 0.25), (0.0, 2.0 ** 100), (2.0 ** -126, 0.25), (2.0 ** -126, 2.0 ** 100)):
        n, hd = 3000, 64
        scores = q4_ref.bf16_toward(rng.uniform(-1, 1, n), True)
        codes = rng.integers(0, 16, (n, hd))
        step, low = rng.uniform(0.5, 1.0, (n, 1)) * later, np.zeros((n, 1))
        step[:70] = first
        scores[100:1000:3] = -130.0
        step[100:1000:3] *= 2.0 ** 20
        batch = Shared(scores, codes, step, low, 64)
        ref = batch.reference()
        tol = 1e-5 * later * 15 + 0 * ref if dtype == torch.float32 else \
            2.0 ** -8 * np.abs(ref) + 1.25 * 2.0 ** -10 * later * 15
        worst = (np.abs(batch.run(pa, dtype) - ref) / tol).max()
        assert worst <= 1, f"{first} then {later}: error {worst:.2f} of the tolerance"


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [(1.0, 0.5, -1.0), (1.0, -0.25, 0.75, 0.125, -0.5, 0.0), tuple(1.0 - i / 16 for i in range(12))])
@pytest.mark.parametrize("n", [4000, 13000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_references_that_rise_all_along(pa, dtype, n, heads):
    """Scores that climb by 60 over a row, so that units outgrow the last ones' references, for some heads
    (negative multiples: they fall), and steps that fall by 2^20 meanwhile; 13000 tokens: sums put by every 4096."""
    rng = np.random.default_rng(8)
    hd = 128
    scores = q4_ref.bf16_toward(np.linspace(-30, 30, n) + rng.uniform(-1, 1, n), True)
    codes = rng.integers(0, 16, (n, hd))
    step = rng.uniform(0.5, 1.0, (n, 2)) * 2.0 ** np.linspace(20, 0, n)[:, None]
    batch = Shared(scores, codes, step, -7 * step, 64, heads=heads)
    ref = batch.reference()
    for h, a in enumerate(heads):       # each head's tolerance by the values that weigh for it
        x = batch.scores * a
        p = np.exp(x - x.max())
        big = (p @ np.abs(batch.values).max(1)) / p.sum()
        out = batch.run(pa, dtype)[:, h]
        # a score of 30 is off by up to 30 * 1.44 * 2^-22 (fp32) or 2^-17 in the exponent
        off = 2 * 31 * 1.4427 * 2.0 ** (-22 if dtype == torch.float32 else -17) * np.log(2) * 2 * big
        tol = off + (1e-5 * big + 0 * ref[h] if dtype == torch.float32 else
                     2.0 ** -8 * np.abs(ref[h]) + 1.25 * 2.0 ** -10 * big)
        # the floors: the other heads' products may be the larger by the steps' 2^20
        floor = 2.0 ** (-43 if dtype == torch.float32 else -32) * (batch.step.max() * 15 * n) / p.sum()
        worst = (np.abs(out - ref[h]) / (tol + floor)).max()
        assert worst <= 1, f"head {h}: error {worst:.2f} of the tolerance"


@pytest.mark.gpu
@pytest.mark.parametrize("hd,bs,group", [(64, 16, 32), (128, 32, 64)])
def test_peaked_scores_in_fp32(pa, hd, bs, group):
    """Scores of size 50 and more.  A score is a sum over the row's terms q (s (c - 7.5)) and q (m + 7.5 s); the parts
    of q, the codes' products and the fp32 sums leave it within 2^-21 of the terms' absolute sum (q's two
    fp16 parts 2^-22, and fp32 sums of hd + 4 terms, on tensor cores a few steps of the largest).  A
    score off by d moves the output by at most 2 d max|v|."""
    for scale in (3.0, -1.0, 0.5):
        case = test_q4_decode.make([1, 300, 1000], 8, 2, hd, bs, group, torch.float32, 9)
        out, flags = test_q4_decode.on_gpu(pa, case, scale, group, torch.float32, partition_size=128)
        assert flags == 0
        q, kc, vc, tables, lens = case
        with np.errstate(invalid="ignore"):
            k, v = q4_ref.values(kc, bs, hd, group), q4_ref.values(vc, bs, hd, group)
        ref = q4_ref.attend(q.double().numpy(), k, v, tables, lens, scale, bs)
        vmax = np.abs(v[np.isfinite(v)]).max()
        # |s (c - 7.5)| + |m + 7.5 s| is at most 7.5 * 0.4 + 3.5 + 7.5 * 0.4 (test_q4_decode.make's ranges)
        terms = np.abs(q.double().numpy()).sum(-1, keepdims=True) * 9.9 * abs(scale)
        tol = (1e-5 + 2 * terms * 2.0 ** -21) * vmax
        worst = (np.abs(out.double().cpu().numpy() - ref) / tol).max()
        assert worst <= 1, f"scale {scale}: error {worst:.2f} of the tolerance"
