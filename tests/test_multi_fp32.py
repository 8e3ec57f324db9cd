"""pa_decode_tree and pa_decode_cross over fp32 caches keep what fp32 operations keep: their tensor-core products are in two
parts a side and their sums are rounded, not cut off."""
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


# (most queries, query heads, KV heads): up to 16 rows per sequence, and more
ROWS = [(12, 4, 4), (3, 8, 2), (60, 4, 4), (50, 24, 2)]


def run(pa, b, scale):
    """(result, reference, bound on their difference, what the row's sum before its division comes to)."""
    out, spread, size, total = multi_gpu_ref.batch(b, scale)
    got, flags = b.on_gpu(pa, scale)
    assert flags == 0
    bound = multi_gpu_ref.f32_bound(out, spread, size, max(b.lens), b.q.shape[2])
    return got[:len(out)].double(), out, bound, spread * total[..., None]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", multi_ref.KINDS)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("most,Hq,Hkv", ROWS)
def test_as_exact_as_fp32_operations(pa, kind, hd, most, Hq, Hkv):
    """In the 2-norm.  Scores are of size 1, off by 10^-7 in the root mean square (their sum's roundings, 16 of 2^-25 or
    so, and products of 2^-23 that average out); the exponential by as much; the results' sums by as much again, and each is
    independent from token to token, as the values are: sqrt(3) * 10^-7, and 3 * 10^-7 leaves room."""
    b = Batch(kind, [700, 2500, 90], [most] * 3, Hq, Hkv, hd, 16, torch.float32, 3)
    got, out, bound, _ = run(pa, b, hd ** -0.5)
    assert ((got - out).abs() <= bound).all()
    assert (got - out).norm() <= 3e-7 * out.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 3.0])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("most,Hq,Hkv", ROWS)
def test_flat_and_peaked_scores(pa, scale, hd, most, Hq, Hkv):
    b = Batch("cross", [700, 40, 1], [most] * 3, Hq, Hkv, hd, 32, torch.float32, 10)
    got, out, bound, _ = run(pa, b, scale)
    assert ((got - out).abs() <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("most,Hq,Hkv", ROWS)
def test_the_largest_values_stay_finite(pa, sign, most, Hq, Hkv):
    """They would not if they were rounded to a tf32 part.  (Sums are divided at their end, so a row whose weights with
    regard to the largest bring its sum past the largest fp32 is not finite.)"""
    b = Batch("chain", [200, 150], [most] * 2, Hq, Hkv, 64, 16, torch.float32, 5)
    top = torch.finfo(torch.float32).max
    for i, u in ((0, 7), (0, 190), (1, 149)):
        b.v[int(b.tables[i, u // 16]), :, u % 16, 3] = sign * top * (1 if u == 7 else 0.25)
    b.k[int(b.tables[0, 2]), :, 0, 5] = top
    b.q[..., 5] = 1e-37
    got, out, bound, before = run(pa, b, 0.125)
    fits = before < top
    assert fits[..., 3].any()
    assert got[fits].isfinite().all()
    assert ((got - out).abs() <= bound)[fits].all()
