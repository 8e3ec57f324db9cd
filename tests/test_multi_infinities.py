"""Infinite values that a query sees, in pa_decode_tree and pa_decode_cross: the result's column is that infinity, as in the
formula (two of different signs, and a NaN, leave a NaN), in every pass and type, and no other column changes."""
import pytest
import torch

import multi_gpu_ref
from helpers import assert_decode_close
from multi_ref import Batch

INF = float("inf")


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


def at(b, i, u):
    return int(b.tables[i, u // b.bs]), slice(None), u % b.bs


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["chain", "cross"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("most,Hq,Hkv", [(1, 2, 2), (12, 2, 1), (60, 2, 1), (40, 16, 1)])
def test_infinities_stay_what_they_are(pa, kind, dtype, hd, most, Hq, Hkv):
    """In the context, at weights of any size: one of them is its row's largest, which is 1 exactly."""
    b = Batch(kind, [400, 90, 700], [most, 3, most], Hq, Hkv, hd, 16, dtype, 16)
    scale = hd ** -0.5
    clean = multi_gpu_ref.batch(b, scale)[0]
    peak = at(b, 0, 55)
    b.q[..., 7] = b.q[..., 7].abs() + 0.5
    b.k[peak][..., 7] = 60.0
    clean = multi_gpu_ref.batch(b, scale)[0]
    want = clean.clone()
    rows = slice(0, most)
    for u, col, x in ((7, 0, INF), (300, 1, -INF), (200, 2, INF), (201, 2, -INF), (9, 3, float("nan")), (55, 4, INF),
                      (55, 5, -INF), (330, 6, -INF)):
        b.v[at(b, 0, u)][..., col] = x
        want[rows, :, col] = want[rows, :, col] + x
    got = b.on_gpu(pa, scale)[0].double()
    assert_decode_close(torch.where(want.isfinite(), got, 0.0), torch.where(want.isfinite(), want, 0.0), dtype)
    odd = ~want.isfinite()
    assert odd[rows, :, :7].all() and not odd[rows, :, 7:].any() and not odd[most:].any()
    assert torch.equal(got[odd].nan_to_num(nan=7.0), want[odd].nan_to_num(nan=7.0))
