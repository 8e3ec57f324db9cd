"""The 4-bit format fixes the sign of a zero minimum: +0, whatever zeros the
group holds and in whatever order, so every writer gives the same bytes."""
import numpy as np
import pytest
import torch

import q4_ref


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hd,bs,group", [(128, 16, 64), (128, 32, 32), (64, 16, 32), (64, 32, 64)])
def test_bytes_are_fixed_for_zero_minima(hd, bs, group, dtype):
    from paged_kv_cache_237_gb300 import binding as pa
    x = torch.zeros(7, 2, hd)
    x[1] = -0.0                                     # nothing but negative zeros
    x[2, :, ::2] = -0.0                             # both, alternately
    x[3] = torch.linspace(0, 3, hd)                 # a step, and a minimum of +0 in the first group
    x[4] = torch.linspace(0, 3, hd)
    x[4, :, 0], x[4, :, 1] = -0.0, 0.0
    x[5] = torch.linspace(0, 3, hd)
    x[5, :, 0], x[5, :, 1] = 0.0, -0.0
    x[6, :, -1] = -0.0
    x = x.to(dtype)
    assert torch.signbit(x).any()
    slots = torch.arange(7) * 2
    kc = torch.zeros(1, 2, q4_ref.page_bytes(hd, bs, group), dtype=torch.uint8)
    want = kc.numpy().copy()
    q4_ref.write(want, (x.double() + 0.0).numpy(), slots.numpy(), bs, group)      # -0 + 0 = +0
    dk, dv = kc.cuda(), kc.cuda()
    pa.pa_reshape_and_cache_q4(x.cuda(), x.cuda(), dk, dv, slots.cuda(), group_size=group)
    assert np.array_equal(dk.cpu().numpy(), want) and np.array_equal(dv.cpu().numpy(), want)
