"""A decode step follows its attributes: what is assigned to it counts from the
next call on, with and without a window, over both kinds of cache."""
import numpy as np
import pytest
import torch

import q4_ref
import test_q4_decode
from helpers import assert_decode_close, make_case


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


class _Fake:
    """Stands for a prepared call: what it was made from, and a workspace that is the step's."""

    def __init__(self, *made_from):
        self.made_from = made_from

    def owns_workspace(self, workspace):
        return True

    def __call__(self, stream=None, phase=None):
        return self.made_from


@pytest.mark.parametrize("kind", ["window", "q4"])
def test_a_kept_call_is_made_anew_after_an_assignment(pa, monkeypatch, kind):
    """On the CPU: the arguments a step's call is made from."""
    from paged_kv_cache_237_gb300 import engine
    made = []
    name = "_decode_call" if kind == "window" else "_decode_q4_call"
    monkeypatch.setattr(pa, name, lambda *a: made.append(a) or _Fake(*a))
    status = object()
    q = torch.zeros(2, 4, 64)
    tables, lens = torch.zeros(2, 8, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    if kind == "window":
        cache = torch.zeros(3, 2, 16, 64)
        step = engine.DecodeStep(q, cache, cache, tables, lens, 0.1, 100, 64, window=40, status=status)
    else:
        cache = torch.zeros(3, 2, pa.pa_q4_page_bytes(64, 16, 64), dtype=torch.uint8)
        monkeypatch.setattr(pa, "_q4_geometry", lambda *a: (3, 2, 16))
        step = engine.Q4DecodeStep(q, cache, cache, tables, lens, 0.1, 100, 64, window=40, status=status)
    step.decode()
    n = len(made)
    assert step.decode() == made[-1] and len(made) == n              # kept
    for attribute, value in (("q", q + 1), ("scale", 0.7), ("block_tables", tables + 1), ("context_lens", lens + 1),
                             ("k_cache", cache + 1), ("v_cache", cache + 2), ("out", q + 3), ("window", 7),
                             ("num_sinks", 3), ("max_context_len", 90), ("partition_size", 32), ("status", object()),
                             ("workspace", torch.zeros(8))):
        setattr(step, attribute, value)
        args = step.decode()
        assert any(a is value for a in args), attribute
    n = len(made)
    assert step.decode() == made[-1] and len(made) == n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_results_follow_assignments_with_a_window(pa, dtype):
    from paged_kv_cache_237_gb300.engine import DecodeStep
    q, kc, vc, tables, lens = make_case([300, 70, 999], 8, 2, 128, 16, dtype, 5)
    step = DecodeStep(q, kc, vc, tables, lens, 0.09, 1000, 64, window=200, num_sinks=3)
    step.decode()
    for change in (dict(q=q * 2), dict(scale=0.05), dict(k_cache=kc.flip(0).contiguous(), v_cache=vc.flip(0).contiguous(),
                                                         block_tables=(kc.shape[0] - 1 - tables).clamp(min=-1)),
                   dict(window=50), dict(context_lens=lens - 20)):
        for name, value in change.items():
            setattr(step, name, value)
        out = step.decode()
        n = step.context_lens.cpu().numpy()
        dead = torch.nan_to_num     # slots past the end hold NaN, which a sum over visible tokens never meets
        ref = q4_ref.attend(step.q.double().cpu().numpy(), dead(step.k_cache.double()).cpu().numpy(),
                            dead(step.v_cache.double()).cpu().numpy(), step.block_tables.cpu().numpy(), n, step.scale,
                            16, step.window, 3)
        assert_decode_close(out, torch.from_numpy(ref), dtype, what=str(list(change)))
    assert step.status.read() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_results_follow_assignments_over_a_four_bit_cache(pa, dtype):
    case = test_q4_decode.make([300, 70, 999], 8, 2, 128, 16, 64, dtype, 5)
    other = test_q4_decode.make([300, 70, 999], 8, 2, 128, 16, 64, dtype, 6)
    step = test_q4_decode.step(pa, case, 64, partition_size=64)
    test_q4_decode.check(step.decode(), case, 0.09, 16, 64)
    step.q = other[0].cuda()
    test_q4_decode.check(step.decode(), (other[0], *case[1:]), 0.09, 16, 64, what="q")
    step.k_cache, step.v_cache = (torch.from_numpy(x).cuda() for x in other[1:3])
    step.block_tables = torch.from_numpy(other[3]).cuda()
    test_q4_decode.check(step.decode(), other, 0.09, 16, 64, what="caches")
    step.scale = 0.04
    test_q4_decode.check(step.decode(), other, 0.04, 16, 64, what="scale")
    step.window, step.num_sinks = 100, 5
    test_q4_decode.check(step.decode(), other, 0.04, 16, 64, 100, 5, what="window")
    assert step.block_size == 16 and step.status.read() == 0 and np.isfinite(other[0].float().numpy()).all()
