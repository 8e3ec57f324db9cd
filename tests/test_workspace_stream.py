"""A call that makes its own workspace makes it on the stream it runs on,
whatever form the stream is given in: None, a torch stream, another object
with a cuda_stream, or a raw handle, of which 0 is the default stream."""
import contextlib
import types

import pytest
import torch

from helpers import assert_decode_close, make_case, oracle_decode


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_237_gb300 import build
    build.build()
    from paged_kv_cache_237_gb300 import binding
    return binding


@pytest.mark.parametrize("stream,made_on", [
    (None, "current"), (0, "default 1"), (types.SimpleNamespace(cuda_stream=0), "default 1"), (0x7000, "handle 28672 1"),
    (types.SimpleNamespace(cuda_stream=0x7000), "handle 28672 1"),
])
def test_the_stream_a_workspace_is_made_on(pa, monkeypatch, stream, made_on):
    """On the CPU: which of torch's streams is current when the zeros are made."""
    now = ["current"]

    @contextlib.contextmanager
    def use(s):
        now.append(s)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev=None: f"default {dev.index}")
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda h, device=None: f"handle {h} {device.index}" if h else "a stream of the pool")
    monkeypatch.setattr(torch, "zeros", lambda n, dtype=None, device=None: (now[-1], n))
    (where, n), clean = pa._workspace(None, 1024, False, torch.device("cuda", 1), stream)
    assert where == made_on and n == 1024 and clean


@pytest.mark.gpu
@pytest.mark.parametrize("other", [False, True])
def test_default_stream_by_its_handle(pa, other):
    """stream=0 with the default stream current, and with a busy stream current
    that does not wait for it: memory that held junk is zeroed in time."""
    dtype = torch.bfloat16
    q, kc, vc, tables, lens = make_case([3000, 700, 2500], 8, 2, 128, 16, dtype, 4)
    ref = oracle_decode(q, kc, vc, tables, lens, 0.09)
    outs = [torch.full_like(q, float("nan")) for _ in range(3)]
    side = torch.cuda.Stream()
    assert torch.cuda.default_stream().cuda_stream == 0
    junk = torch.full((64 << 20,), 0xAB, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del junk
    for out in outs:
        with torch.cuda.stream(side) if other else contextlib.nullcontext():
            torch.cuda._sleep(5_000_000)
            pa.pa_decode(out, q, kc, vc, tables, lens, 0.09, max_context_len=3000, partition_size=64, stream=0)
    torch.cuda.synchronize()
    for out in outs:
        assert_decode_close(out, ref, dtype)
