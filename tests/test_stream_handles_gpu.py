"""Calls that are given the default stream's handle, in order with the work queued there before and
after them."""
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from tests.test_streams_gpu import DEV, calls

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [0, 1, "current", "default"])
@pytest.mark.parametrize("name", ["rope", "gather", "tree", "accept"])
def test_default_streams_handle(name, handle):
    """The handle of the default stream (0, cudaStreamLegacy, a stream object's): the call waits for
    what was queued there, and what is queued after it waits for the call."""
    call = calls()[0][name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    given = {"current": torch.cuda.current_stream().cuda_stream,
             "default": torch.cuda.default_stream()}.get(handle, handle)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda._sleep(100_000_000)  # (cycles: about 50 ms)
    start.record()
    got = call(stream=given)
    copies = [t.clone() for t in got]
    end.record()
    assert not start.query()  # the call returned while its stream was still busy with the sleep
    assert not end.query()
    torch.cuda.synchronize()
    for a, b, c in zip(got, copies, want):
        assert torch.equal(a, c) and torch.equal(b, c)


def test_inputs_queued_before_the_call():
    """x is written behind a sleep on the default stream; a rotation on any other stream would
    read what was there before."""
    x = torch.zeros(40, 12, 64, dtype=torch.bfloat16, device=DEV)
    values = torch.randn(40, 12, 64, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    positions = torch.arange(40, device=DEV)
    rope = mla.mla_rope_init()
    want = mla.mla_rope(rope, values, positions)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    x.copy_(values)
    got = mla.mla_rope(rope, x, positions, stream=0)
    x.zero_()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
