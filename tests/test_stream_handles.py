"""Raw stream handles, without a GPU: torch's stream classes are stood in for."""
import contextlib

import pytest
import torch

import mla_latent_kv_attention_gb300 as mla


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def streams(monkeypatch):
    """default_stream, ExternalStream and stream as torch.cuda has them: ExternalStream(0) is a new
    stream of the pool, whatever its argument means to CUDA."""
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: Stream(handle or 0xF001))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext(s))


@pytest.mark.parametrize("given,handle", [(0, 0), (1, 0), (2, 2), (0x7F00, 0x7F00), (Stream(0), 0),
                                          (Stream(0x7F00), 0x7F00)])
def test_handles(streams, given, handle):
    """0 is the default stream's handle (what its cuda_stream is), 1 another name for it."""
    with mla._current(given) as s:
        assert s.cuda_stream == handle
