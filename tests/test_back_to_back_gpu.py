"""Calls queued one behind the other on one workspace, where no sequence is split: the merge kernel
has nothing to merge, and must all the same not let the next call's attention kernel, its
programmatic dependent, past the attention kernel in front of it."""
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("H,n_q", [(12, 1), (8, 2), (12, 4)])
@pytest.mark.parametrize("f32", [False, True])
def test_one_sequence_an_sm(H, n_q, f32):
    """As many equal sequences as SMs, so that every CTA takes one whole sequence: other queries
    and outputs in every call, each result equal to the call alone."""
    B, rounds = sms(), 12
    inp = W.make_inputs("even", [640] * B, H=H, n_q=n_q, seed=H)
    kv = mla.KVCache.from_inputs(inp, DEV)
    g = torch.Generator().manual_seed(n_q)
    qs = [torch.randn(inp.q.shape, generator=g).bfloat16().to(DEV) for _ in range(rounds)]
    ws = mla.workspace(mla.MLA_OP_VERIFY, B, H, n_q, DEV)
    call = mla.mla_verify_f32 if f32 else mla.mla_verify
    alone = []
    for q in qs:
        alone.append(call(kv, q, inp.sm_scale, ws=ws))
        torch.cuda.synchronize()
        assert mla.mla_read_status(ws) == 0
    results = [tuple(torch.empty_like(t) for t in alone[0]) for _ in range(rounds)]

    def queue():
        for q, (out, lse) in zip(qs, results):
            call(kv, q, inp.sm_scale, out=out, lse=lse, ws=ws)

    def check():
        torch.cuda.synchronize()
        assert mla.mla_read_status(ws) == 0
        for (out, lse), (want, want_lse) in zip(results, alone):
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
            out.zero_()

    queue()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        queue()
    for _ in range(5):
        graph.replay()
        check()


def test_output_read_by_the_next_call():
    """A call's outputs, written behind nothing but whole sequences, are the next call's queries (of
    the latent dims): a chain of calls against the same chain with a wait after every call."""
    B, H, rounds = sms(), 12, 10
    inp = W.make_inputs("chain", [512] * B, H=H, n_q=1, seed=3)
    kv = mla.KVCache.from_inputs(inp, DEV)
    ws = mla.workspace(mla.MLA_OP_DECODE, B, H, 1, DEV)

    def chain(wait):
        q = inp.q[:, 0].to(DEV).contiguous()
        out, lse = torch.empty(B, H, 512, dtype=torch.bfloat16, device=DEV), torch.empty(B, H, device=DEV)
        for _ in range(rounds):
            mla.mla_decode(kv, q, inp.sm_scale, out=out, lse=lse, ws=ws)
            if wait:
                torch.cuda.synchronize()
            q[..., :512] += out
        torch.cuda.synchronize()
        return q

    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), want)
