"""Every call that is given a stream allocates on it: outputs, a workspace, what lies between. (The
calls around a speculative step are in test_streams_gpu.py.) The caller's own stream still has
writes to make into memory that it has freed; a result placed there would be written over."""
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import dcp
from mla_latent_kv_attention_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


def calls():
    """{name: (call, bytes of the workspace that it allocates)}"""
    H = 12
    inp = W.make_inputs("streams", [4000, 900], H=H, n_q=2, seed=1)
    kv, q = mla.KVCache.from_inputs(inp, DEV), inp.q.to(DEV)
    chunk = W.make_inputs("chunk", [700], H=H, n_q=200, seed=2)
    chunk_kv, chunk_q = mla.KVCache.from_inputs(chunk, DEV), chunk.q[0].to(DEV).contiguous()
    m = W.mha_prefill_inputs(200, 300, H=2, seed=3)
    m_kv, m_q, m_w = mla.KVCache.from_inputs(m.cache, DEV), m.q.to(DEV), m.w_ukv.to(DEV)
    g = torch.Generator().manual_seed(4)
    po, pl = torch.randn(5, 300, 512, generator=g).to(DEV), torch.randn(5, 300, generator=g).to(DEV)
    probs = torch.softmax(3 * torch.randn(64, 3000, generator=g), -1).to(DEV)
    first, sc = q[:, 0].contiguous(), inp.sm_scale
    views = dcp.rank_views(kv, dcp.shard_plan(inp.seq_lens.tolist(), 64, 2, 2)[0])
    size = mla.mla_workspace_size
    verify_ws = size(mla.MLA_OP_VERIFY, 2, H, 2)
    return {
        "decode": (lambda **k: mla.mla_decode(kv, first, sc, **k), size(mla.MLA_OP_DECODE, 2, H, 1)),
        "verify": (lambda **k: mla.mla_verify(kv, q, sc, **k), verify_ws),
        "verify_f32": (lambda **k: mla.mla_verify_f32(kv, q, sc, **k), verify_ws),
        "shard": (lambda **k: mla.mla_verify_f32(kv, q, sc, visible_shift=1, **k), verify_ws),
        "prefill": (lambda **k: mla.mla_prefill(chunk_kv, chunk_q, sc, **k), size(mla.MLA_OP_PREFILL, 1, H, 200)),
        "mha": (lambda **k: mla.mla_prefill_mha(m_kv, m_q, m_w, m.cache.sm_scale, **k),
                int(mla.library().mla_prefill_mha_workspace_size(500, 2, 0))),
        "mha_bf16": (lambda **k: mla.mla_prefill_mha(m_kv, m_q, m_w, m.cache.sm_scale, L=500, bf16=True, **k),
                     int(mla.library().mla_prefill_mha_workspace_size(500, 2, 0))),
        "merge": (lambda **k: mla.mla_merge_lse(po, pl, **k), 1),
        "top_k": (lambda **k: (mla.mla_top_k_renorm_prob(probs, 20, **k),), 1),
        "rank_partials": (lambda **k: dcp.rank_partials(views, q, sc, **k), verify_ws),
        "merge_partials": (lambda **k: dcp.merge_partials(po.view(5, 10, 2, 15, 512), pl.view(5, 10, 2, 15), **k), 1),
        "dcp": (lambda **k: dcp.dcp_attention(kv, q, sc, 3, **k), verify_ws),
    }


NAMES = ["decode", "verify", "verify_f32", "shard", "prefill", "mha", "mha_bf16", "merge", "top_k", "rank_partials",
         "merge_partials", "dcp"]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_results_belong_to_the_stream(name, raw):
    call, ws = calls()[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = [torch.empty_like(t) for t in want]
    late.append(torch.empty(ws, dtype=torch.uint8, device=DEV))
    torch.cuda._sleep(40_000_000)  # (cycles: about 20 ms before the writes below)
    for t in late:
        t.fill_(1)
    del late, t
    got = call(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.cuda.current_stream() != side  # the caller's stream is the current one again


@pytest.mark.parametrize("name", ["decode", "verify", "verify_f32", "prefill", "merge", "top_k"])
def test_own_outputs_and_the_default_stream(name):
    """Given everything that it writes, a call allocates nothing and takes the handle as it is; the
    default stream's handle, 0, too."""
    call, ws = calls()[name]
    want = [t.clone() for t in call()]
    out = [torch.zeros_like(t) for t in want]
    given = dict(zip(("out", "lse"), out))
    if ws > 1:
        given["ws"] = torch.zeros(ws, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        before = torch.cuda.memory_stats()["allocation.all.allocated"]
        call(stream=stream, **given)
        assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        for a, b in zip(call(stream=stream), want):
            torch.cuda.synchronize()
            assert torch.equal(a, b)
