"""Calls that are given a stream: what they allocate belongs to it. The caller's own stream still
has writes to make into memory that it has freed; a result or a workspace placed there would be
written over."""
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


def calls():
    g = torch.Generator().manual_seed(1)
    n, H, V = 6, 12, 1000
    inp = W.make_inputs("streams", [400, 90], H=H, n_q=n, seed=1)
    kv = mla.KVCache.from_inputs(inp, DEV)
    q = inp.q.to(DEV)
    mask = torch.randint(0, 64, (2, n), generator=g).to(DEV)
    rope = mla.mla_rope_init()
    x = torch.randn(300, H, 64, generator=g).bfloat16().to(DEV)
    positions = torch.arange(300, device=DEV)
    rows = torch.randn(50, 576, generator=g).bfloat16().to(DEV)
    slots = torch.arange(7, 57, device=DEV)
    pool = torch.zeros(2, 64, 576, dtype=torch.uint8, device=DEV)
    cu = torch.tensor([0, 300, 380], device=DEV)
    probs = torch.softmax(3 * torch.randn(2, n, V, generator=g), -1).to(DEV)
    tokens = torch.randint(0, V, (2, n), generator=g).int().to(DEV)
    u = torch.rand(2, n + 1, generator=g).to(DEV)

    def append(**k):
        pool.zero_()
        torch.cuda.synchronize()
        mla.mla_cache_append_rope(pool, rows, slots, 0.0125, rope, positions[:50], **k)
        return (pool,)

    return {
        "rope": lambda **k: (mla.mla_rope(rope, x, positions, **k),),
        "append": append,
        "gather": lambda **k: (mla.mla_cache_gather(kv, cu, 380, **k),),
        "tree": lambda **k: mla.mla_verify_tree(kv, q, mask, inp.sm_scale, **k),
        "accept": lambda **k: mla.mla_accept_drafts(probs, tokens, u, **k),
    }, {"tree": mla.workspace(mla.MLA_OP_VERIFY_TREE, 2, H, n, DEV).numel()}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["rope", "append", "gather", "tree", "accept"])
def test_results_belong_to_the_stream(name, raw):
    made, workspaces = calls()
    call = made[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = [torch.empty_like(t) for t in want]
    late.append(torch.empty(workspaces.get(name, 1), dtype=torch.uint8, device=DEV))
    if name != "append":
        torch.cuda._sleep(40_000_000)  # (cycles: about 20 ms before the writes below)
    for t in late:
        t.fill_(1)
    del late, t
    got = call(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.cuda.current_stream() != side  # the caller's stream is the current one again


def test_a_call_within_a_stream_is_the_call_on_it():
    made, _ = calls()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for name in ("rope", "gather", "tree", "accept"):
        want = made[name]()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = made[name]()
        again = made[name](stream=side)
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, again):
            assert torch.equal(a, b) and torch.equal(a, c)
