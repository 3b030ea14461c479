"""mla_decode, mla_verify and mla_prefill with many short units a CTA, most of them one tile long:
the queries' images, their scales and their buffers are handed over as soon as the unit before is
done with them, at 16, 32 and 48 rows a unit (one query buffer at 32 and 48, two at 16)."""
import random

import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import workloads as W
from tests import parity
from tests.test_verify_tree_gpu import reference

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("B,H,n_q,top", [(900, 12, 1, 64), (2000, 5, 1, 130), (700, 16, 2, 100), (600, 12, 4, 128),
                                         (400, 16, 4, 70), (500, 11, 4, 300)])
def test_many_short_sequences(B, H, n_q, top):
    r = random.Random(B)
    lens = [r.choice([0, n_q, r.randint(n_q, top), r.randint(n_q, top)]) for _ in range(B)]
    inp = W.make_inputs("short", lens, H=H, n_q=n_q, seed=B)
    # queries of very different sizes from one sequence to the next: a scale taken from the wrong
    # unit is off by powers of two
    inp.q.mul_(torch.tensor([2.0 ** r.randint(-6, 1) for _ in range(B)])[:, None, None, None].bfloat16())
    ref = reference(inp, [[(2 << j) - 1 for j in range(n_q)]] * B)
    kv = mla.KVCache.from_inputs(inp, DEV)
    q, ws = inp.q.to(DEV), mla.workspace(mla.MLA_OP_VERIFY, B, H, n_q, DEV)
    first = mla.mla_verify(kv, q, inp.sm_scale, ws=ws)
    assert mla.mla_read_status(ws) == 0
    parity.compare(*first, *ref, f"B={B}", max_abs_row=parity.MAX_ABS)
    for _ in range(20):
        out, lse = mla.mla_verify(kv, q, inp.sm_scale, ws=ws)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    if n_q == 1:
        out, lse = mla.mla_decode(kv, q[:, 0].contiguous(), inp.sm_scale, ws=ws)
        assert torch.equal(out[:, None], first[0]) and torch.equal(lse[:, None], first[1])
    out, _ = mla.mla_verify_f32(kv, q, inp.sm_scale, ws=ws)
    assert torch.equal(out.bfloat16(), first[0])
    assert mla.mla_read_status(ws) == 0


@pytest.mark.parametrize("H,T,L", [(12, 128, 128), (16, 1000, 1000), (1, 2000, 2010)])
def test_short_prefill_units(H, T, L):
    """A chunk without a prefix: its first units see a single tile."""
    inp = W.make_inputs("chunk", [L], H=H, n_q=T, seed=T)
    q, kv = inp.q[0].to(DEV).contiguous(), mla.KVCache.from_inputs(inp, DEV)
    rows = sorted(random.Random(T).sample(range(T), 40))
    keys = inp.pool[inp.page_table[0].long()].reshape(-1, 576)[:L].view(torch.float8_e4m3fn).double() * inp.kv_scale
    first = mla.mla_prefill(kv, q, inp.sm_scale)
    x = inp.q[0, rows].double() @ keys.T * inp.sm_scale
    hidden = torch.arange(L) > torch.tensor(rows)[:, None] + L - T
    x.masked_fill_(hidden[:, None], -float("inf"))
    want = torch.softmax(x, -1) @ keys[:, :512]
    parity.compare(first[0][rows], first[1][rows], want.numpy(), torch.logsumexp(x, -1).numpy(), "prefill",
                   max_abs_row=parity.MAX_ABS)
    for _ in range(10):
        out, lse = mla.mla_prefill(kv, q, inp.sm_scale)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
