"""Infinite entries in queries of mla_verify_tree and mla_prefill_mha. By the formula every output of such a row is NaN (its scores are
infinite or NaN, and infinity less infinity is NaN); the other rows are bit for bit what they are
without it. A row that sees no key stays empty."""
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import workloads as W
from tests.test_verify_tree_gpu import as_tensor, tree_masks

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


def check(call, q, heads):
    """call(q) -> (out, lse), both laid out as q; the rows named in `heads` get an infinity."""
    out, lse = call(q)
    assert torch.isfinite(out).all()
    bad = torch.zeros(q.shape[:-1], dtype=torch.bool, device=DEV)
    for k, place in enumerate(heads):
        bad[place] = True
        q[place][(5, 570, 0)[k % 3]] = (INF, -INF)[k % 2]
    got, got_lse = call(q)
    assert torch.isnan(got[bad]).all() and torch.isnan(got_lse[bad]).all()
    assert torch.equal(got[~bad], out[~bad]) and torch.equal(got_lse[~bad], lse[~bad])


@pytest.mark.parametrize("H,n,lens", [(12, 8, [700, 300]), (12, 8, [20000, 300]), (5, 9, [500, 90]), (1, 64, [9000, 64]),
                                      (12, 16, [9000] * 12)])
def test_tree(H, n, lens):
    inp = W.make_inputs("inf", lens, H=H, n_q=n, seed=n)
    kv, mask = mla.KVCache.from_inputs(inp, DEV), as_tensor(tree_masks(len(lens), n, 1)).to(DEV)
    check(lambda q: mla.mla_verify_tree(kv, q, mask, inp.sm_scale), inp.q.to(DEV),
          [(0, 0, 0), (0, n - 1, H - 1), (1, n // 2, 0)])


def test_no_key():
    inp = W.make_inputs("inf", [0, 5], H=12, n_q=5, seed=1)
    inp.q[0, 1, 2, 7] = inp.q[1, 2, 3, 4] = INF
    kv = mla.KVCache.from_inputs(inp, DEV)
    out, lse = mla.mla_verify_tree(kv, inp.q.to(DEV), torch.zeros(2, 5, dtype=torch.int64, device=DEV), inp.sm_scale)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("bf16", [False, True])
def test_mha_prefill(bf16):
    m = W.mha_prefill_inputs(300, 200, H=3, seed=1)
    kv, w, q = mla.KVCache.from_inputs(m.cache, DEV), m.w_ukv.to(DEV), m.q.to(DEV)
    out, _ = mla.mla_prefill_mha(kv, q, w, m.cache.sm_scale, bf16=bf16)
    q[7, 1, 100], q[299, 2, 190] = INF, -INF
    got, _ = mla.mla_prefill_mha(kv, q, w, m.cache.sm_scale, bf16=bf16)
    bad = torch.zeros(300, 3, dtype=torch.bool, device=DEV)
    bad[7, 1] = bad[299, 2] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], out[~bad])
