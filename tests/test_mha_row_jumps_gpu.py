"""MHA-form prefill where some rows' running maxima jump by more than the rescale threshold (2^8) from
one key tile to the next while their neighbours' stay: rows of one warp differ, and a warp loads tensor
memory as one. Scores rise along the keys, by whole RoPE dims at +448, for every third new position."""
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
import oracle
from mla_latent_kv_attention_gb300 import workloads as W
from tests import parity

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rising(T, prefix, H, nats, seed):
    m = W.mha_prefill_inputs(T, prefix, H=H, seed=seed)
    L = T + prefix
    pos = torch.arange(L)
    W._set_rope_block(m.cache, 0, pos, torch.round(64.0 * pos / L).long())
    a = nats / 64.0 / (448.0 * m.cache.kv_scale * m.cache.sm_scale)
    m.q[..., 128:] = 0.0
    m.q[1::3, :, 128:] = a
    return m


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,prefix,H,nats", [(50, 350, 2, 60.0), (300, 700, 3, 100.0), (130, 1500, 1, 40.0)])
def test_rising_scores(T, prefix, H, nats, bf16):
    m = rising(T, prefix, H, nats, T)
    kv = mla.KVCache.from_inputs(m.cache, DEV)
    ws = torch.zeros(mla.library().mla_prefill_mha_workspace_size(T + prefix, H, 0), dtype=torch.uint8, device=DEV)
    out, lse = mla.mla_prefill_mha(kv, m.q.to(DEV), m.w_ukv.to(DEV), m.cache.sm_scale, L=T + prefix, ws=ws, bf16=bf16)
    assert mla.mla_read_status(ws) == 0
    ref_out, ref_lse = oracle.mha_prefill_rows(m.cache, m.q, m.w_ukv)
    # (the bf16 form rounds each 448 kv_scale to bfloat16, 2^-9 of a row's whole rise, which is most of its lse)
    kw = dict(rel_l2=parity.MHA_BF16_REL_L2, lse_rel=parity.MHA_BF16_LSE_REL) if bf16 else {}
    parity.compare(out, lse, ref_out, ref_lse, "rising", max_abs_row=parity.MHA_MAX_ABS_ROW, **kw)
