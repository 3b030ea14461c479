"""The float32 output under block scales where few keys compete at high scores and the scales are far from 1: the
bound that the header gives.

With w_n the weights and v_n the value rows: the split of the weights, 2^-18 of each, and scores off by d (natural
units) move the output by (2^-18 + 2 (exp(2 d) - 1)) sum w_n |v_n| at most; weights kept to 2^-33 of the largest
weight times scale add 2^-33 max(w s) sum |v_n| / s_n. d has three parts:
  - the score in log2 units is one product and one sum, 2^-24 of |score| + |log2 scale| each;
  - the tensor cores add a score's 576 products in 18 steps of 32 into a float32 accumulator. A step may cut off
    2^-23 of the partial sum, which the products' absolute sum bounds: 18 x 2^-23 of that;
  - the query's two e4m3 terms carry an entry to 2^-21.8 of its row's largest (exactly from 2^-14.8 of it up): that
    times the absolute sum of the key's entries.
(Measured: 2^-21 of the score in lse at 400.) lse: d, the row sum's and the
logarithm's 2^-20, and its own rounding."""
import math

import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from tests.test_scaled_attention_gpu import DEV, SM, cache, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e", [-55, -20, -6, 30, 55])
@pytest.mark.parametrize("nats", [1.0, 40.0, 400.0])
@pytest.mark.parametrize("L,n,H", [(2, 1, 12), (5, 2, 8), (130, 4, 12)])
def test_competing_keys(L, n, H, nats, e):
    kv = cache([L], 1, L + n, low=e - 1, high=e + 1)
    g = torch.Generator().manual_seed(int(nats) + e)
    # the latent of every row nearly one and the same (so that all compete), the rest its own
    flat = kv.pool.view(-1, 576)
    common = flat[0, :512].clone()
    flat[:, :500] = common[:500]
    kv.scales.copy_(torch.full_like(kv.scales, 2.0 ** e))
    flat_scales = kv.scales.view(-1)
    flat_scales[1::2] *= 1.0 + 2.0 ** -9  # (and no power of two)
    k = rows(kv, 0, L)
    toward = k[0, :512] / k[0, :512].norm()
    q = 0.05 * torch.randn(1, n, H, 576, generator=g).to(DEV).double() / k[0].norm() * 24
    q[..., :512] += toward * nats / SM / k[0, :512].norm()
    q = q.bfloat16()
    out, lse = mla.mla_verify_f32(kv, q, SM)
    s = kv.scales[kv.page_table[0, :-(-L // 64)].long()].double().reshape(-1)[:L]
    for j in range(n):
        last = L - n + j
        kk, sc = k[:last + 1], s[:last + 1]
        x = q[0, j].double() @ kk.T * SM
        ref_lse = torch.logsumexp(x, -1)
        w = torch.exp(x - ref_lse[:, None])
        ref = w @ kk[:, :512]
        terms = q[0, j].double().abs() @ kk.abs().T * SM
        d = math.log(2) * 2.0 ** -23 * (x.abs() / math.log(2) + sc.log2().abs()) + 18 * 2.0 ** -23 * terms
        d = (d + 2.0 ** -21.8 * q[0, j].double().abs().amax(-1)[:, None] * kk.abs().sum(-1) * SM).amax(-1)
        size = kk[:, :512].norm(dim=-1)
        allowed = (2.0 ** -18 + 2 * torch.expm1(2 * d)) * (w @ size) + 2.0 ** -33 * (w * sc).amax(-1) * (size / sc).sum()
        err = (out[0, j].double() - ref).norm(dim=-1)
        assert bool((err <= allowed).all()), float((err / allowed).max())
        lse_off = (lse[0, j].double() - ref_lse).abs()
        assert bool((lse_off <= d + 2.0 ** -20 + 2.0 ** -23 * ref_lse.abs()).all()), float(lse_off.max())
