"""The MHA-form prefill over a cache with block scales, at any scale that a block may have.

Rows under different scales differ in size, so every row (new position, head) is held to a bound of its
own, the sum of the precise form's roundings in the worst case. With w_n its softmax weights and v_n the
value rows:
  - the output to bfloat16: 2^-8 |ref|;
  - values and probabilities to float16, 2^-11 each: 2^-10 sum w_n |v_n|;
  - scores off by d at most move a weight by a factor within exp(+-2 d): 2 (exp(2 d) - 1) sum w_n |v_n|. d: the
    keys as bfloat16 pairs (2^-16 of each product q_d k_d), float32 steps (2^-22 of score and log2 of the
    scale);
  - float16's subnormals: a probability, in units of the row's largest weight times scale or less, by 2^-25,
    an entry of a value, in units of 2^8 codes, by 2^-25.
The bf16 form: 2^-8 in the place of 2^-11 and of the pairs' 2^-16, no subnormals, and where a scale is no power of
two the latent's own 2^-8, which the sums of the up-projection take entry by entry. The row sum's
float32 additions: 2^-24 each, in lse."""
import math

import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import workloads as W
from tests import parity
from tests.test_scaled_attention_gpu import cache, compare, rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
SM = W.SM_SCALE


def reference(kv, q, w, L):
    """float64 out, lse, and what the rows' bounds need: weights and scores [T, H, L], keys, values, and the
    sums of the up-projection's absolute terms."""
    T, H = q.shape[:2]
    k = rows(kv, 0, L)
    up = torch.einsum("nc,chd->nhd", k[:, :512], w.double())
    terms = torch.einsum("nc,chd->nhd", k[:, :512].abs(), w.double().abs())
    key = torch.cat([up[..., :128], k[:, None, 512:].expand(L, H, 64)], -1)
    x = torch.einsum("thd,nhd->thn", q.double(), key) * SM
    hidden = torch.arange(L, device=DEV) > (L - T + torch.arange(T, device=DEV))[:, None]
    x.masked_fill_(hidden[:, None, :], -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    value = up[..., 128:]
    return torch.einsum("thn,nhd->thd", p, value), lse, p, x, key, value, terms


def scale_of(kv, L):
    page = kv.pool.shape[1]
    block = page // kv.scales.shape[1]
    return kv.scales[kv.page_table[0, :-(-L // page)].long()].double().reshape(-1).repeat_interleave(block)[:L]


def check_rows(kv, q, w, L, out, lse, bf16, odd):
    ref, ref_lse, p, x, key, value, terms = reference(kv, q, w, L)
    s = scale_of(kv, L)
    off = key.abs() * (2.0 ** -8 if bf16 else 2.0 ** -16)
    size = value.norm(dim=-1).T  # [H, n]
    value_off = size * (2.0 ** -8 if bf16 else 2.0 ** -11)
    if bf16 and odd:
        off[..., :128] += 2.0 ** -8 * terms[..., :128]
        off[..., 128:] += 2.0 ** -8 * key[..., 128:].abs()
        value_off = value_off + 2.0 ** -8 * terms[..., 128:].norm(dim=-1).T
    d = torch.einsum("thd,nhd->thn", q.double().abs(), off) * SM + 2.0 ** -22 * (x.abs() + s.log2().abs())
    d = torch.where(torch.isfinite(x), d, 0.0).amax(-1)
    spread = (p * size).sum(-1)
    allowed = 2.0 ** -8 * ref.norm(dim=-1) + (p * value_off).sum(-1) + torch.expm1(2 * d) * 2 * spread
    allowed += (2.0 ** -8 if bf16 else 2.0 ** -11) * spread
    if not bf16:
        seen = torch.isfinite(x)
        allowed += 2.0 ** -25 * (p * s).amax(-1) * torch.where(seen, size / s, 0.0).sum(-1)
        allowed += 2.0 ** -25 * 2.0 ** 8 * math.sqrt(128) * (p * s).sum(-1)
    err = (out.double() - ref).norm(dim=-1)
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
    assert bool((err <= allowed).all()), float((err / allowed).max())
    assert bool(((lse.double() - ref_lse).abs() <= d + 2.0 ** -22 * (1 + ref_lse.abs()) + 2.0 ** -24 * L).all())


def inputs(T, L, H, seed):
    m = W.mha_prefill_inputs(T, L - T, H=H, seed=seed)
    return m.q.to(DEV), m.w_ukv.to(DEV)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("e", [-60, -30, -16, 12, 60])
def test_one_scale_far_from_one(e, bf16):
    """All blocks alike, the query the inverse, so that the scores are those of unit rows: the outputs are
    the unit ones times the scale, at the tolerances of the calls with one scale."""
    T, L, H = 130, 300, 2
    kv = cache([L], 16, 3, low=e, high=e)
    q, w = inputs(T, L, H, 5)
    q = (q.float() * 2.0 ** -(e + 6)).bfloat16()
    out, lse = mla.mla_prefill_mha(kv, q, w, SM, L=L, bf16=bf16)
    ref, ref_lse = reference(kv, q, w, L)[:2]
    kw = dict(rel_l2=parity.MHA_BF16_REL_L2, lse_rel=parity.MHA_BF16_LSE_REL) if bf16 else {}
    unit = 2.0 ** -(e + 6)
    compare(out.double().cpu().numpy() * unit, lse, (ref.cpu().numpy() * unit, ref_lse.cpu().numpy()), "one", **kw)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("T,L,H,block,page_size,low,high", [
    (200, 200, 2, 16, 64, -30, 12), (130, 500, 3, 1, 192, -24, -4), (97, 97, 4, 64, 64, -12, 0), (300, 777, 2, 32, 128, -8, -5)])
def test_mixed_scales(T, L, H, block, page_size, low, high, odd, bf16):
    """Blocks of any size side by side (with no prefix, the first positions see small blocks alone), powers
    of two or not. The query keeps the largest rows' scores near unit ones."""
    kv = cache([L], block, T, page_size, low=low, high=high, odd=odd)
    q, w = inputs(T, L, H, 7)
    q = (q.float() * 2.0 ** -(high + 6)).bfloat16()
    out, lse = mla.mla_prefill_mha(kv, q, w, SM, L=L, bf16=bf16)
    check_rows(kv, q, w, L, out, lse, bf16, odd)


@pytest.mark.parametrize("bf16", [False, True])
def test_small_blocks_first(bf16):
    """Positions that see blocks of 2^-40 alone, before blocks of 2^3: their outputs are of the small size."""
    T = L = 260
    kv = cache([L], 16, 9, low=3, high=3)
    first = kv.page_table[0, :2].long()
    kv.scales[first] = 2.0 ** -40
    q, w = inputs(T, L, 2, 11)
    q = (q.float() * 2.0 ** -9).bfloat16()
    out, lse = mla.mla_prefill_mha(kv, q, w, SM, L=L, bf16=bf16)
    check_rows(kv, q, w, L, out, lse, bf16, False)
    assert 2.0 ** -50 < float(out[:128].abs().max()) < 2.0 ** -20


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,L,H,block", [(1280, 2280, 16, 16), (1, 95, 3, 16), (1, 97, 16, 16), (96, 96, 1, 16),
                                         (129, 4000, 12, 16), (1280, 2280, 16, 2), (129, 1999, 12, 8), (50, 113, 4, 1)])
def test_units_and_tiles(T, L, H, block, bf16):
    """Whole units, units cut along the keys, tiles that end inside the keys."""
    kv = cache([L], block, T, low=-8, high=-5)
    q, w = inputs(T, L, H, 13)
    ws = torch.zeros(mla.library().mla_prefill_mha_workspace_size(L, H, 0), dtype=torch.uint8, device=DEV)
    ws[256:] = 0xFF  # (NaN in whatever is read before it is written)
    out, lse = mla.mla_prefill_mha(kv, q, w, SM, L=L, ws=ws, bf16=bf16)
    assert mla.mla_read_status(ws) == 0
    # (the bf16 form's tolerances in parity.py are those of unit keys, which the codes' 80 under 2^-5 pass by a
    # factor of 2.5: the scores' errors, which grow with the keys, are in the rows' bounds)
    check_rows(kv, q, w, L, out, lse, bf16, False)
    if not bf16:
        ref, ref_lse = reference(kv, q, w, L)[:2]
        compare(out, lse, (ref.cpu().numpy(), ref_lse.cpu().numpy()), "units")


@pytest.mark.parametrize("bad", [float("nan"), 0.0, -0.5, float("inf"), 2.0 ** -61, 2.0 ** 61])
def test_scales_that_are_none(bad):
    """Precise form: rows that see such a position are NaN, the others as if it had any scale."""
    T, L, H = 150, 333, 2
    kv = cache([L], 1, 15, low=-7, high=-6)
    q, w = inputs(T, L, H, 17)
    want = mla.mla_prefill_mha(kv, q, w, SM, L=L)
    at = 300  # new position 117's
    kv.scales[kv.page_table[0, at // 64].long(), at % 64] = bad
    kv.scales[kv.page_table[0, L // 64].long(), L % 64:] = bad  # behind the last position
    got = mla.mla_prefill_mha(kv, q, w, SM, L=L)
    j = at - (L - T)
    for a, b in zip(got, want):
        assert torch.equal(a[:j], b[:j]) and bool(torch.isnan(a[j:].float()).all())
    out, lse = mla.mla_prefill_mha(kv, q, w, SM, L=L, bf16=True)
    assert bool(torch.isnan(out[j:].float()).all()) and bool(torch.isnan(lse[j:]).all())


@pytest.mark.parametrize("bf16", [False, True])
def test_bad_page(bf16):
    """A page outside the pool is reported; its positions count as zeros, the new ones before it stay."""
    T, L, H = 150, 333, 2
    kv = cache([L], 16, 19, low=-7, high=-6)
    q, w = inputs(T, L, H, 21)
    ws = torch.zeros(mla.library().mla_prefill_mha_workspace_size(L, H, 0), dtype=torch.uint8, device=DEV)
    want = mla.mla_prefill_mha(kv, q, w, SM, L=L, ws=ws, bf16=bf16)
    assert mla.mla_read_status(ws) == 0
    kv.page_table[0, 4] = kv.pool.shape[0]
    got = mla.mla_prefill_mha(kv, q, w, SM, L=L, ws=ws, bf16=bf16)
    assert mla.mla_read_status(ws) == mla.MLA_ERR_BOUNDS
    j = 256 - (L - T)
    for a, b in zip(got, want):
        assert torch.equal(a[:j], b[:j]) and bool(torch.isfinite(a.float()).all())


def test_captured_and_on_another_stream():
    T, L, H = 200, 500, 3
    kv = cache([L], 16, 23, low=-9, high=-5)
    q, w = inputs(T, L, H, 25)
    ws = torch.zeros(mla.library().mla_prefill_mha_workspace_size(L, H, 0), dtype=torch.uint8, device=DEV)
    want = mla.mla_prefill_mha(kv, q, w, SM, L=L)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = mla.mla_prefill_mha(kv, q, w, SM, L=L, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.mla_prefill_mha(kv, q, w, SM, L=L, out=out, lse=lse, ws=ws)
    for _ in range(2):
        out.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip((out, lse), want, got):
            assert torch.equal(a, b) and torch.equal(c, b)
    kv.scales *= 2.0 ** -3  # the next replay reads the scales of its own time
    graph.replay()
    again = mla.mla_prefill_mha(kv, q, w, SM, L=L)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
