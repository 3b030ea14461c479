"""Attention over a cache with block scales against float64 attention over the dequantised rows, at the
tolerances of the calls without (tests/parity.py).

The kernels and their arithmetic are those calls' but for three things: a score is multiplied by its
key's scale and has log2 of it added (float32: one more rounding of a number that is as large as the
score, and the rounded log2, which enters weight and row sum alike), the row sum divides by the scale
(2^-24), and the weights' e5m2 terms are precise relative to the largest weight times scale, which is
relative to the largest term of the output. Each is far below the tolerances. Value rows differ in size
here, so the largest error is taken relative to max(1, the row's largest entry), as for draft trees."""
import math

import numpy as np
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import dcp
from mla_latent_kv_attention_gb300 import workloads as W
from tests import parity
from tests.test_verify_tree_gpu import as_tensor, tree_masks

pytestmark = pytest.mark.gpu
DEV = "cuda"
SM = W.SM_SCALE


def compare(out, lse, want, what, **kw):
    return parity.compare(out, lse, want[0], want[1], what, max_abs_row=parity.MAX_ABS, **kw)


def cache(lens, block, seed, page_size=64, low=-9, high=-5, odd=False):
    """Codes of N(0, 1) rows (about 80 a unit) under random scales a block: powers of two from 2^low to
    2^high, or (odd) any numbers between."""
    inp = W.make_inputs("scaled", lens, H=1, seed=seed, page_size=page_size)
    g = torch.Generator().manual_seed(seed + 1)
    shape = (inp.pool.shape[0], page_size // block)
    e = torch.rand(shape, generator=g) * (high - low) + low if odd else torch.randint(low, high + 1, shape, generator=g)
    return mla.KVCache(inp.pool.to(DEV), inp.page_table.to(DEV), inp.seq_lens.to(DEV), 1.0,
                       scales=torch.exp2(e.float()).to(DEV))


def queries(seed, *shape):
    return torch.randn(*shape, 576, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)


def rows(kv, b, L):
    page = kv.pool.shape[1]
    block = page // kv.scales.shape[1]
    pages = kv.page_table[b, :-(-L // page)].long()
    k = kv.pool[pages].view(torch.float8_e4m3fn).double().view(len(pages), -1, block, 576)
    return (k * kv.scales[pages].double()[:, :, None, None]).reshape(-1, 576)[:L]


def reference(kv, q, masks=None, shift=0):
    """q [B, n, H, 576]: every new position sees the prefix and those before it (moved by `shift`), or the
    nodes that its mask names."""
    B, n, H = q.shape[:3]
    out = torch.zeros(B, n, H, 512, dtype=torch.float64, device=DEV)
    lse = torch.full((B, n, H), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        L = int(kv.seq_lens[b])
        if L <= 0:
            continue
        k = rows(kv, b, L)
        node = torch.arange(L, device=DEV) - (L - n)
        for j in range(n):
            if masks is None:
                keep = node <= j + shift
            else:
                keep = torch.tensor([m < 0 or bool(masks[b][j] >> m & 1) for m in node.tolist()], device=DEV)
            if not bool(keep.any()):
                continue
            x = torch.where(keep, q[b, j].double() @ k.T * SM, -math.inf)
            lse[b, j] = torch.logsumexp(x, -1)
            v = torch.where(keep[:, None], k[:, :512], 0.0)  # (what is hidden may be NaN)
            out[b, j] = torch.where(keep, torch.exp(x - lse[b, j][:, None]), 0.0) @ v
    return out.cpu().numpy(), lse.cpu().numpy()


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("H", [1, 8, 12, 16])
@pytest.mark.parametrize("lens,block,page_size", [
    ([1], 16, 64), ([1024], 64, 64), ([700, 0, 129, 64, 65, 3], 1, 64), ([5000, 127, 128], 32, 192), ([20000], 2, 128),
    ([300] * 200, 8, 64)])
def test_decode(lens, block, page_size, H, odd):
    kv = cache(lens, block, H, page_size, odd=odd)
    q = queries(H + 5, len(lens), H)
    ws = mla.workspace(mla.MLA_OP_DECODE, len(lens), H, 1)
    out, lse = mla.mla_decode(kv, q, SM, ws=ws)
    assert mla.mla_read_status(ws) == 0
    compare(out[:, None], lse[:, None], reference(kv, q[:, None]), "decode")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,H", [(1, 5), (2, 16), (3, 16), (4, 12), (4, 16)])
@pytest.mark.parametrize("lens,block,page_size", [([4, 5000], 16, 64), ([900, 0, 2, 300], 1, 128), ([130] * 70, 64, 64)])
def test_verify(lens, block, page_size, n, H, f32):
    kv = cache(lens, block, n + H, page_size)
    q = queries(n, len(lens), n, H)
    out, lse = (mla.mla_verify_f32 if f32 else mla.mla_verify)(kv, q, SM)
    want = reference(kv, q)
    compare(out, lse, want, "verify")
    assert out.dtype == (torch.float32 if f32 else torch.bfloat16)
    if f32:
        out, lse = mla.mla_verify_f32(kv, q, SM, visible_shift=n + 5)
        compare(out, lse, reference(kv, q, shift=n - 1), "shifted")


@pytest.mark.parametrize("n,H", [(1, 1), (1, 16), (2, 12), (3, 11), (3, 16), (4, 12), (4, 16)])
def test_float32_output(n, H):
    """The float32 output keeps the weights to 2^-18 (six e5m2 terms), or 2^-33 of the row's largest weight
    times scale. A row's error is a mean of the value rows with those errors for weights, so at most 2^-18 of
    about the row's size however the keys' errors add up; the scores' own float32 rounding (up to 46 in log2
    units here, 2^-24 each of product and sum: 2^-17.5 of a weight, of random sign) comes on top. 2e-5 is
    2^-18 and 2^-17.5 with a factor of two; bfloat16's 2^-9 is 100 times that."""
    lens = [5000, n, 0, 333, 128 + n]
    kv = cache(lens, 16, n + H, low=-8, high=-6)
    q = queries(H, len(lens), n, H)
    out, lse = mla.mla_verify_f32(kv, q, SM)
    ref, ref_lse = reference(kv, q)
    got = out.double().cpu().numpy()
    for b in range(len(lens)):
        assert np.linalg.norm(got[b] - ref[b]) <= 2e-5 * np.linalg.norm(ref[b])
    fin = np.isfinite(ref_lse)
    assert np.abs(lse.cpu().numpy()[fin] - ref_lse[fin]).max() <= 1e-5 * np.abs(ref_lse[fin]).max()


@pytest.mark.parametrize("B,n,H,lens,block,page_size", [
    (1, 1, 12, [1000], 16, 64), (3, 8, 12, [2000, 0, 9], 1, 64), (2, 64, 16, [300, 64], 64, 64), (5, 16, 4, [700] * 5, 32, 128),
    (40, 5, 3, [200] * 40, 4, 192), (1, 33, 16, [9000], 8, 64)])
def test_tree(B, n, H, lens, block, page_size):
    kv = cache(lens, block, n + H, page_size)
    q = queries(n, B, n, H)
    masks = tree_masks(B, n, n)
    masks[0][0] = 0  # a node that sees the prefix alone
    ws = mla.workspace(mla.MLA_OP_VERIFY_TREE, B, H, n)
    out, lse = mla.mla_verify_tree(kv, q, as_tensor(masks).to(DEV), SM, ws=ws)
    assert mla.mla_read_status(ws) == 0
    compare(out, lse, reference(kv, q, masks), "tree")


@pytest.mark.parametrize("T,prefix,H,block,page_size", [
    (1, 0, 12, 16, 64), (100, 0, 12, 64, 64), (37, 1000, 16, 1, 128), (200, 333, 5, 32, 192), (650, 100, 12, 16, 64)])
def test_prefill(T, prefix, H, block, page_size):
    kv = cache([prefix + T], block, T, page_size)
    q = queries(T, T, H)
    ws = mla.workspace(mla.MLA_OP_PREFILL, 1, H, T)
    out, lse = mla.mla_prefill(kv, q, SM, ws=ws)
    assert mla.mla_read_status(ws) == 0
    compare(out[None], lse[None], reference(kv, q[None]), "prefill")


def test_prefill_split_last_round():
    """A last round of a few units runs as halves along the keys (the third kernel merges them): 152 full
    units and some."""
    H, sms = 12, torch.cuda.get_device_properties(0).multi_processor_count
    T = 4 * sms + 50
    kv = cache([500 + T], 16, 3)
    q = queries(3, T, H)
    out, lse = mla.mla_prefill(kv, q, SM)
    assert mla.mla_last_launch_count() == 3
    compare(out[None], lse[None], reference(kv, q[None]), "prefill")


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,L,H,block", [(1, 1, 2, 16), (200, 700, 4, 1), (130, 130, 3, 64)])
def test_prefill_mha(T, L, H, block, bf16):
    """Against the up-projection in float64; values and keys of unit size, as the tolerances' derivation has
    them (tests/parity.py), so scales around 1 / 80."""
    kv = cache([L], block, T, low=-7, high=-6)
    m = W.mha_prefill_inputs(T, L - T, H=H, seed=4)
    q, w = m.q.to(DEV), m.w_ukv.to(DEV)
    out, lse = mla.mla_prefill_mha(kv, q, w, SM, L=L, bf16=bf16)
    k = rows(kv, 0, L)
    up = torch.einsum("nc,chd->nhd", k[:, :512], w.double())
    key = torch.cat([up[..., :128], k[:, None, 512:].expand(L, H, 64)], -1)
    x = torch.einsum("thd,nhd->thn", q.double(), key) * SM
    last = L - T + torch.arange(T, device=DEV)
    x.masked_fill_((torch.arange(L, device=DEV) > last[:, None])[:, None, :], -math.inf)
    ref_lse = torch.logsumexp(x, -1)
    ref = torch.einsum("thn,nhd->thd", torch.exp(x - ref_lse[..., None]), up[..., 128:])
    kw = dict(rel_l2=parity.MHA_BF16_REL_L2, lse_rel=parity.MHA_BF16_LSE_REL) if bf16 else {}
    compare(out, lse, (ref.cpu().numpy(), ref_lse.cpu().numpy()), "mha", **kw)


def test_equal_scales_are_one_scale():
    """Every block under the same power of two: the calls with one scale, to rounding."""
    kv = cache([3000, 90], 16, 1, low=-6, high=-6)
    one = mla.KVCache(kv.pool, kv.page_table, kv.seq_lens, 2.0 ** -6)
    q = queries(1, 2, 3, 12)
    for call in (mla.mla_verify, mla.mla_verify_f32):
        (a, la), (b, lb) = call(kv, q, SM), call(one, q, SM)
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())
        assert float((la - lb).abs().max()) <= 1e-5 * float(lb.abs().max())


def test_wide_scales():
    """Blocks 2^12 apart: the largest rows win the softmax where the query likes them and vanish where it
    does not; far below, blocks of the smallest scale (zeros, as the write leaves them) count in the sum."""
    kv = cache([2000, 500], 16, 2, low=-17, high=-5)
    kv.scales.view(-1)[::5] = 2.0 ** -60
    q = queries(2, 2, 4, 12)
    out, lse = mla.mla_verify_f32(kv, q, SM)
    compare(out, lse, reference(kv, q), "wide")


def test_all_blocks_of_the_smallest_or_largest_scale():
    for e in (-60, 60):
        kv = cache([300], 16, 3, low=e, high=e)
        q = (queries(3, 1, 1, 4).float() * 2.0 ** -(e + 6) if e > 0 else queries(3, 1, 1, 4)).bfloat16()
        out, lse = mla.mla_verify_f32(kv, q, SM)
        ref, ref_lse = reference(kv, q)
        parity.compare(out.double().cpu().numpy() * 2.0 ** -(e + 6), lse, ref * 2.0 ** -(e + 6), ref_lse, "edge",
                       max_abs_row=parity.MAX_ABS)


@pytest.mark.parametrize("bad", [float("nan"), 0.0, -0.5, float("inf"), 2.0 ** -61, 2.0 ** 61])
def test_scales_that_are_none(bad):
    """Rows that see such a block are NaN; scales behind the sequence, of other pages and hidden from a
    position by the mask reach nothing."""
    kv = cache([200, 300, 128], 16, 4)
    q = queries(4, 3, 4, 12)
    want = mla.mla_verify_f32(kv, q, SM)
    kv.scales[kv.page_table[0, 200 // 64].long(), (200 % 64) // 16 + 1:] = bad  # behind sequence 0
    kv.scales[kv.page_table[1, 0].long(), 2] = bad                               # seen by all of sequence 1
    got = mla.mla_verify_f32(kv, q, SM)
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]) and bool(torch.isnan(a[1]).all())
    one = cache([130], 1, 5)  # a scale a position: the last new position's is none
    qs = queries(5, 1, 4, 12)
    want = mla.mla_verify_f32(one, qs, SM)
    one.scales[one.page_table[0, 2].long(), 1] = bad
    got = mla.mla_verify_f32(one, qs, SM)
    for a, b in zip(got, want):
        assert torch.equal(a[0, :3], b[0, :3]) and bool(torch.isnan(a[0, 3]).all())
    chain = as_tensor([[1, 3, 7, 15]]).to(DEV)
    got = mla.mla_verify_tree(one, qs, chain, SM)
    assert bool(torch.isnan(got[0][0, 3].float()).all()) and bool(torch.isnan(got[1][0, 3]).all())
    compare(got[0][:, :3], got[1][:, :3], (want[0][:, :3].cpu().numpy(), want[1][:, :3].cpu().numpy()), "hidden")
    out, lse = mla.mla_prefill(one, qs[0], SM)
    assert bool(torch.isnan(out[3].float()).all()) and bool(torch.isfinite(out[:3].float()).all())
    compare(out[None, :3], lse[None, :3], (want[0][:, :3].cpu().numpy(), want[1][:, :3].cpu().numpy()), "hidden")


def test_bad_pages_and_lengths():
    kv = cache([200, 300], 16, 6)
    q = queries(6, 2, 12)
    ws = mla.workspace(mla.MLA_OP_DECODE, 2, 12, 1)
    good = mla.mla_decode(kv, q, SM, ws=ws)
    kv.page_table[1, 3] = kv.pool.shape[0]
    got = mla.mla_decode(kv, q, SM, ws=ws)
    assert mla.mla_read_status(ws) == mla.MLA_ERR_BOUNDS
    assert torch.equal(got[0][0], good[0][0])
    kv.page_table[1, 3] = -7
    kv.seq_lens[0] = 10 ** 9
    got = mla.mla_decode(kv, q, SM, ws=ws)
    assert mla.mla_read_status(ws) == mla.MLA_ERR_BOUNDS


def test_dcp():
    kv = cache([3000, 70, 0, 640], 16, 7)
    q = queries(7, 4, 3, 12)
    out, lse = dcp.dcp_attention(kv, q, SM, 3)
    compare(out, lse, reference(kv, q), "dcp")


def test_scales_past_32_bits():
    """A pool of 5 GiB with a scale for every position; the sequence sits on its last pages."""
    pages = (5 << 30) // (64 * 576)
    pool = torch.zeros(pages, 64, 576, dtype=torch.uint8, device=DEV)
    scales = torch.full((pages, 64), float("nan"), device=DEV)
    small = cache([300], 1, 8)
    n = small.pool.shape[0]
    pool[-n:], scales[-n:] = small.pool, small.scales
    kv = mla.KVCache(pool, small.page_table + (pages - n), small.seq_lens, 1.0, scales=scales)
    q = queries(8, 1, 12)
    for a, b in zip(mla.mla_decode(kv, q, SM), mla.mla_decode(small, q, SM)):
        assert torch.equal(a, b)


def test_refusals():
    kv = cache([100], 16, 9)
    bad = mla.KVCache(kv.pool, kv.page_table, kv.seq_lens, 0.5, scales=kv.scales)
    q = queries(9, 1, 1, 4)
    mask = torch.ones(1, 1, dtype=torch.int64, device=DEV)
    for kv in (bad, mla.KVCache(kv.pool, kv.page_table, kv.seq_lens, 1.0, scales=kv.scales.cpu())):
        for call in (lambda: mla.mla_decode(kv, q[0], SM), lambda: mla.mla_verify(kv, q, SM),
                     lambda: mla.mla_verify_f32(kv, q, SM), lambda: mla.mla_verify_tree(kv, q, mask, SM),
                     lambda: mla.mla_prefill(kv, q[0], SM)):
            with pytest.raises(ValueError):
                call()


def test_another_device():
    """A cache that says it lies on another device than q and the current one is refused (no such device is
    needed: nothing is launched)."""
    from tests.test_kv_cache import OnDevice
    kv = cache([100], 16, 9)
    far = mla.KVCache(*(OnDevice(t, 1) for t in (kv.pool, kv.page_table, kv.seq_lens)), 1.0, scales=OnDevice(kv.scales, 1))
    q = queries(9, 1, 1, 4)
    for call in (lambda: mla.mla_decode(far, q[0], SM), lambda: mla.mla_verify(far, q, SM),
                 lambda: mla.mla_verify_f32(far, q, SM), lambda: mla.mla_prefill(far, q[0], SM)):
        with pytest.raises(ValueError, match="have to be one"):
            call()


def test_more_sequences_than_the_cache_has():
    kv = cache([100, 60], 16, 9)
    q = queries(9, 3, 1, 4)
    for call in (lambda: mla.mla_decode(kv, q[:, 0].contiguous(), SM), lambda: mla.mla_verify(kv, q, SM),
                 lambda: mla.mla_verify_f32(kv, q, SM),
                 lambda: mla.mla_verify_tree(kv, q, torch.ones(3, 1, dtype=torch.int64, device=DEV), SM)):
        with pytest.raises(ValueError, match="sequences"):
            call()
