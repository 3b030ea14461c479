"""NaN in queries and in cached rows: a row that sees one comes out NaN (out and lse), every other
row is what it is without it. References are plain float64 (which carry NaN by themselves) at
the tolerances of the other tests of each call."""
import numpy as np
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import workloads as W
from tests import parity
from tests.test_verify_tree_gpu import reference, run, tree_masks

pytestmark = pytest.mark.gpu
DEV = "cuda"


def compare(out, lse, ref_out, ref_lse, what, **kw):
    """NaN for exactly the rows that are NaN in the reference; the others by parity.compare."""
    out, lse = parity.to_np(out), parity.to_np(lse)
    bad = np.isnan(ref_lse)
    assert np.array_equal(np.isnan(lse), bad), f"{what}: lse is NaN for other rows"
    assert np.isnan(out[bad]).all(), f"{what}: rows that see NaN must be NaN"
    assert np.array_equal(np.isnan(out).any(-1), bad), f"{what}: NaN reached rows that see none"
    kw.setdefault("max_abs_row", parity.MAX_ABS)
    parity.compare(np.where(bad[..., None], 0, out), np.where(bad, 0, lse),
                   np.where(bad[..., None], 0, ref_out), np.where(bad, 0, ref_lse), what, **kw)


def cached(inp, b, pos):
    """The codes of position pos of sequence b (a view of the pool)."""
    return inp.pool[int(inp.page_table[b, pos // inp.page_size]), pos % inp.page_size]


def causal(n):
    return [(2 << j) - 1 for j in range(n)]


@pytest.mark.parametrize("H,n,lens,pos", [(12, 8, [700, 300], 5), (12, 8, [20000, 300], 10000), (5, 9, [500, 90], 3),
                                          (16, 64, [9000, 64], 8999 - 64), (12, 16, [9000] * 12, 4000)])
def test_tree_prefix_with_nan(H, n, lens, pos):
    """A prefix row in one piece of many, or in the only one: every node of the sequence is NaN."""
    inp = W.make_inputs("prefix", lens, H=H, n_q=n, seed=n)
    cached(inp, 0, pos)[77] = 0xFF
    rows = tree_masks(len(lens), n, seed=1)
    ref = reference(inp, rows)
    assert np.isnan(ref[1][0]).all() and np.isfinite(ref[1][1:]).all()
    compare(*run(inp, rows), *ref, "prefix")


@pytest.mark.parametrize("H,n,lens", [(12, 8, [700, 300]), (12, 8, [20000, 300]), (5, 9, [500, 9]), (1, 64, [9000]),
                                      (12, 16, [9000] * 12)])
def test_tree_queries_with_nan(H, n, lens):
    """NaN in a query row: that row alone, the first of a group among them; one that sees no key
    stays empty."""
    inp = W.make_inputs("query", lens, H=H, n_q=n, seed=n)
    for k, j in enumerate((0, n // 2, n - 1)):
        inp.q[0, j, k % H, (5, 511, 575)[k]] = float("nan")
    rows = tree_masks(len(lens), n, seed=2)
    rows[-1][n - 1] = 0
    inp.q[-1, n - 1, 0, 0] = float("nan")
    compare(*run(inp, rows), *reference(inp, rows), "queries")


@pytest.mark.parametrize("lens,n,H,pos", [([900, 300], 1, 12, 3), ([142000], 1, 12, 70000), ([20000] * 3, 1, 16, 19998),
                                          ([5000] * 32, 1, 8, 100), ([20000, 500], 4, 12, 9000), ([300] * 160, 2, 12, 7),
                                          ([20000, 500], 4, 16, 9000)])
def test_decode_and_verify(lens, n, H, pos):
    """One NaN query row, one visible cached row with NaN: whole sequences, sequences in a few
    pieces and in as many as there are SMs; bf16 and float32 outputs."""
    inp = W.make_inputs("decode", lens, H=H, n_q=n, seed=len(lens))
    cached(inp, 0, pos)[400] = 0x7F
    if len(lens) > 1:
        inp.q[1, n - 1, H - 1, 8] = float("nan")
    else:  # (the whole sequence is NaN; its next neighbour is another call)
        other = W.make_inputs("decode", lens, H=H, n_q=n, seed=9)
        other.q[0, 0, 3, 8] = float("nan")
        compare(*mla.mla_verify(mla.KVCache.from_inputs(other, DEV), other.q.to(DEV), other.sm_scale),
                *reference(other, [causal(n)]), "one query")
    ref = reference(inp, [causal(n)] * len(lens))
    kv = mla.KVCache.from_inputs(inp, DEV)
    compare(*mla.mla_verify(kv, inp.q.to(DEV), inp.sm_scale), *ref, "verify")
    compare(*mla.mla_verify_f32(kv, inp.q.to(DEV), inp.sm_scale), *ref, "verify_f32")
    if n == 1:
        out, lse = mla.mla_decode(kv, inp.q[:, 0].to(DEV).contiguous(), inp.sm_scale)
        compare(out, lse, ref[0][:, 0], ref[1][:, 0], "decode")


@pytest.mark.parametrize("T,L", [(70, 500), (700, 2000)])
def test_prefill(T, L):
    """Query rows with NaN alone; then a prefix row that every position sees. (Units whole and, in
    the longer one, cut along the keys.)"""
    H = 12
    inp = W.make_inputs("prefill", [L], H=H, n_q=T, seed=T)
    inp.q[0, 3, 1, 0] = inp.q[0, T - 1, H - 1, 575] = float("nan")
    rows = [[(2 << j) - 1 for j in range(T)]]
    for _ in range(2):
        ref = reference(inp, rows)
        out, lse = mla.mla_prefill(mla.KVCache.from_inputs(inp, DEV), inp.q[0].to(DEV).contiguous(), inp.sm_scale)
        compare(out, lse, ref[0][0], ref[1][0], "prefill")
        cached(inp, 0, L - T - 1)[9] = 0x7F
    assert np.isnan(ref[1]).all()


@pytest.mark.parametrize("S,R", [(1, 3), (4, 7), (9, 200), (300, 5), (700, 160)])
def test_merge(S, R):
    """A partial whose lse is NaN makes its row NaN, beside finite ones, beside empty ones and
    alone; past the 256th partial too."""
    g = torch.Generator().manual_seed(S)
    out = torch.randn(S, R, 512, generator=g)
    lse = torch.randn(S, R, generator=g)
    lse[torch.rand(S, R, generator=g) < 0.3] = float("-inf")
    lse[S - 1, 0] = float("nan")
    if R > 3:
        lse[:, 1], lse[0, 1] = float("-inf"), float("nan")
        lse[:, 2], lse[S // 2, 2] = float("-inf"), float("nan")
        lse[:, 3] = float("-inf")
    w = torch.softmax(lse.double(), 0)
    empty = torch.isneginf(lse).all(0)
    want = (torch.where(torch.isneginf(lse), 0.0, w)[..., None] * out.double()).sum(0)
    want[empty] = 0
    want_lse = torch.logsumexp(lse.double(), 0)
    got, got_lse = mla.mla_merge_lse(out.to(DEV), lse.to(DEV))
    assert torch.isnan(want_lse).any() and torch.isnan(want[torch.isnan(want_lse)]).all()
    compare(got, got_lse, want.numpy(), want_lse.numpy(), f"S={S} R={R}")


@pytest.mark.parametrize("T,prefix,H", [(200, 300, 2), (300, 0, 3), (1280, 1000, 16)])
@pytest.mark.parametrize("bf16", [False, True])
def test_mha_prefill(T, prefix, H, bf16):
    """Query rows with NaN alone are NaN, the others bit for bit what they are without; then a
    prefix row that every position sees. (In the largest some units are cut along the keys.)"""
    m = W.mha_prefill_inputs(T, prefix, H=H, seed=T)
    w, q = m.w_ukv.to(DEV), m.q.to(DEV)

    def call():
        return mla.mla_prefill_mha(mla.KVCache.from_inputs(m.cache, DEV), q, w, m.cache.sm_scale, bf16=bf16)

    out, lse = call()
    bad = torch.zeros(T, H, dtype=torch.bool, device=DEV)
    bad[[0, T // 2, T - 1], [0, H // 2, H - 1]] = bad[T // 3] = True
    q[..., 150] = torch.where(bad, float("nan"), q[..., 150])
    got, got_lse = call()
    assert torch.isnan(got[bad]).all() and torch.isnan(got_lse[bad]).all()
    assert torch.equal(got[~bad], out[~bad]) and torch.equal(got_lse[~bad], lse[~bad])
    if prefix:
        cached(m.cache, 0, prefix // 2)[17] = 0x7F
        got, got_lse = call()
        assert torch.isnan(got).all() and torch.isnan(got_lse).all()
