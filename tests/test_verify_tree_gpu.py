"""mla_verify_tree against float64 attention over the dequantised rows, at the tolerances of the
other attention calls (tests/parity.py: the kernel and its arithmetic are theirs; only the
visible keys differ).

One bound is parity.py's relative one: a node that sees few keys gives close to one value row,
whose N(0, 1) entries reach 4 and more; rounding an entry of [4, 8) to bfloat16 is off by up to
half of 2^-5 = 1.6e-2, more than the absolute 1e-2 meant for averages of many keys. So the largest
error is taken relative to max(1, the row's largest entry), where that rounding is at most 2^-8."""
import math
import random

import numpy as np
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import workloads as W
from tests import parity

pytestmark = pytest.mark.gpu
DEV = "cuda"


def compare(out, lse, ref_out, ref_lse, what):
    return parity.compare(out, lse, ref_out, ref_lse, what, max_abs_row=parity.MAX_ABS)


def tree_masks(B, n, seed, reach=4):
    """Ancestor masks of random trees: node j hangs below one of the `reach` nodes before it."""
    r = random.Random(seed)
    rows = []
    for _ in range(B):
        seen = []
        for j in range(n):
            seen.append((seen[r.randint(max(0, j - reach), j - 1)] if j else 0) | 1 << j)
        rows.append(seen)
    return rows


def as_tensor(rows):
    return torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in rows], dtype=torch.int64)


def reference(inp, rows):
    """float64 attention node by node: prefix, then the nodes the mask names."""
    B, n, H = inp.q.shape[:3]
    out = np.zeros((B, n, H, 512))
    lse = np.full((B, n, H), -np.inf)
    for b in range(B):
        L = int(inp.seq_lens[b])
        if L == 0:
            continue
        pages = inp.page_table[b, :-(-L // inp.page_size)].long()
        k = inp.pool[pages].reshape(-1, 576)[:L].view(torch.float8_e4m3fn).to(torch.float64) * inp.kv_scale
        for j in range(n):
            seen = [p for p in range(max(0, L - n))]
            seen += [L - n + i for i in range(n) if rows[b][j] >> i & 1 and L - n + i >= 0]
            if not seen:
                continue
            x = inp.q[b, j].double() @ k[seen].T * inp.sm_scale
            lse[b, j] = torch.logsumexp(x, -1)
            out[b, j] = torch.softmax(x, -1) @ k[seen][:, :512]
    return out, lse


def run(inp, rows, **kw):
    kv = mla.KVCache.from_inputs(inp, DEV)
    ws = mla.workspace(mla.MLA_OP_VERIFY_TREE, inp.B, inp.H, inp.n_q, DEV)
    out, lse = mla.mla_verify_tree(kv, inp.q.to(DEV), as_tensor(rows).to(DEV), inp.sm_scale, ws=ws, **kw)
    assert mla.mla_read_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("H,n", [(12, 1), (12, 2), (12, 4), (12, 5), (12, 8), (1, 64), (1, 33), (16, 3), (16, 7),
                                 (16, 64), (8, 16), (5, 13), (7, 6), (11, 9), (13, 4), (2, 24), (3, 17)])
def test_shapes(H, n):
    """Every way nodes fall into groups: one group, several, a short last one; 16, 32, 48 rows."""
    lens = [n, n + 1, 400, 1000 + n, 127 + n, 128 + n]
    inp = W.make_inputs("tree", lens, H=H, n_q=n, seed=100 * H + n)
    rows = tree_masks(len(lens), n, seed=n)
    ref = reference(inp, rows)
    compare(*run(inp, rows), *ref, f"H={H} n={n}")


@pytest.mark.parametrize("B,H,n,lens", [(1, 12, 8, [20000]), (3, 12, 16, [9000, 70, 5000]), (40, 12, 6, None),
                                        (2, 16, 64, [3000, 4500])])
def test_long_and_batched(B, H, n, lens):
    """Sequences split over many CTAs, and more groups than CTAs."""
    r = random.Random(B)
    lens = lens or [r.randint(n, 2500) for _ in range(B)]
    inp = W.make_inputs("tree", lens, H=H, n_q=n, seed=B + n)
    rows = tree_masks(B, n, seed=B)
    ref = reference(inp, rows)
    compare(*run(inp, rows), *ref, f"B={B} n={n}")


@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_chain_is_verify(n):
    """A chain's masks give what mla_verify gives: the same kernel and split (12 heads: up to 48
    rows), apart from when a row's running max moves. Both are within 2^-8 of the same row's
    exact value by bfloat16's rounding alone, so they may differ by one step of it."""
    inp = W.make_inputs("chain", [900, 4100, 64, 20000], H=12, n_q=n, seed=n)
    rows = [[(2 << j) - 1 for j in range(n)]] * 4
    out, lse = run(inp, rows)
    kv = mla.KVCache.from_inputs(inp, DEV)
    want, want_lse = mla.mla_verify(kv, inp.q.to(DEV), inp.sm_scale)
    a, b = out.double(), want.double()
    assert torch.all((a - b).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + 1e-4)
    assert torch.all((lse - want_lse).abs() <= 2e-6 * (1 + want_lse.abs()))


def test_masks_of_any_kind():
    """Nothing at all, everything, later nodes, single nodes, bits past n; on prefixes that are
    empty (the rows then see nothing), short and long. Padding nodes' rows hold NaN codes."""
    n, H = 9, 12
    lens = [n, n, 300, 2 * n, 140]
    inp = W.make_inputs("masks", lens, H=H, n_q=n, seed=7)
    every = (1 << n) - 1
    rows = [[0, 1, every, 1 << 8, 0, every ^ 1, 2, 0, 1 << 3],
            [0] * n,
            [0] * n,
            [every | 1 << 63 | 1 << 40] * n,
            [(2 << j) - 1 for j in range(5)] + [1] * 4]  # nodes 5..8 pad: nobody sees them
    ref = reference(inp, [[m & every for m in row] for row in rows])
    assert np.isneginf(ref[1][0, 0]).all() and np.isneginf(ref[1][1]).all()
    for b, first in ((1, 0), (4, 5)):  # keys that no node sees
        for i in range(first, n):
            pos = lens[b] - n + i
            inp.pool[int(inp.page_table[b, pos // 64]), pos % 64] = 0x7F
    compare(*run(inp, rows), *ref, "masks")


def test_short_and_empty_sequences():
    """A padded batch: no cached position at all, and fewer than n (the missing ones are the
    first nodes' keys)."""
    n = 6
    inp = W.make_inputs("short", [0, 3, 500, 1, 0], H=12, n_q=n, seed=11)
    rows = [[(2 << j) - 1 for j in range(n)]] * 5
    ref = reference(inp, rows)
    assert np.isneginf(ref[1][1, :3]).all() and np.isfinite(ref[1][1, 3:]).all()
    compare(*run(inp, rows), *ref, "short")


@pytest.mark.parametrize("B,H,n,top", [(30, 16, 64, 260), (200, 12, 2, 130), (160, 1, 20, 70), (90, 5, 9, 900),
                                       (25, 11, 31, 400)])
def test_many_short_sequences(B, H, n, top):
    """Many units a CTA, most of them one tile long: query images staged ahead, their scales and
    buffers handed over as soon as the unit before is done (16, 32 and 48 rows a unit)."""
    r = random.Random(B)
    lens = [r.choice([0, n, r.randint(n, top), r.randint(n, top)]) for _ in range(B)]
    inp = W.make_inputs("many", lens, H=H, n_q=n, seed=B)
    rows = tree_masks(B, n, seed=B)
    ref = reference(inp, rows)
    first = run(inp, rows)
    compare(*first, *ref, f"B={B}")
    for _ in range(5):  # and the same every time
        out, lse = run(inp, rows)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("page_size,contiguous", [(128, False), (192, False), (64, True)])
def test_page_sizes(page_size, contiguous):
    n = 10
    inp = W.make_inputs("pages", [1500, 333, n], H=12, n_q=n, seed=page_size, page_size=page_size,
                        contiguous=contiguous)
    rows = tree_masks(3, n, seed=2)
    compare(*run(inp, rows), *reference(inp, rows), f"page_size={page_size}")


def test_wide_table_takes_the_same_answers():
    """The groups follow the page table's width: a short sequence in a wide table (large groups)
    and in a narrow one (small groups) gives the same rows."""
    n = 8
    inp = W.make_inputs("narrow", [700], H=12, n_q=n, seed=3)
    rows = tree_masks(1, n, seed=3)
    ref = reference(inp, rows)
    compare(*run(inp, rows), *ref, "narrow")
    wide = torch.full((1, 2000), -1, dtype=torch.int32)
    wide[:, :inp.page_table.shape[1]] = inp.page_table
    inp.page_table = wide
    compare(*run(inp, rows), *ref, "wide")


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, give what they give alone; without an
    lse the outputs are the same."""
    n = 12
    a = W.make_inputs("a", [5000, 800], H=12, n_q=n, seed=1)
    b = W.make_inputs("b", [300] * 20, H=12, n_q=n, seed=2)
    made = []
    for inp, seed in ((a, 1), (b, 2)):
        kv = mla.KVCache.from_inputs(inp, DEV)
        made.append((kv, inp.q.to(DEV), as_tensor(tree_masks(inp.B, n, seed)).to(DEV),
                     mla.workspace(mla.MLA_OP_VERIFY_TREE, inp.B, 12, n, DEV)))
    alone = [mla.mla_verify_tree(kv, q, m, a.sm_scale, ws=ws) for kv, q, m, ws in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, (kv, q, m, ws) in zip(streams, made):
            with torch.cuda.stream(s):
                got.append(mla.mla_verify_tree(kv, q, m, a.sm_scale, ws=ws))
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, alone):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    kv, q, m, ws = made[0]
    out = torch.zeros_like(alone[0][0])
    assert mla.library().mla_verify_tree(kv.c_struct(), q.data_ptr(), a.B, n, 12, a.sm_scale, m.data_ptr(),
                                         out.data_ptr(), None, ws.data_ptr(), ws.numel(), None) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, alone[0][0])


def test_dominant_key_over_a_long_tail():
    """One prefix key far above the others, and siblings whose keys it must not see."""
    inp = W.attention_sink(L=30000, H=12, n_q=7, B=1, seed=3)
    rows = tree_masks(1, 7, seed=1, reach=7)
    ref = reference(inp, rows)
    compare(*run(inp, rows), *ref, "sink")


def test_bounds_status():
    n = 5
    inp = W.make_inputs("bad", [300, 200], H=12, n_q=n, seed=1)
    kv = mla.KVCache.from_inputs(inp, DEV)
    kv.page_table[1, 1] = kv.pool.shape[0] + 5
    rows = as_tensor(tree_masks(2, n, 1)).to(DEV)
    ws = mla.workspace(mla.MLA_OP_VERIFY_TREE, 2, 12, n, DEV)
    mla.mla_verify_tree(kv, inp.q.to(DEV), rows, inp.sm_scale, ws=ws)
    assert mla.mla_read_status(ws) == mla.MLA_ERR_BOUNDS
    kv = mla.KVCache.from_inputs(inp, DEV)
    kv.seq_lens[0] = 64 * kv.page_table.shape[1] + 1
    out, lse = mla.mla_verify_tree(kv, inp.q.to(DEV), rows, inp.sm_scale, ws=ws)
    assert mla.mla_read_status(ws) == mla.MLA_ERR_BOUNDS
    kv = mla.KVCache.from_inputs(inp, DEV)
    out, lse = mla.mla_verify_tree(kv, inp.q.to(DEV), rows, inp.sm_scale, ws=ws)
    assert mla.mla_read_status(ws) == 0


@pytest.mark.parametrize("B,n", [(2, 8), (40, 1), (30, 7)])
def test_bounded_wait_reports_timeout(B, n):
    """Waits that nothing satisfies (the test hook switches one call's key loads off) give up after
    their limit, in every warp of a warpgroup and in CTAs with several units: the kernel
    returns, the status says so, and the next call on the workspace is correct."""
    inp = W.make_inputs("stall", [900] * B, H=12, n_q=n, seed=41)
    kv = mla.KVCache.from_inputs(inp, DEV)
    q, rows = inp.q.to(DEV), tree_masks(B, n, 1)
    mask = as_tensor(rows).to(DEV)
    ws = mla.workspace(mla.MLA_OP_VERIFY_TREE, B, 12, n, DEV)
    mla.library().mla_test_stall_next_call()
    mla.mla_verify_tree(kv, q, mask, inp.sm_scale, ws=ws)
    assert mla.mla_read_status(ws) == mla.MLA_ERR_TIMEOUT
    out, lse = mla.mla_verify_tree(kv, q, mask, inp.sm_scale, ws=ws)
    assert mla.mla_read_status(ws) == 0
    compare(out, lse, *reference(inp, rows), "after a timed-out call")


def test_captured_and_replayed():
    """A captured call reads new queries, masks and lengths when it is replayed, on a side
    stream; two graphs may share a workspace when they run one after the other."""
    n = 8
    inp = W.make_inputs("graph", [700, 1500], H=12, n_q=n, seed=5)
    other = W.make_inputs("graph", [700, 1500], H=12, n_q=n, seed=6)
    kv = mla.KVCache.from_inputs(inp, DEV)
    q = inp.q.to(DEV)
    mask = as_tensor(tree_masks(2, n, 1)).to(DEV)
    ws = mla.workspace(mla.MLA_OP_VERIFY_TREE, 2, 12, n, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = mla.mla_verify_tree(kv, q, mask, inp.sm_scale, ws=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            mla.mla_verify_tree(kv, q, mask, inp.sm_scale, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    want = mla.mla_verify_tree(kv, other.q.to(DEV), mask.flip(0), inp.sm_scale)
    q.copy_(other.q)
    mask.copy_(mask.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_refusals():
    n = 4
    inp = W.make_inputs("refuse", [300, 200], H=12, n_q=n, seed=1)
    kv = mla.KVCache.from_inputs(inp, DEV)
    q, mask = inp.q.to(DEV), as_tensor(tree_masks(2, n, 1)).to(DEV)
    for bad in (mask.int(), mask[:, :3], mask[:1], mask.cpu()):
        with pytest.raises(ValueError):
            mla.mla_verify_tree(kv, q, bad, inp.sm_scale)
    with pytest.raises(ValueError):
        mla.mla_verify_tree(kv, q.expand(2, n, 12, 576)[:1].expand(3, n, 12, 576).contiguous(),
                            mask[:1].expand(3, n).contiguous(), inp.sm_scale)
    with pytest.raises(mla.MlaError):
        mla.mla_verify_tree(kv, q, mask, inp.sm_scale, ws=torch.zeros(4096, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        mla.workspace(mla.MLA_OP_VERIFY_TREE, 2, 12, 65, DEV)
