"""A key that a tree's mask hides from a node cannot reach it, whatever its cache row holds: NaN codes
in rows that other nodes of the same group see (a padding node's own, a drafted node's)."""
import numpy as np
import pytest
import torch

from tests.test_nan_rows_gpu import cached, compare
from tests.test_verify_tree_gpu import reference, run, tree_masks
from mla_latent_kv_attention_gb300 import workloads as W

pytestmark = pytest.mark.gpu

# groups of 16, 32 and 48 rows, by the table's width (one user): several nodes a group
GROUPS = [(5, 9, 500), (7, 8, 500), (12, 8, 3000), (12, 8, 9000), (1, 64, 700), (16, 7, 20000), (2, 33, 300)]


@pytest.mark.parametrize("H,n,L", GROUPS)
@pytest.mark.parametrize("code", [0x7F, 0xFF])
def test_padding_nodes_that_see_themselves(H, n, L, code):
    """The last third of the nodes pads: masks of their own bit alone, cache rows never written.
    The drafted nodes come out as without them."""
    inp = W.make_inputs("padding", [L, n], H=H, n_q=n, seed=H + n)
    real = n - n // 3
    rows = tree_masks(2, n, seed=n)
    for b in range(2):
        for j in range(real, n):
            rows[b][j] = 1 << j
            cached(inp, b, int(inp.seq_lens[b]) - n + j)[:] = code
    inp.q[0, 0, 0] = 0  # a query of zeros, the first row of its group: its score with NaN is NaN too
    inp.q[1, n // 2] = 0
    ref = reference(inp, rows)
    assert np.isfinite(ref[1][:, :real]).all() and np.isnan(ref[1][:, real:]).all()
    compare(*run(inp, rows), *ref, f"H={H} n={n} L={L}")


@pytest.mark.parametrize("H,n,L", GROUPS)
@pytest.mark.parametrize("dims", [slice(0, 576), slice(3, 4), slice(300, 301), slice(511, 512), slice(570, 571)])
def test_a_drafted_node_with_nan(H, n, L, dims):
    """One node in the middle of the tree: it and its descendants are NaN, whatever part of its
    row holds the code (one latent dim, a RoPE dim alone, all)."""
    inp = W.make_inputs("middle", [L, 130], H=H, n_q=n, seed=2 * H + n)
    rows = tree_masks(2, n, seed=3)
    at = n // 2
    cached(inp, 0, L - n + at)[dims] = 0x7F
    ref = reference(inp, rows)
    sees = [bool(m >> at & 1) for m in rows[0]]
    assert sees[at] and not all(sees) and np.array_equal(np.isnan(ref[1][0, :, 0]), sees)
    compare(*run(inp, rows), *ref, f"H={H} n={n} L={L} {dims}")


@pytest.mark.parametrize("H,n,L", GROUPS)
def test_queries_and_keys_with_nan(H, n, L):
    """NaN in the first query row of the first group, beside keys without any: the other rows of
    the group keep their values; and beside a node's key with NaN."""
    inp = W.make_inputs("both", [L, 200], H=H, n_q=n, seed=3 * H + n)
    rows = tree_masks(2, n, seed=4)
    inp.q[0, 0, 0, 9] = inp.q[1, 0, 0, 9] = float("nan")
    cached(inp, 1, 200 - 1)[:] = 0x7F  # the last node's
    rows[0][n - 1] &= ~1
    compare(*run(inp, rows), *reference(inp, rows), f"H={H} n={n} L={L}")


@pytest.mark.parametrize("H,n,L", GROUPS)
def test_nodes_across_a_tile(H, n, L):
    """Nodes that straddle the border of two key tiles, every second one with NaN, each seen by
    itself alone; a node that none sees between them."""
    L = L // 128 * 128 + max(1, n // 2)
    inp = W.make_inputs("border", [L], H=H, n_q=n, seed=4 * H + n)
    rows = [[1 << j if j % 2 else (1 << j) | 1 for j in range(n)]]
    for j in range(1, n, 2):
        cached(inp, 0, L - n + j)[j % 576:] = 0xFF if j % 4 == 1 else 0x7F
    rows[0][n - 1] = 1
    ref = reference(inp, rows)
    assert np.isfinite(ref[1][0, 0::2]).all()
    compare(*run(inp, rows), *ref, f"H={H} n={n} L={L}")
