"""mla_accept_drafts where probabilities lie outside [0, 1]: below 0 they count as 0, above 1 as 1,
NaN is neither accepted nor drawn. Whole numbers: every output has to be equal to that of the same
call on weights brought into range beforehand."""
import numpy as np
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from tests.test_accept_gpu import DEV, inputs, reference

pytestmark = pytest.mark.gpu


def in_range(p, q):
    """The weights that the call's definition gives these: NaN in the target draws and accepts
    nothing (0); where the draft is NaN, 1 leaves nothing of the target."""
    return p.nan_to_num(nan=0.0).clamp(0, 1), None if q is None else q.nan_to_num(nan=1.0).clamp(0, 1)


def spoil(t, seed):
    """A tenth of the entries negative, above one, infinite or NaN."""
    g = torch.Generator().manual_seed(seed)
    odd = torch.tensor([-1.0, -0.25, 1.5, 3e38, float("inf"), float("-inf"), float("nan"), -1e-6, 1.0000001])
    pick = odd[torch.randint(0, len(odd), t.shape, generator=g)]
    return torch.where(torch.rand(t.shape, generator=g) < 0.1, pick, t)


@pytest.mark.parametrize("tree,drafted", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("B,n,V", [(64, 4, 7), (30, 9, 64), (20, 5, 1001), (4, 3, 40000)])
def test_outside_the_range(B, n, V, tree, drafted):
    p, tokens, u, parents, q = inputs(B, n, V, tree, drafted, seed=V)
    p = spoil(p, 1)
    q = None if q is None else spoil(q, 2)
    clean, clean_q = in_range(p, q)
    host = [None if t is None else t.numpy() for t in (clean, tokens, u, parents, clean_q)]
    want = reference(*host)
    if q is not None:  # a NaN draft entry is never accepted (1 would be, under a larger target entry)
        for b in range(B):
            for j in range(1, n):
                if torch.isnan(q[b, j - 1, tokens[b, j]]) and want[2][b] >= j:
                    tokens[b, j] = int(torch.nonzero(~torch.isnan(q[b, j - 1]))[0])
        host[1] = tokens.numpy()
        want = reference(*host)
    dev = [None if t is None else t.to(DEV) for t in (p, tokens, u, parents, q)]
    got = mla.mla_accept_drafts(dev[0], dev[1], dev[2], parents=dev[3], draft_probs=dev[4])
    for a, b, name in zip(got, want, ("tokens", "path", "accepted")):
        assert np.array_equal(a.cpu().numpy(), b), name


def test_small_cases():
    """Draft entries below zero add nothing to what is drawn and accept nothing where the target
    gives nothing; both infinite leave nothing; a NaN draft entry is refused whatever the target."""
    V, nan, inf = 4, float("nan"), float("inf")
    p = torch.tensor([[0.0, 0.5, 0.5, 0.0], [0.25, 0.25, 0.25, 0.25], [inf, 0.5, 0.0, 0.0], [1.0, 0, 0, 0]])
    q = torch.tensor([[-1.0, 0.5, 0.0, -3.0], [-0.5, 1.0, 1.0, 1.0], [inf, 0.0, 0.0, 0.0], [nan, 0.0, 0.0, 0.0]])
    tokens = torch.tensor([[0, 0], [0, 1], [0, 0], [0, 0]], dtype=torch.int32)
    u = torch.tensor([[0.5, 0.9, 0.9], [0.9, 0.0, 0.5], [0.999, 0.0, 0.0], [0.0, 0.0, 0.5]])
    out, path, count = mla.mla_accept_drafts(p[:, None].repeat(1, 2, 1).to(DEV), tokens.to(DEV), u.to(DEV),
                                             draft_probs=q[:, None].contiguous().to(DEV))
    # 0: token 0 has no probability, and what is left is token 2's; 1: 0.9 * 1 is not below 0.25, and
    # token 0's 0.25 is left; 2: accepted (0.999 < 1), the next token from (1, 0.5): 0;
    # 3: refused, nothing left of the row: drawn from it
    assert count.tolist() == [0, 0, 1, 0]
    assert out[:, 0].tolist() == [2, 0, 0, 0] and out[2, 1].item() == 0
