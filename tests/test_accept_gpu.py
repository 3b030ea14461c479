"""mla_accept_drafts against its definition, restated here node by node in whole numbers (Python
integers, no rounding): every output has to be equal."""
import random

import numpy as np
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla

pytestmark = pytest.mark.gpu
DEV = "cuda"


def weight(w):
    """float32 probabilities as whole multiples of 2^-43 (ties to even; exact in float64)."""
    w = np.where(np.asarray(w, np.float32) > 0, np.minimum(w, np.float32(1)), np.float32(0))
    return np.rint(w.astype(np.float64) * 2.0 ** 43).astype(np.int64)


def uniform(u, bits):
    u = float(u) if u > 0 else 0.0
    return min(int(min(u, 1.0) * 2 ** bits), 2 ** bits - 1)


def reference(p, tokens, u, parents=None, q=None):
    B, n, V = p.shape
    out, path, count = (np.full((B, n), -1), np.full((B, n), -1), np.zeros(B, int))
    for b in range(B):
        par = list(range(-1, n - 1)) if parents is None else [int(x) for x in parents[b]]
        real = [j > 0 and 0 <= tokens[b, j] < V and 0 <= par[j] < j for j in range(n)]
        at = 0
        path[b, 0] = 0
        while True:
            kids = [j for j in range(1, n) if real[j] and par[j] == at]
            row, took = weight(p[b, at]), None
            if q is None:
                below, had = 0, set()
                for j in kids:
                    if tokens[b, j] in had:
                        continue
                    had.add(tokens[b, j])
                    if below <= uniform(u[b, at], 43) < below + int(row[tokens[b, j]]):
                        took = j
                    below += int(row[tokens[b, j]])
            else:
                for j in kids:
                    ua = np.float32(min(max(u[b, at], 0.0), 1 - 2.0 ** -24)) if u[b, at] == u[b, at] else 0
                    with np.errstate(invalid="ignore"):
                        if np.float32(ua) * np.float32(q[b, j - 1, tokens[b, j]]) < p[b, at, tokens[b, j]]:
                            took = j
            if took is None:
                break
            out[b, count[b]] = tokens[b, took]
            count[b] += 1
            at = took
            path[b, count[b]] = at
        left = row.copy()
        if q is None:
            left[[tokens[b, j] for j in kids]] = 0
        elif kids:
            with np.errstate(invalid="ignore"):
                left = weight(np.asarray(p[b, at], np.float32) - np.asarray(q[b, at], np.float32))
        if left.sum() == 0:
            left = row
        total = int(left.sum())
        if total > 0:
            mark = total * uniform(u[b, n], 31) >> 31
            out[b, count[b]] = np.searchsorted(np.cumsum(left), mark, side="right")
    return out, path, count


def check(p, tokens, u, parents=None, q=None):
    dev = [None if t is None else torch.as_tensor(t).to(DEV) for t in (p, tokens, u, parents, q)]
    got = mla.mla_accept_drafts(dev[0], dev[1], dev[2], parents=dev[3], draft_probs=dev[4])
    host = [None if t is None else t.cpu().numpy() for t in dev]
    want = reference(*host)
    for g, w, name in zip(got, want, ("tokens", "path", "accepted")):
        assert np.array_equal(g.cpu().numpy(), w), name
    return want


def inputs(B, n, V, tree, drafted, seed, sharp=4.0):
    g = torch.Generator().manual_seed(seed)
    r = random.Random(seed)
    parents = torch.tensor([[-1] + [r.randint(max(0, j - 3), j - 1) if tree else j - 1 for j in range(1, n)]
                            for _ in range(B)], dtype=torch.int32)
    logits = sharp * torch.randn(B, n, V, generator=g)
    guess = torch.softmax(logits + 0.5 * torch.randn(B, n, V, generator=g), -1)
    guess = torch.take_along_dim(guess, parents[:, 1:, None].clamp(min=0).long(), 1)
    tokens = torch.zeros(B, n, dtype=torch.int32)
    if n > 1:
        tokens[:, 1:] = torch.multinomial(guess.reshape(-1, V), 1, generator=g).view(B, n - 1).int()
    u = torch.rand(B, n + 1, generator=g)
    return torch.softmax(logits, -1), tokens, u, parents if tree else None, guess if drafted else None


@pytest.mark.parametrize("tree,drafted", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (3, 2, 5), (8, 4, 1000), (5, 64, 257), (4, 33, 4096), (2, 3, 40001),
                                   (6, 8, 32000)])
def test_random(B, n, V, tree, drafted):
    check(*inputs(B, n, V, tree, drafted, seed=n + V))


@pytest.mark.parametrize("V", [129280, 163840, 262147, 1 << 19])
def test_vocabularies(V):
    check(*inputs(2, 3, V, False, True, seed=1))
    check(*inputs(2, 5, V, True, False, seed=2))


@pytest.mark.parametrize("B", [1, 40, 310])
@pytest.mark.parametrize("w", [2.0 ** -21 * (1 - 2.0 ** -10), 2.0 ** -21 * (1 + 2.0 ** -10), 2.0 ** -19])
def test_largest_rows_of_equal_weights(B, w):
    """Every weight of a row of 2^19 the same, where the fine halves of the sums are largest (to
    either side); one CTA a sequence, several, eight."""
    V = 1 << 19
    p = torch.full((B, 1, V), w, device=DEV)
    u = torch.rand(B, 2, generator=torch.Generator().manual_seed(B))
    out, _, _ = mla.mla_accept_drafts(p, torch.zeros(B, 1, dtype=torch.int32, device=DEV), u.to(DEV))
    W = int(weight(np.float32(w)))
    want = [(V * W * uniform(x, 31) >> 31) // W for x in u[:, 1].numpy()]
    assert out[:, 0].tolist() == want


def test_many_sequences():
    _, _, count = check(*inputs(300, 6, 2000, False, True, seed=3))
    assert 0 < count.mean() < 5 and count.max() == 5  # every outcome, all drafts accepted among them
    check(*inputs(300, 12, 999, True, False, seed=4))


def test_every_number_of_the_draw():
    """Probabilities in eighths and thresholds on their borders: a border belongs to the token
    above it, zero-probability tokens are never drawn, ends included."""
    p = torch.tensor([0, 0.25, 0, 0.5, 0.125, 0.125, 0], dtype=torch.float32).repeat(64, 1, 1)
    u = torch.zeros(64, 2)
    u[:, 1] = torch.cat([torch.arange(60) / 60, torch.tensor([1.0, 1 - 2.0 ** -24, -1.0, float("nan")])])
    out, _, _ = check(p, torch.zeros(64, 1, dtype=torch.int32), u)
    assert out[:, 0].tolist()[:15] == [1] * 15 and out[15, 0] == 3  # 15 / 60 = 0.25
    assert out[60:, 0].tolist() == [5, 5, 1, 1]


def test_acceptance_borders_and_rows_without_weight():
    """u * q = p is a refusal; q = 0 accepts whatever p gives; p = q leaves nothing, so the draw
    falls back on p; a row of zeros draws -1; NaN and infinite entries count as 0 and 1."""
    V = 8
    p, q = torch.zeros(7, 2, V), torch.zeros(7, 1, V)
    p[:, :, 0], p[:, :, 1] = 0.5, 0.5
    q[:, 0, 0], q[:, 0, 1] = 0.25, 0.75
    tokens = torch.zeros(7, 2, dtype=torch.int32)
    u = torch.full((7, 3), 0.5)
    tokens[0, 1], u[0, 0] = 1, 2 / 3           # 2/3 * 0.75 = 0.5 (float32): refused
    tokens[1, 1] = 5                           # q = p = 0 there: refused
    q[2, 0], tokens[2, 1] = p[2, 0], 3         # nothing left: from p
    p[3] = 0                                   # no weight anywhere
    p[4, 0, 6], p[4, 0, 7], tokens[4, 1] = float("nan"), float("inf"), 6
    q[5, 0], tokens[5, 1], u[5, 0] = 0, 1, 0.999
    tokens[6, 1] = -1                          # padding: the draw is from p itself
    out, path, count = check(p, tokens, u, q=q)
    assert count.tolist()[:5] == [0] * 5 and count[5] == 1 and out[3, 0] == -1
    assert np.float32(2 / 3) * np.float32(0.75) == np.float32(0.5)


@pytest.mark.parametrize("drafted", [False, True])
def test_uniforms_outside_their_range(drafted):
    """Below 0 and NaN count as 0 (accepted wherever the target gives anything), 1 and above as the
    number below 1."""
    p, tokens, _, _, q = inputs(6, 4, 300, False, drafted, seed=3)
    bad = torch.tensor([float("nan"), -1.0, float("-inf"), 1.0, 7.0, float("inf")])
    _, _, count = check(p, tokens, bad[:, None].expand(6, 5).contiguous(), q=q)
    assert count.tolist()[:3] == [3, 3, 3]


def test_odd_trees():
    """The same token twice among siblings, children without probability, parents that are not
    before their node, tokens outside the vocabulary, nodes below an unusable one."""
    r = random.Random(1)
    B, n, V = 200, 10, 6
    g = torch.Generator().manual_seed(2)
    p = torch.softmax(2 * torch.randn(B, n, V, generator=g), -1)
    p[::3, :, 2] = 0
    tokens = torch.randint(-2, V + 2, (B, n), generator=g).int()
    parents = torch.tensor([[r.randint(-2, n) if r.random() < 0.2 else r.randint(0, max(0, j - 1)) for j in range(n)]
                            for _ in range(B)], dtype=torch.int32)
    _, _, count = check(p, tokens, torch.rand(B, n + 1, generator=g), parents)
    assert count.max() == 2 and 0 < (count > 0).mean() < 1  # (the definition's own counts)


def test_children_that_hold_all_the_weight():
    """p sums to less than one and every token of weight is a child: u above the sum refuses
    all, and the draw falls back on the row."""
    p = torch.tensor([[[0.25, 0.5, 0, 0]] * 3])
    check(p, torch.tensor([[0, 0, 1]], dtype=torch.int32), torch.tensor([[0.9, 0.5, 0.5, 0.4]]),
          torch.tensor([[-1, 0, 0]], dtype=torch.int32))


def test_emits_the_target_distribution():
    """20,000 chains of one draft: the first emitted token is distributed as the target, far
    closer than the draft (5 sigma of a binomial count)."""
    g = torch.Generator().manual_seed(5)
    V, B = 6, 20000
    p = torch.tensor([0.4, 0.3, 0.15, 0.1, 0.05, 0.0])
    q = torch.tensor([0.05, 0.1, 0.15, 0.3, 0.2, 0.2])
    tokens = torch.zeros(B, 2, dtype=torch.int32)
    tokens[:, 1] = torch.multinomial(q, B, replacement=True, generator=g).int()
    u = torch.rand(B, 3, generator=g)
    out, _, _ = mla.mla_accept_drafts(p.expand(B, 2, V).contiguous().to(DEV), tokens.to(DEV), u.to(DEV),
                                      draft_probs=q.expand(B, 1, V).contiguous().to(DEV))
    share = torch.bincount(out[:, 0].cpu().long(), minlength=V).double() / B
    assert torch.all((share - p.double()).abs() <= 5 * (p * (1 - p) / B).sqrt().double() + 1e-12)


def test_misaligned_rows():
    """Rows off the 16-byte grid: the tensors start one element in."""
    p, tokens, u, _, q = inputs(3, 4, 1000, False, True, seed=9)

    def shifted(t):
        d = torch.zeros(t.numel() + 1, device=DEV)[1:].view(t.shape)
        d.copy_(t)
        return d

    got = mla.mla_accept_drafts(shifted(p), tokens.to(DEV), u.to(DEV), draft_probs=shifted(q))
    for g, w in zip(got, reference(p.numpy(), tokens.numpy(), u.numpy(), q=q.numpy())):
        assert np.array_equal(g.cpu().numpy(), w)


def test_refusals():
    p, tokens, u, parents, _ = (None if t is None else t.to(DEV) for t in inputs(3, 4, 100, True, False, seed=1))
    q = torch.zeros(3, 3, 100, device=DEV)
    for bad in (dict(target_probs=p.double()), dict(target_probs=p[0]), dict(target_probs=p[:, :, ::2]),
                dict(tokens=tokens.long()), dict(uniforms=u[:, :4]), dict(parents=parents[:, 1:]),
                dict(draft_probs=q[:, :2]), dict(uniforms=u.cpu())):
        with pytest.raises(ValueError):
            mla.mla_accept_drafts(**dict(dict(target_probs=p, tokens=tokens, uniforms=u), **bad))
    with pytest.raises(mla.MlaError) as e:
        mla.mla_accept_drafts(p, tokens, u, parents=parents, draft_probs=q)
    assert e.value.status == mla.MLA_ERR_UNSUPPORTED
