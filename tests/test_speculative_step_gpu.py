"""The calls of a speculative decoding step run together, as a serving loop would: draft rows
written through norm and rotation, queries rotated, the draft tree verified, drafts accepted
against top-k renormalised probabilities, the accepted path's rows kept, and the cache read
back. Checked by what the step promises: the accepted path attends like plain decoding over
the kept rows, position by position, and the rows read back are the ones attended to."""
import random

import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import workloads as W
from tests import parity

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, V = 12, 4000


def tree(n, r, reach=3):
    """Parents, depths and ancestor masks of a random tree."""
    parents, depth, seen = [-1], [0], [1]
    for j in range(1, n):
        a = r.randint(max(0, j - reach), j - 1)
        parents.append(a)
        depth.append(depth[a] + 1)
        seen.append(seen[a] | 1 << j)
    return parents, depth, [m - (1 << 64) if m >> 63 else m for m in seen]


class Step:
    """One step's buffers and calls (everything on the current stream, nothing waits)."""

    def __init__(self, prefix, n, seed):
        g = torch.Generator().manual_seed(seed)
        r = random.Random(seed)
        self.B, self.n, self.prefix = len(prefix), n, prefix
        inp = W.make_inputs("step", [p + n for p in prefix], H=H, n_q=n, seed=seed)
        self.scale = inp.sm_scale
        self.kv = mla.KVCache.from_inputs(inp, DEV)
        made = [tree(n, r) for _ in prefix]
        self.parents = torch.tensor([m[0] for m in made], dtype=torch.int32, device=DEV)
        depth = torch.tensor([m[1] for m in made], device=DEV)
        self.mask = torch.tensor([m[2] for m in made], dtype=torch.int64, device=DEV)
        start = torch.tensor(prefix, device=DEV)[:, None]
        # node j sits in cache position prefix + j, but its rotary position is its depth's
        self.positions = (start + depth).flatten()
        place = start + torch.arange(n, device=DEV)
        pages = self.kv.page_table.gather(1, place // 64).long()
        self.slots = (pages * 64 + place % 64).flatten()
        rows = self.B * n
        self.latent = torch.randn(rows, 2112, generator=g).bfloat16().to(DEV)[:, 1536:]
        self.q = torch.randn(rows, H, 576, generator=g).bfloat16().to(DEV)
        self.q_rope = torch.randn(rows, H, 192, generator=g).bfloat16().to(DEV)[..., 128:]
        self.weight = (1 + 0.1 * torch.randn(512, generator=g)).bfloat16().to(DEV)
        self.head = (torch.randn(H * 512, V, generator=g) / 30).to(DEV)
        self.tokens = torch.randint(0, V, (self.B, n), generator=g).int().to(DEV)
        u = torch.rand(self.B, n + 1, generator=g)
        u[::2, :n] = 0.0  # every other sequence accepts the first child it comes to
        self.u = u.to(DEV)
        self.rope = mla.mla_rope_init(factor=40.0, original_positions=4096)
        self.ws = mla.workspace(mla.MLA_OP_VERIFY_TREE, self.B, H, n, DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self):
        mla.mla_cache_append_rope(self.kv.pool, self.latent, self.slots, self.kv.kv_scale, self.rope,
                                  self.positions, norm_weight=self.weight, status=self.status)
        mla.mla_rope(self.rope, self.q_rope, self.positions, out=self.q[..., 512:])
        out, lse = mla.mla_verify_tree(self.kv, self.q.view(self.B, self.n, H, 576), self.mask, self.scale,
                                       ws=self.ws)
        probs = torch.softmax(out.float().view(self.B * self.n, -1) @ self.head, -1)
        probs = mla.mla_top_k_renorm_prob(probs, 50).view(self.B, self.n, V)
        # drafts that stand a chance: children take their parent's most likely tokens in turn
        best = probs.topk(8, -1).indices
        turn = (torch.arange(self.n, device=DEV) % 8).expand(self.B, self.n)
        parent = self.parents.clamp(min=0).long()
        drafts = best[torch.arange(self.B, device=DEV)[:, None], parent, turn]
        self.tokens.copy_(drafts.int())
        tokens, path, count = mla.mla_accept_drafts(probs, self.tokens, self.u, parents=self.parents)
        return out, lse, probs, tokens, path, count


def test_accepted_path_is_plain_decoding():
    prefix, n = [700, 64, 3000, 1, 129], 12
    s = Step(prefix, n, seed=21)
    out, lse, probs, tokens, path, count = s.run()
    assert int(s.status) == 0 and mla.mla_read_status(s.ws) == 0
    counts = count.tolist()
    assert max(counts) >= 1
    flat = s.kv.pool.view(-1, 576)
    slots = s.slots.view(s.B, n)
    for b, c in enumerate(counts):
        keep = path[b, :c + 1].long()
        # keep the path: its rows move up behind the prefix
        flat[slots[b, :c + 1]] = flat[slots[b, keep]]
        for k in range(c + 1):
            view = mla.KVCache(s.kv.pool, s.kv.page_table[b:b + 1].contiguous(),
                               torch.tensor([prefix[b] + k + 1], dtype=torch.int32, device=DEV), s.kv.kv_scale)
            node = int(keep[k])
            want, want_lse = mla.mla_decode(view, s.q.view(s.B, n, H, 576)[b, node][None].contiguous(), s.scale)
            parity.compare(out[b, node], lse[b, node], want[0].double().cpu().numpy(),
                           want_lse[0].double().cpu().numpy(), f"b={b} node={node}",
                           rel_l2=2 * parity.REL_L2, max_abs_row=parity.MAX_ABS)  # (two roundings)
            # and the emitted token: the accepted child's, or one the row gives weight to
            t = int(tokens[b, k])
            assert t == int(s.tokens[b, keep[k + 1]]) if k < c else float(probs[b, node, t]) > 0
    # the kept rows read back: codes times the scale
    lens = [p + c + 1 for p, c in zip(prefix, counts)]
    cu = torch.tensor([0] + torch.tensor([c + 1 for c in counts]).cumsum(0).tolist(), device=DEV)
    starts = torch.tensor(prefix, dtype=torch.int32, device=DEV)
    s.kv.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    got = mla.mla_cache_gather(s.kv, cu, int(cu[-1]), starts=starts, dtype=torch.float32)
    want = torch.cat([flat[slots[b, :c + 1]] for b, c in enumerate(counts)])
    assert torch.equal(got, want.view(torch.float8_e4m3fn).float() * s.kv.kv_scale)


def test_step_captured():
    """The whole step as one graph on a side stream, replayed twice with the same and with new
    inputs, equals the eager step."""
    s, other = Step([500, 90], 7, seed=3), Step([500, 90], 7, seed=4)
    other.kv.kv_scale = s.kv.kv_scale  # a host value: the graph keeps the one it was captured with
    want = [t.clone() for t in other.run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = s.run()
    graph.replay()
    torch.cuda.synchronize()
    for name in ("latent", "q", "q_rope", "weight", "head", "u", "mask", "parents", "positions", "slots"):
        getattr(s, name).copy_(getattr(other, name))
    s.kv.pool.copy_(other.kv.pool)
    s.kv.page_table.copy_(other.kv.page_table)
    graph.replay()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
