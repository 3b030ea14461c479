"""A serving loop over a cache with block scales, positions with three axes: prompts written and
attended to in chunks, tokens decoded, drafts verified and partly refused, everything read back. Checked
by float64 attention over the rows that the read-back gives (which its own tests pin), so that the rows
that attention sees are the ones that were written, at every step."""
import math

import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import workloads as W
from tests import parity
from tests.test_verify_tree_gpu import as_tensor

pytestmark = pytest.mark.gpu
DEV, H, SM = "cuda", 12, W.SM_SCALE


class Loop:
    """Two sequences; every call's buffers are the loop's own, so that a step can be captured."""

    def __init__(self, block, page=64, pages=12, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        B = 2
        order = torch.randperm(B * pages, generator=self.g).int().view(B, pages)
        pool = torch.randint(0, 255, (B * pages, page, 576), dtype=torch.uint8, generator=self.g)  # (stale rows)
        scales = torch.full((B * pages, page // block), float("nan"))                              # (and scales)
        self.kv = mla.KVCache(pool.to(DEV), order.to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV), 1.0,
                              scales=scales.to(DEV))
        self.weight = (1 + 0.1 * torch.randn(512, generator=self.g)).bfloat16().to(DEV)
        self.rope = mla.mla_rope_init(factor=4.0, original_positions=4096)
        self.axes = mla.mla_rope_axes_init([8, 12, 12], interleaved=True)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def inputs(self, new):
        """Projection rows, queries (their RoPE part apart) and positions of new[b] tokens a sequence."""
        n = sum(new)
        latent = (torch.randn(n, 640, generator=self.g) * torch.exp(torch.randn(n, 1, generator=self.g))).bfloat16()
        q = torch.randn(n, H, 576, generator=self.g).bfloat16()
        part = torch.randn(n, H, 192, generator=self.g).bfloat16()
        at = torch.randint(0, 2000, (3, n), generator=self.g)
        cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist())
        return [t.to(DEV) for t in (latent, q, part, at, cu)]

    def write(self, x, grow):
        latent, q, part, at, cu = x
        self.kv.seq_lens += grow
        mla.mla_cache_append_scaled(self.kv, latent[:, 64:], cu, self.rope, at, self.axes, norm_weight=self.weight,
                                    status=self.status)
        mla.mla_rope(self.rope, part[..., 128:], at, out=q[..., 512:], axes=self.axes)
        return q

    def check(self, q, out, lse, masks=None):
        """q, out, lse [B, n, ...] of the last n positions of both sequences."""
        lens = self.kv.seq_lens.tolist()
        cu = torch.tensor([0, lens[0], sum(lens)], device=DEV)
        back = mla.mla_cache_gather(self.kv, cu, sum(lens), dtype=torch.float32, status=self.status).double()
        assert int(self.status) == 0 and bool(torch.isfinite(back).all())
        n = q.shape[1]
        for b, L in enumerate(lens):
            k = back[cu[b]:cu[b + 1]]
            x = torch.einsum("jhd,kd->jhk", q[b].double(), k) * SM
            node = torch.arange(L, device=DEV) - (L - n)
            seen = node <= torch.arange(n, device=DEV)[:, None]
            if masks is not None:
                seen = torch.tensor([[m < 0 or bool(masks[j] >> m & 1) for m in node.tolist()] for j in range(n)], device=DEV)
            x = torch.where(seen[:, None], x, -math.inf)
            ref_lse = torch.logsumexp(x, -1)
            ref = torch.einsum("jhk,kd->jhd", torch.exp(x - ref_lse[..., None]), k[:, :512])
            parity.compare(out[b], lse[b], ref.cpu().numpy(), ref_lse.cpu().numpy(), f"sequence {b}",
                           max_abs_row=parity.MAX_ABS)


@pytest.mark.parametrize("block,page", [(1, 64), (16, 64), (64, 64), (32, 192)])
def test_loop(block, page):
    s = Loop(block, page, pages=12 if page == 64 else 4, seed=block)
    # prompts, in chunks of odd sizes, each sequence's attended to by itself
    for chunk in ((37, 90), (130, 5), (64, 100)):
        grow = torch.tensor(chunk, dtype=torch.int32, device=DEV)
        q = s.write(s.inputs(chunk), grow)
        one = []
        for b in range(2):
            view = mla.KVCache(s.kv.pool, s.kv.page_table[b:b + 1], s.kv.seq_lens[b:b + 1], 1.0, scales=s.kv.scales)
            lo = sum(chunk[:b])
            one.append(mla.mla_prefill(view, q[lo:lo + chunk[b]].contiguous(), SM))
        n = min(chunk)
        qs = torch.stack([q[:chunk[0]][-n:], q[chunk[0]:][-n:]])
        s.check(qs, torch.stack([o[0][-n:] for o in one]), torch.stack([o[1][-n:] for o in one]))
    # tokens one by one, then four drafts of which sequence 0 keeps one and sequence 1 three
    for _ in range(5):
        q = s.write(s.inputs((1, 1)), 1)
        out, lse = mla.mla_decode(s.kv, q, SM)
        s.check(q[:, None], out[:, None], lse[:, None])
    q = s.write(s.inputs((4, 4)), 4).view(2, 4, H, 576)
    s.check(q, *mla.mla_verify(s.kv, q, SM))
    chain = mla.mla_verify_tree(s.kv, q, as_tensor([[1, 3, 7, 15]] * 2).to(DEV), SM)
    s.check(q, *chain)
    branches = [1, 3, 5, 11]  # nodes 1 and 2 below 0, 3 below 1
    s.check(q, *mla.mla_verify_tree(s.kv, q, as_tensor([branches] * 2).to(DEV), SM), masks=branches)
    s.kv.seq_lens -= torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    q = s.write(s.inputs((1, 1)), 1)  # over the refused rows; their blocks' scales stay
    out, lse = mla.mla_decode(s.kv, q, SM)
    s.check(q[:, None], out[:, None], lse[:, None])


def test_step_captured():
    """A decode step (write, rotation, decode, read-back) as one graph on a side stream, replayed over
    new inputs and growing sequences, equals the eager steps."""
    a, b = Loop(16, seed=1), Loop(16, seed=1)
    first = a.inputs((40, 7)), b.inputs((40, 7))
    for s, x in zip((a, b), first):
        s.write(x, torch.tensor([40, 7], dtype=torch.int32, device=DEV))
    ws = mla.workspace(mla.MLA_OP_DECODE, 2, H, 1)
    starts, cu = torch.zeros(2, dtype=torch.int32, device=DEV), torch.tensor([0, 30, 35], device=DEV)

    def step(s, x):
        q = s.write(x, 1)
        out, lse = mla.mla_decode(s.kv, q, SM, ws=ws)
        return out, lse, mla.mla_cache_gather(s.kv, cu, 35, starts=starts), s.kv.scales, s.kv.pool

    xs = [a.inputs((1, 1)) for _ in range(20)]
    static = [t.clone() for t in xs[0]]
    want = [[t.clone() for t in step(a, [t.clone() for t in x])] for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            got = step(b, static)
    torch.cuda.synchronize()
    for x, w in zip(xs, want):
        for t, u in zip(static, x):
            t.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        for t, u in zip(got, w):
            assert torch.equal(t.view(torch.uint8), u.view(torch.uint8))
    assert int(a.status) == int(b.status) == 0


def test_two_streams_at_once():
    """Two loops' calls on two streams, each with its own cache and workspace, at the same time: each gives
    what it gives alone."""
    def calls(seed, stream=None):
        s = Loop(8, seed=seed)
        ws = mla.workspace(mla.MLA_OP_VERIFY, 2, H, 3)
        xs = [s.inputs((200, 150))] + [s.inputs((3, 3)) for _ in range(15)]
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            out = []
            for i, x in enumerate(xs):
                q = s.write(x, torch.tensor([200, 150], dtype=torch.int32).to(DEV) if i == 0 else 3)
                if i:
                    out += mla.mla_verify_f32(s.kv, q.view(2, 3, H, 576), SM, ws=ws)
        return out + [s.kv.pool, s.kv.scales]

    alone = [calls(seed) for seed in (1, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = [calls(seed, st) for seed, st in zip((1, 2), streams)]
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        for t, u in zip(x, y):
            assert torch.equal(t.contiguous().view(torch.uint8), u.contiguous().view(torch.uint8))


@pytest.mark.parametrize("H,n_q", [(12, 1), (8, 2), (12, 4)])
def test_calls_queued_on_one_workspace(H, n_q):
    """As many equal sequences as SMs, calls one behind the other on one workspace (programmatic
    dependents of each other): each equal to the call alone."""
    B = torch.cuda.get_device_properties(0).multi_processor_count
    inp = W.make_inputs("even", [640] * B, H=H, n_q=n_q, seed=H)
    g = torch.Generator().manual_seed(n_q)
    scales = torch.exp2(torch.randint(-9, -4, (inp.pool.shape[0], 4), generator=g).float()).to(DEV)
    kv = mla.KVCache(inp.pool.to(DEV), inp.page_table.to(DEV), inp.seq_lens.to(DEV), 1.0, scales=scales)
    qs = [torch.randn(inp.q.shape, generator=g).bfloat16().to(DEV) for _ in range(10)]
    ws = mla.workspace(mla.MLA_OP_VERIFY, B, H, n_q)
    alone = []
    for q in qs:
        alone.append(mla.mla_verify(kv, q, SM, ws=ws))
        torch.cuda.synchronize()
        assert mla.mla_read_status(ws) == 0
    for _ in range(3):
        got = [mla.mla_verify(kv, q, SM, ws=ws) for q in qs]
        torch.cuda.synchronize()
        for x, y in zip(alone, got):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def scaled_calls():
    g = torch.Generator().manual_seed(1)
    inp = W.make_inputs("streams", [400, 90], H=H, n_q=2, seed=1)
    scales = torch.exp2(torch.randint(-9, -4, (inp.pool.shape[0], 4), generator=g).float()).to(DEV)
    kv = mla.KVCache(inp.pool.to(DEV), inp.page_table.to(DEV), inp.seq_lens.to(DEV), 1.0, scales=scales)
    one = mla.KVCache(kv.pool, kv.page_table[:1], kv.seq_lens[:1], 1.0, scales=scales)
    q, mask = inp.q.to(DEV), torch.tensor([[1, 3]] * 2, device=DEV)
    first = q[:, 0].contiguous()
    rope, axes = mla.mla_rope_init(), mla.mla_rope_axes_init([12, 10, 10])
    x = torch.randn(300, H, 64, generator=g).bfloat16().to(DEV)
    at = torch.randint(0, 900, (3, 300), generator=g).to(DEV)
    rows, cu = torch.randn(60, 576, generator=g).bfloat16().to(DEV), torch.tensor([0, 40, 60], device=DEV)
    m = W.mha_prefill_inputs(50, 350, H=2, seed=3)
    mq, mw = m.q.to(DEV), m.w_ukv.to(DEV)
    long = torch.tensor([0, 300, 380], device=DEV)

    def append(**k):
        pool, s = kv.pool.clone(), scales.clone()
        torch.cuda.synchronize()
        mla.mla_cache_append_scaled(mla.KVCache(pool, kv.page_table, kv.seq_lens, 1.0, scales=s), rows, cu, rope,
                                    at[:, :60].contiguous(), axes, **k)
        return pool, s

    return {
        "rope": lambda **k: (mla.mla_rope(rope, x, at, axes=axes, **k),),
        "append": append,
        "gather": lambda **k: (mla.mla_cache_gather(kv, long, 380, **k),),
        "decode": lambda **k: mla.mla_decode(kv, first, SM, **k),
        "verify": lambda **k: mla.mla_verify(kv, q, SM, **k),
        "verify_f32": lambda **k: mla.mla_verify_f32(kv, q, SM, visible_shift=1, **k),
        "tree": lambda **k: mla.mla_verify_tree(kv, q, mask, SM, **k),
        "prefill": lambda **k: mla.mla_prefill(one, first, SM, **k),
        "mha": lambda **k: mla.mla_prefill_mha(one, mq, mw, SM, L=400, **k),
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["rope", "append", "gather", "decode", "verify", "verify_f32", "tree", "prefill", "mha"])
def test_results_belong_to_the_stream(name, raw):
    """A call given a stream runs and allocates there: the caller's own stream still has writes to make
    into memory that it has freed."""
    call = scaled_calls()[name]
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = [torch.empty_like(t) for t in want] + [torch.empty(40 << 20, dtype=torch.uint8, device=DEV)]
    if name != "append":
        torch.cuda._sleep(40_000_000)  # (cycles: about 20 ms before the writes below)
    for t in late:
        t.fill_(1)
    del late, t
    got = call(stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
