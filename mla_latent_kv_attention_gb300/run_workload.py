"""Run one named seeded workload through the C ABI a few times (for profilers).

    python -m mla_latent_kv_attention_gb300.run_workload batched_paged_decode --iters 5
    python -m mla_latent_kv_attention_gb300.run_workload causal_prefill --T 2048 --iters 3
    python -m mla_latent_kv_attention_gb300.run_workload cache_append --iters 5
    python -m mla_latent_kv_attention_gb300.run_workload top_k_renorm --iters 5
    python -m mla_latent_kv_attention_gb300.run_workload speculative_step --iters 5
    python -m mla_latent_kv_attention_gb300.run_workload block_scaled_step --iters 5

Prints the device status word after the last call. Intended as the command line that
ncu wraps: every launch it makes is a library launch on the named inputs.
"""
from __future__ import annotations

import argparse
import sys

import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import workloads as W


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("workload", choices=sorted(W.WORKLOADS) + ["cache_append", "top_k_renorm",
                                                                 "mha_prefill", "speculative_step", "block_scaled_step"])
    ap.add_argument("--iters", type=int, default=5)
    ap.add_argument("--heads", type=int, default=12, help="long_history_decode only")
    ap.add_argument("--T", type=int, default=8192, help="causal_prefill and mha_prefill only")
    ap.add_argument("--bf16", action="store_true", help="mha_prefill only: the all-bf16 form")
    ap.add_argument("--block", type=int, default=0, choices=[0, 1, 2, 4, 8, 16, 32, 64],
                    help="mha_prefill only: a scale for every so many positions (0: one scale)")
    args = ap.parse_args(argv)
    if args.workload == "cache_append":
        return _cache_append(args.iters)
    if args.workload == "mha_prefill":
        return _mha_prefill(args.T, args.iters, args.bf16, args.block)
    if args.workload == "speculative_step":
        return _speculative_step(args.iters)
    if args.workload == "block_scaled_step":
        return _block_scaled_step(args.iters)
    if args.workload == "top_k_renorm":
        return _top_k_renorm(args.iters)
    if args.workload == "long_history_decode":
        inp = W.long_history_decode(args.heads)
    elif args.workload == "causal_prefill":
        inp = W.causal_prefill(T=args.T)
    else:
        inp = W.WORKLOADS[args.workload]()
    kv = mla.KVCache.from_inputs(inp, "cuda")
    if args.workload == "causal_prefill":
        q = inp.q[0].contiguous().cuda()
        ws = mla.workspace(mla.MLA_OP_PREFILL, 1, inp.H, inp.n_q)
        for _ in range(args.iters):
            mla.mla_prefill(kv, q, inp.sm_scale, ws=ws)
    else:
        q = inp.q.contiguous().cuda()
        ws = mla.workspace(mla.MLA_OP_VERIFY, inp.B, inp.H, inp.n_q)
        for _ in range(args.iters):
            if inp.n_q == 1:
                mla.mla_decode(kv, q[:, 0].contiguous(), inp.sm_scale, ws=ws)
            else:
                mla.mla_verify(kv, q, inp.sm_scale, ws=ws)
    torch.cuda.synchronize()
    status = mla.mla_read_status(ws)
    print(f"{args.workload}: {args.iters} calls, status {mla.STATUS.get(status, status)}")
    return 0 if status == 0 else 1


def _cache_append(iters: int) -> int:
    """8,192 bf16 rows (a prefill chunk) into a 302 MB pool of 64-position pages at random
    slots, a different slot set each call."""
    g = torch.Generator().manual_seed(7)
    pool = torch.zeros(8192, 64, mla.MLA_D, dtype=torch.uint8, device="cuda")
    x = torch.randn(8192, mla.MLA_D, generator=g).to(torch.bfloat16).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for i in range(iters):
        slots = torch.randperm(pool.shape[0] * 64, generator=g)[:8192].cuda()
        mla.mla_cache_append(pool, x, slots, 0.0125, status=status)
    torch.cuda.synchronize()
    st = int(status.item())
    print(f"cache_append: {iters} calls, status {mla.STATUS.get(st, st)}")
    return 0 if st == 0 else 1


def _mha_prefill(T: int, iters: int, bf16: bool = False, block: int = 0) -> int:
    """The causal prefill chunk (T new positions on a 32,768 prefix, 12 heads) in the MHA form
    (the default form, or the all-bf16 one), under one scale or one for every `block` positions."""
    m = W.mha_prefill(T=T)
    kv = mla.KVCache.from_inputs(m.cache, "cuda")
    if block:
        pages, size, _ = kv.pool.shape
        g = torch.Generator(device="cuda").manual_seed(1)
        kv.scales = torch.exp2(torch.randint(-8, -5, (pages, size // block), generator=g, device="cuda").float())
        kv.kv_scale = 1.0
    q = m.q.cuda()
    w = m.w_ukv.cuda()
    L = int(m.cache.seq_lens[0])
    ws = torch.zeros(mla.library().mla_prefill_mha_workspace_size(L, m.H, 0), dtype=torch.uint8,
                     device="cuda")
    for _ in range(iters):
        mla.mla_prefill_mha(kv, q, w, m.cache.sm_scale, L=L, ws=ws, bf16=bf16)
    torch.cuda.synchronize()
    status = mla.mla_read_status(ws)
    print(f"mha_prefill: {iters} calls, status {mla.STATUS.get(status, status)}")
    return 0 if status == 0 else 1


def _speculative_step(iters: int) -> int:
    """Eight sequences on a 32,768-position prefix, 16 drafted nodes each (a binary tree): draft
    rows written (norm, rotation, quantisation), queries rotated, the tree verified, drafts
    accepted against synthetic target probabilities (129,280 entries a row), the last 512
    positions of every sequence read back."""
    B, n, H, V = 8, 16, 12, 129280
    inp = W.make_inputs("speculative_step", [32768 + n] * B, H=H, n_q=n, seed=0)
    kv = mla.KVCache.from_inputs(inp, "cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    parents = [-1] + [(j - 1) // 2 for j in range(1, n)]
    masks, depth = [], []
    for j, a in enumerate(parents):
        masks.append((masks[a] if a >= 0 else 0) | 1 << j)
        depth.append(depth[a] + 1 if a >= 0 else 0)
    tree_mask = torch.tensor([masks] * B, device="cuda")
    place = 32768 + torch.arange(n, device="cuda").expand(B, n)
    positions = (32768 + torch.tensor(depth, device="cuda").expand(B, n)).flatten()
    slots = (kv.page_table.gather(1, place // 64).long() * 64 + place % 64).flatten()
    latent = torch.randn(B * n, mla.MLA_D, generator=g, device="cuda").bfloat16()
    weight = torch.ones(mla.MLA_DV, dtype=torch.bfloat16, device="cuda")
    q = inp.q.cuda()
    q_rope = torch.randn(B * n, H, mla.MLA_ROPE, generator=g, device="cuda").bfloat16()
    probs = torch.softmax(5 * torch.randn(B, n, V, generator=g, device="cuda"), -1)
    tokens = torch.randint(0, V, (B, n), generator=g, device="cuda", dtype=torch.int32)
    uniforms = torch.rand(B, n + 1, generator=g, device="cuda")
    parents = torch.tensor([parents] * B, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, device="cuda") * 512
    starts = torch.full((B,), 32768 + n - 512, dtype=torch.int32, device="cuda")
    rope = mla.mla_rope_init(factor=40.0, original_positions=4096)
    ws = mla.workspace(mla.MLA_OP_VERIFY_TREE, B, H, n)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(iters):
        mla.mla_cache_append_rope(kv.pool, latent, slots, kv.kv_scale, rope, positions,
                                  norm_weight=weight, status=word)
        mla.mla_rope(rope, q_rope, positions, out=q.view(B * n, H, mla.MLA_D)[..., mla.MLA_DV:])
        mla.mla_verify_tree(kv, q, tree_mask, inp.sm_scale, ws=ws)
        mla.mla_accept_drafts(probs, tokens, uniforms, parents=parents)
        mla.mla_cache_gather(kv, cu, B * 512, starts=starts, status=word)
    torch.cuda.synchronize()
    status = mla.mla_read_status(ws) or int(word.item())
    print(f"speculative_step: {iters} calls, status {mla.STATUS.get(status, status)}")
    return 0 if status == 0 else 1


def _block_scaled_step(iters: int) -> int:
    """Steps over a cache with a scale for every 16 positions, positions with three axes: eight
    sequences on a 32,768-position prefix write four new rows each (norm, rotation, scales), their
    queries are rotated and verified, the last 512 positions are read back; a 2,048-position chunk of
    a ninth sequence is written and prefilled."""
    B, n, T, H, block = 8, 4, 2048, 12, 16
    inp = W.make_inputs("block_scaled_step", [32768 + n] * B + [32768 + T], H=H, n_q=1, seed=0)
    g = torch.Generator(device="cuda").manual_seed(1)
    scales = torch.exp2(torch.randint(-8, -5, (inp.pool.shape[0], 64 // block), generator=g, device="cuda").float())
    kv = mla.KVCache(inp.pool.cuda(), inp.page_table.cuda(), inp.seq_lens.cuda(), 1.0, scales=scales)
    some = mla.KVCache(kv.pool, kv.page_table[:B], kv.seq_lens[:B], 1.0, scales=scales)
    last = mla.KVCache(kv.pool, kv.page_table[B:], kv.seq_lens[B:], 1.0, scales=scales)
    rope, axes = mla.mla_rope_init(factor=40.0, original_positions=4096), mla.mla_rope_axes_init([8, 12, 12])
    weight = torch.ones(mla.MLA_DV, dtype=torch.bfloat16, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")

    def tokens(rows):
        return (torch.randn(rows, mla.MLA_D, generator=g, device="cuda").bfloat16(),
                torch.randn(rows, H, mla.MLA_D, generator=g, device="cuda").bfloat16(),
                torch.randint(0, 32768, (3, rows), generator=g, device="cuda"))

    x, q, at = tokens(B * n)
    px, pq, pat = tokens(T)
    cu, pcu = torch.arange(B + 1, device="cuda") * n, torch.tensor([0, T], device="cuda")
    back = torch.arange(B + 1, device="cuda") * 512
    starts = torch.full((B,), 32768 + n - 512, dtype=torch.int32, device="cuda")
    ws = mla.workspace(mla.MLA_OP_VERIFY, B, H, n)
    pws = mla.workspace(mla.MLA_OP_PREFILL, 1, H, T)
    for _ in range(iters):
        mla.mla_cache_append_scaled(some, x, cu, rope, at, axes, norm_weight=weight, status=word)
        part = q[..., mla.MLA_DV:]
        mla.mla_rope(rope, part, at, out=part, axes=axes)
        mla.mla_verify(some, q.view(B, n, H, mla.MLA_D), inp.sm_scale, ws=ws)
        mla.mla_cache_gather(some, back, B * 512, starts=starts, status=word)
        mla.mla_cache_append_scaled(last, px, pcu, rope, pat, axes, norm_weight=weight, status=word)
        mla.mla_prefill(last, pq, inp.sm_scale, ws=pws)
    torch.cuda.synchronize()
    status = mla.mla_read_status(ws) or mla.mla_read_status(pws) or int(word.item())
    print(f"block_scaled_step: {iters} calls, status {mla.STATUS.get(status, status)}")
    return 0 if status == 0 else 1


def _top_k_renorm(iters: int) -> int:
    """32 probability rows over a 129,280-entry vocabulary, k drawn per row in [1, 1024)."""
    g = torch.Generator().manual_seed(1)
    probs = torch.softmax(torch.randn(32, 129280, generator=g) * 3, dim=1).cuda()
    ks = torch.randint(1, 1024, (32,), generator=g, dtype=torch.int32).cuda()
    out = torch.empty_like(probs)
    for _ in range(iters):
        mla.mla_top_k_renorm_prob(probs, ks, out=out)
    torch.cuda.synchronize()
    ok = bool(torch.isfinite(out).all().item())
    print(f"top_k_renorm: {iters} calls, {'finite' if ok else 'NON-FINITE'} output")
    return 0 if ok else 1


if __name__ == "__main__":
    sys.exit(main())
