"""mla_cache_append_scaled and mla_cache_gather from a cache with block scales, against the definitions.

Scales. The kernel's float32 values are within 2^-20 of the exact ones (latent) or 2^-19 (|a| + |b|)
(RoPE part; see test_cache_rope_gather_gpu.py), so its largest entry lies between the largest lower
and the largest upper bound of the block, and the scale is the power of two for some number between
them (one and the same for both in all but the rarest block). Codes: half a step of e4m3 besides, the
division by a power of two being exact. Codes of earlier positions: exact."""
import math
import random

import numpy as np
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from tests.test_cache_rope_gather_gpu import decode, expected
from tests.test_rope_axes_gpu import rotate
from tests.test_rope_gpu import frequencies

pytestmark = pytest.mark.gpu
DEV = "cuda"


def cache(lens, block, g, page_size=64, spare=2, empty=False):
    """Random codes under random power-of-two scales on randomly ordered pages."""
    pages = [-(-n // page_size) for n in lens]
    order = torch.randperm(sum(pages) + spare, generator=g).int()
    table = torch.full((len(lens), max(pages + [1])), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = order[at:at + k]
        at += k
    pool = torch.randint(0, 256, (sum(pages) + spare, page_size, 576), dtype=torch.uint8, generator=g)
    pool[(pool & 0x7F) == 0x7F] = 0  # no NaN codes
    scales = torch.exp2(torch.randint(-9, -4, (sum(pages) + spare, page_size // block), generator=g).float())
    return mla.KVCache(pool.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), 1.0,
                       scales=scales.to(DEV))


def power_for(top):
    """The exponent of the smallest power of two that brings `top` to 448 or less."""
    k = -60
    while k < 60 and top > 448.0 * 2.0 ** k:
        k += 1
    return k


def check_append(kv, before, scales_before, lens, new, y, slack, page_size):
    """kv after the rows y (float64, with float32 errors up to slack) were appended, against the pool and
    the scales before."""
    block = page_size // kv.scales.shape[1]
    flat, scale = decode(kv.pool).reshape(-1, 576), kv.scales.cpu().view(-1).double().numpy()
    raw, raw_before = kv.pool.cpu().view(-1, 576), before.view(-1, 576)
    was = scales_before.view(-1)
    touched_rows, touched_blocks = torch.zeros(len(raw), dtype=torch.bool), set()
    row = 0
    for b, (m, L) in enumerate(zip(new, lens)):
        for k in range((L - m) // block, (L - 1) // block + 1 if m else 0):
            lo, hi = max(L - m, k * block), min(L, (k + 1) * block)
            at = int(kv.page_table[b, k * block // page_size]) * page_size + k * block % page_size
            r = slice(row + lo - (L - m), row + hi - (L - m))
            old = lo - k * block
            s_old = float(was[at // block])
            fits = [2.0 ** power_for(t) for t in (max(0.0, (np.abs(y[r]) - slack[r]).max()), (np.abs(y[r]) + slack[r]).max())]
            if old:
                fits = [max(s_old, t) for t in fits]
            s = scale[at // block]
            assert s in fits, (b, k, s, fits)
            assert fits[0] == fits[1] or fits[1] == 2 * fits[0]
            touched_blocks.add(at // block)
            touched_rows[at:at + hi - k * block] = True
            if old:  # the codes that were there, moved exactly
                want = (raw_before[at:at + old].view(torch.float8_e4m3fn).float() * np.float32(s_old / s))
                want = want.to(torch.float8_e4m3fn).view(torch.uint8)
                got = raw[at:at + old]
                assert torch.equal(got, want)
            v, dv = y[r] / s, slack[r] / s
            v = np.clip(v, -448, 448)
            e = np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 1e-30))), -6)
            assert np.all(np.abs(flat[at + old:at + hi - k * block] - v) <= 2.0 ** (e - 4) + dv)
        row += m
    assert torch.equal(raw[~touched_rows], raw_before[~touched_rows])
    rest = torch.tensor([i not in touched_blocks for i in range(len(scale))])
    assert torch.equal(kv.scales.cpu().view(-1)[rest], was[rest])


CASES = [  # new rows, earlier positions, block, page size
    ([1], [0], 16, 64), ([1], [0], 1, 64), ([1] * 33, list(range(33)), 16, 64), ([1] * 40, list(range(100, 140)), 64, 64),
    ([4, 0, 3, 1, 0], [30, 50, 63, 64, 0], 8, 64), ([200, 1, 77], [0, 63, 190], 32, 128), ([5, 6, 7, 8], [1, 2, 3, 4], 2, 192),
    ([3, 300], [125, 3], 4, 64), ([64, 128, 65], [64, 0, 63], 64, 64), ([1000], [37], 64, 128), ([1000], [1], 1, 64),
    ([9000], [3], 16, 64), ([1] * 1100, [i % 70 for i in range(1100)], 16, 64), ([0, 0, 2], [5, 0, 0], 16, 64)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(case, interleaved):
    new, earlier, block, page_size = CASES[case]
    g = torch.Generator().manual_seed(case)
    lens = [m + e for m, e in zip(new, earlier)]
    kv = cache(lens, block, g, page_size)
    before, scales_before = kv.pool.cpu().clone(), kv.scales.cpu().clone()
    n, stride = sum(new), [576, 640, 2112][case % 3]
    x = (torch.randn(n + 3, stride, generator=g) * torch.exp(2 * torch.randn(n + 3, 1, generator=g))).bfloat16()
    x = x.to(DEV)[:, stride - 576:]
    positions = torch.randint(-100, 150000, (n + 3,), generator=g)
    weight = torch.randn(512, generator=g).bfloat16().to(DEV)
    rope = mla.mla_rope_init(factor=40.0, original_positions=4096, interleaved=interleaved)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = torch.tensor(np.cumsum([0] + new), device=DEV)
    mla.mla_cache_append_scaled(kv, x, cu, rope, positions.to(DEV), norm_weight=weight, eps=1e-5, status=status)
    assert int(status) == 0
    y, slack = expected(x[:n], 1.0, weight, 1e-5, frequencies(10000.0, 40.0, 4096), positions[:n], interleaved)
    check_append(kv, before, scales_before, lens, new, y, slack, page_size)


@pytest.mark.parametrize("block", [1, 2, 4, 8, 16, 32, 64])
def test_axes_and_rows_before_the_first_sequence(block):
    g = torch.Generator().manual_seed(block)
    new, earlier = [1, 70, 0, 9], [40, 11, 8, 100]
    lens = [m + e for m, e in zip(new, earlier)]
    kv = cache(lens, block, g)
    before, scales_before = kv.pool.cpu().clone(), kv.scales.cpu().clone()
    n = sum(new)
    x = torch.randn(n + 5, 576, generator=g).bfloat16().to(DEV)
    positions = torch.randint(0, 5000, (3, n + 5), generator=g)
    axes, rope = mla.mla_rope_axes_init([8, 12, 12]), mla.mla_rope_init()
    cu = torch.tensor(np.cumsum([2] + new), device=DEV)  # two rows ahead, three behind
    mla.mla_cache_append_scaled(kv, x, cu, rope, positions.to(DEV), axes=axes)
    y = x[2:2 + n].double().cpu().numpy()
    turned, size = rotate(y[:, None, 512:], positions[:, 2:2 + n].tolist(), list(axes.axis), frequencies(10000.0, 1.0, 0),
                          1.0, True)
    slack = np.zeros_like(y)
    y[:, 512:], slack[:, 512:] = turned[:, 0], 2.0 ** -19 * size[:, 0]
    check_append(kv, before, scales_before, lens, new, y, slack, 64)


def test_one_row_a_step_as_if_written_once():
    """A sequence written a row, or a few, a step ends with the scales and (subnormals of the codes
    aside) the codes of one written at once: scales only grow, by powers of two."""
    g = torch.Generator().manual_seed(5)
    L = 150
    x = (torch.randn(L, 576, generator=g) * torch.exp(torch.randn(L, 1, generator=g))).bfloat16().to(DEV)
    for block in (1, 16, 64):
        once, steps = cache([L], block, g), cache([L], block, g)
        steps.page_table.copy_(once.page_table)
        mla.mla_cache_append_scaled(once, x, torch.tensor([0, L], device=DEV))
        done = 0
        r = random.Random(block)
        while done < L:
            m = min(L - done, r.choice([1, 1, 1, 4, 30]))
            steps.seq_lens.fill_(done + m)
            mla.mla_cache_append_scaled(steps, x[done:done + m], torch.tensor([0, m], device=DEV))
            done += m
        at = once.page_table[0].long()
        assert torch.equal(once.scales[at].view(-1)[:-(-L // block)], steps.scales[at].view(-1)[:-(-L // block)])
        a, b = (c.pool[at].view(-1, 576)[:L].view(torch.float8_e4m3fn).float() for c in (once, steps))
        normal = a.abs() >= 2.0 ** -6
        assert torch.equal(a[normal], b[normal])
        # a subnormal was rounded at most once a growth, each time by half a step or less
        assert float((a - b).abs().max()) <= 2.0 ** -9


def test_special_values():
    """Infinities saturate and do not set the scale, NaN stays with its entry, zeros get the smallest
    scale, huge and tiny blocks the clamped ones."""
    g = torch.Generator().manual_seed(6)
    kv = cache([16 * 6], 16, g)
    x = torch.randn(96, 576, generator=g).bfloat16()
    x[3, 7], x[4, 520], x[5, 100] = float("inf"), -float("inf"), float("nan")
    x[16:32] = 0
    x[32:48] = 1e30
    x[48:64] = 1e-30
    x[64:80] = float("nan")
    x[80:96] = -float("inf")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.mla_cache_append_scaled(kv, x.to(DEV), torch.tensor([0, 96], device=DEV), status=status)
    at = kv.page_table[0].long()
    s = kv.scales[at].view(-1)[:6].tolist()
    codes = kv.pool[at].view(-1, 576)[:96].cpu()
    v = codes.view(torch.float8_e4m3fn).float()
    top = x[:16].float()
    assert s[0] == 2.0 ** power_for(float(top[torch.isfinite(top)].abs().max()))
    assert s[1:] == [2.0 ** -60, 2.0 ** 60, 2.0 ** -60, 2.0 ** -60, 2.0 ** -60]
    assert v[3, 7] == 448 and v[4, 520] == -448 and torch.isnan(v[5, 100])
    assert int(torch.isnan(v[:16]).sum()) == 1 and torch.all(codes[16:32] == 0)
    assert torch.all(v[32:48] == 448) and torch.all(v[48:64] == 0)  # 1e-30 is below half the smallest step
    assert torch.all(torch.isnan(v[64:80])) and torch.all(v[80:] == -448)
    assert int(status) == 0


@pytest.mark.parametrize("old", [float("nan"), 0.0, -1.0, float("inf"), 2.0 ** -61, 2.0 ** 61])
def test_earlier_positions_without_a_scale_become_nan(old):
    g = torch.Generator().manual_seed(7)
    kv = cache([20], 16, g)
    kv.scales.fill_(old)
    x = torch.randn(1, 576, generator=g).bfloat16().to(DEV)
    mla.mla_cache_append_scaled(kv, x, torch.tensor([0, 1], device=DEV))
    page = int(kv.page_table[0, 0])
    v = kv.pool[page].view(torch.float8_e4m3fn).float()
    assert torch.all(torch.isnan(v[16:19])) and torch.all(torch.isfinite(v[19]))
    assert float(kv.scales[page, 1]) == 2.0 ** power_for(float(x.float().abs().max()))


def test_other_scales_than_powers_of_two():
    """A block under any other scale keeps it while it is large enough, and moves to a power of two after."""
    g = torch.Generator().manual_seed(8)
    for old, grows in ((0.3, False), (0.003, True)):
        kv = cache([20], 32, g)
        kv.scales.fill_(old)
        before = kv.pool.clone()
        x = (8 * torch.randn(1, 576, generator=g)).clamp(-20, 20).bfloat16()
        x[0, 0] = 17.0
        mla.mla_cache_append_scaled(kv, x.to(DEV), torch.tensor([0, 1], device=DEV))
        page = int(kv.page_table[0, 0])
        s = kv.scales[page, 0]
        assert float(s) == (2.0 ** power_for(float(x.float().abs().max())) if grows else np.float32(old))
        was = before[page, :19].view(torch.float8_e4m3fn).float()
        now = kv.pool[page, :19].view(torch.float8_e4m3fn).float()
        step = torch.exp2(torch.floor(torch.log2((was * (old / float(s))).abs().clamp(min=2.0 ** -6))) - 3)
        assert torch.all((now - was * (old / float(s))).abs() <= step / 2 * (1 + 2.0 ** -10))
        if not grows:
            assert torch.equal(before[page, :19], kv.pool[page, :19])


def test_bounds():
    """Sequences too short for their rows, longer than their table, with rows outside x, and pages outside
    the pool: reported, not written; the others are."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(12, 576, generator=g).bfloat16().to(DEV)

    def run(change, cu, n=12, refused=()):
        kv = cache([64 + 3, 70, 40], 16, g)
        change(kv)
        pool, scales = kv.pool.clone(), kv.scales.clone()
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        mla.mla_cache_append_scaled(kv, x[:n], torch.tensor(cu, device=DEV), status=status)
        assert int(status) == mla.MLA_ERR_BOUNDS
        same = (kv.pool == pool).all(-1)
        for b in range(3):
            L = [67, 70, 40][b]
            m = cu[b + 1] - cu[b]
            pos = torch.arange(L - m, L)
            changed = ~same.cpu()[kv.page_table[b].cpu()[pos // 64].long().clamp(0, len(pool) - 1), pos % 64]
            assert bool(changed.all()) != (b in refused), b
        assert int((~same).sum()) <= 12 + 3 * 15

    def set_len(b, v):
        return lambda kv: kv.seq_lens.__setitem__(b, v)

    run(set_len(1, 3), [0, 4, 8, 12], refused=(1,))
    run(set_len(2, 129), [0, 4, 8, 12], refused=(2,))
    run(set_len(0, -5), [0, 4, 8, 12], refused=(0,))
    run(lambda kv: None, [0, 4, 8, 12], n=10, refused=(2,))
    run(lambda kv: None, [0, 4, 8, 12], n=8, refused=(2,))
    run(lambda kv: kv.page_table.__setitem__((1, 1), len(kv.pool)), [0, 4, 8, 12], refused=(1,))
    run(lambda kv: kv.page_table.__setitem__((0, 1), -1), [0, 3, 8, 12], refused=(0,))


@pytest.mark.parametrize("block", [1, 2, 16])
def test_decreasing_rows(block):
    """cu_rows that decreases (units 0 to 6 of blocks of one are led to the first sequence, whose own begin at 7) is
    reported, and nothing but the sequences' last positions is written."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn(20, 576, generator=g).bfloat16().to(DEV)
    kv = cache([2, 40, 20], block, g)
    pool = kv.pool.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.mla_cache_append_scaled(kv, x, torch.tensor([7, 9, 0, 20], device=DEV), status=status)
    assert int(status) == mla.MLA_ERR_BOUNDS
    changed = ~(kv.pool == pool).all(-1)
    pages = kv.page_table[:, 0].tolist()
    allowed = torch.zeros_like(changed)
    allowed[pages[0], :2] = True
    allowed[pages[2], :20] = True
    assert not bool((changed & ~allowed).any())


def test_refusals():
    g = torch.Generator().manual_seed(10)
    kv = cache([64], 16, g)
    x = torch.zeros(4, 576, dtype=torch.bfloat16, device=DEV)
    cu, rope = torch.tensor([0, 4], device=DEV), mla.mla_rope_init()
    plain = mla.KVCache(kv.pool, kv.page_table, kv.seq_lens, 1.0)
    at = torch.zeros(4, dtype=torch.int64, device=DEV)
    for kw in (dict(kv=plain), dict(x=x.float()), dict(x=x[:, :512]), dict(x=x.cpu()), dict(cu_rows=cu.int()),
               dict(cu_rows=cu[:0]), dict(cu_rows=torch.zeros(3, dtype=torch.int64, device=DEV)), dict(cu_rows=cu[None]),
               dict(rope=rope), dict(positions=at), dict(rope=rope, positions=at[:3]),
               dict(rope=rope, positions=at, axes=mla.mla_rope_axes_init([32])), dict(axes=mla.mla_rope_axes_init([32])),
               dict(norm_weight=torch.ones(512, device=DEV)), dict(status=torch.zeros(1, device=DEV))):
        with pytest.raises(ValueError):
            mla.mla_cache_append_scaled(**dict(dict(kv=kv, x=x, cu_rows=cu), **kw))
    before = kv.pool.clone()
    mla.mla_cache_append_scaled(kv, x[:0], torch.tensor([0, 0], device=DEV))
    mla.mla_cache_append_scaled(kv, x, cu[:1])
    assert torch.equal(kv.pool, before)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,starts,block,page_size", [
    ([1], None, 16, 64), ([64, 65, 63], None, 64, 64), ([100, 0, 7, 300], [99, 0, 0, 5], 1, 64),
    ([5000, 1, 129], [0, 1, 100], 32, 128), ([33] * 70, None, 2, 192)])
def test_gather(lens, starts, block, page_size, dtype):
    g = torch.Generator().manual_seed(len(lens))
    kv = cache(lens, block, g, page_size)
    kv.scales *= 1.37  # any scale will do
    lo = starts or [0] * len(lens)
    cu = np.cumsum([0] + [n - a for n, a in zip(lens, lo)])
    n = int(cu[-1]) + 3
    out = torch.full((n, 576), 5.0, dtype=dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = mla.mla_cache_gather(kv, torch.tensor(cu, device=DEV), n, out=out, status=status,
                               starts=None if starts is None else torch.tensor(lo, dtype=torch.int32, device=DEV))
    assert got is out and int(status) == 0
    v = kv.pool.view(torch.float8_e4m3fn).float().view(-1, page_size // block, block, 576)
    v = (v * kv.scales[:, :, None, None]).view(-1, page_size, 576)  # one product, one rounding
    want = []
    for b, (m, a) in enumerate(zip(lens, lo)):
        pos = torch.arange(a, m, device=DEV)
        want.append(v[kv.page_table[b][pos // page_size].long(), pos % page_size])
    assert torch.equal(out[:-3], torch.cat(want).to(dtype))
    assert torch.all(out[-3:] == 5.0)


def test_written_rows_read_back():
    """The pair: what is written comes back within half an e4m3 step of its block's scale."""
    g = torch.Generator().manual_seed(11)
    kv = cache([130, 40], 32, g)
    x = torch.randn(170, 576, generator=g).bfloat16().to(DEV)
    weight = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    positions = torch.cat([torch.arange(130), torch.arange(40)])
    cu = torch.tensor([0, 130, 170], device=DEV)
    mla.mla_cache_append_scaled(kv, x, cu, mla.mla_rope_init(), positions.to(DEV), norm_weight=weight)
    out = mla.mla_cache_gather(kv, cu, 170, dtype=torch.float32).double().cpu().numpy()
    y, slack = expected(x, 1.0, weight, 1e-6, frequencies(10000.0, 1.0, 0), positions, True)
    # every block holds an entry above 1, so no scale is below 2^-8: subnormal steps of 2^-17 and less
    assert np.all(np.abs(out - y) <= 2.0 ** -4 * np.abs(y) + slack + 2.0 ** -16)


def test_offsets_past_32_bits():
    """A pool of 5 GiB: bytes past 2^32, rows past 2^22, written and read."""
    pages = (5 << 30) // (64 * 576)
    pool = torch.zeros(pages, 64, 576, dtype=torch.uint8, device=DEV)
    scales = torch.ones(pages, 64, device=DEV)
    table = torch.tensor([[pages - 1, pages // 2]], dtype=torch.int32, device=DEV)
    kv = mla.KVCache(pool, table, torch.tensor([70], dtype=torch.int32, device=DEV), 1.0, scales=scales)
    x = torch.randn(70, 576, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    cu = torch.tensor([0, 70], device=DEV)
    mla.mla_cache_append_scaled(kv, x, cu)
    out = mla.mla_cache_gather(kv, cu, 70, dtype=torch.float32)
    # largest entries of a row are above 1, so its scale is at least 2^-8 and at most 2^-6: steps of 2^-15
    assert torch.all((out - x.float()).abs() <= 2.0 ** -4 * x.float().abs() + 2.0 ** -16)
    assert int((pool.view(-1, 576)[:64] != 0).sum()) == 0
