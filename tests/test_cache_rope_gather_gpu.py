"""mla_cache_append_rope and mla_cache_gather against the definitions in float64.

Codes. The kernel's float32 value is within 2^-20 of the exact one, relatively: a sum of 512
squares in chains of 16 and a tree of 5 (21 roundings of 2^-24, halved by the root), rsqrtf (2
ulp), three products; the RoPE part within 2^-19 (|a| + |b|) (see test_rope_gpu.py). Rounding that
to e4m3 (steps 2^(e - 3) for 2^e <= |v| < 2^(e + 1), e >= -6) leaves at most half a step more."""
import numpy as np
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from tests.test_rope_gpu import frequencies, rotate

pytestmark = pytest.mark.gpu
DEV = "cuda"


def decode(codes):
    return codes.cpu().view(torch.float8_e4m3fn).to(torch.float64).numpy()


def expected(x, kv_scale, weight, eps, f, positions, interleaved):
    """Values before quantisation over kv_scale, and the float32 error they may carry."""
    x = x.double().cpu().numpy()
    c, r = x[:, :512], x[:, 512:]
    if weight is not None:
        c = c / np.sqrt((c ** 2).mean(-1, keepdims=True) + eps) * weight.double().cpu().numpy()
    slack = np.concatenate([2.0 ** -20 * np.abs(c), 0 * r], -1)
    if f is not None:
        y, size = rotate(r[:, None], positions.tolist(), f, 1.0, interleaved)
        r = y[:, 0]
        slack[:, 512:] = 2.0 ** -19 * size[:, 0]
    return np.concatenate([c, r], -1) / kv_scale, slack / kv_scale


def check_codes(got, v, slack):
    v = np.clip(v, -448, 448)
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 1e-30))), -6)
    bound = 2.0 ** (e - 4) + slack + 2.0 ** -22 * np.abs(v)  # (the last: 1 / kv_scale, two roundings)
    assert np.all(np.abs(got - v) <= bound)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,stride,page_size", [(1, 576, 64), (2, 2112, 64), (37, 640, 128), (1000, 576, 64),
                                                (12000, 2112, 64)])
def test_append_rope(n, stride, page_size, interleaved):
    g = torch.Generator().manual_seed(n)
    pages = -(-2 * n // page_size)
    pool = torch.randint(0, 256, (pages, page_size, 576), dtype=torch.uint8, generator=g)
    x = (torch.randn(n, stride, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g))).bfloat16()
    x = x.to(DEV)[:, stride - 576:]
    slots = torch.randperm(pages * page_size, generator=g)[:n]
    slots[3::5] = -1
    positions = torch.randint(-100, 150000, (n,), generator=g)
    weight = torch.randn(512, generator=g).bfloat16().to(DEV)
    rope = mla.mla_rope_init(factor=40.0, original_positions=4096, interleaved=interleaved)
    f = frequencies(10000.0, 40.0, 4096)
    d = pool.to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.mla_cache_append_rope(d, x, slots.to(DEV), 0.0125, rope, positions.to(DEV), norm_weight=weight,
                              eps=1e-5, status=status)
    assert int(status) == 0
    flat, before = d.view(-1, 576).cpu(), pool.view(-1, 576).clone()
    keep = slots >= 0
    v, slack = expected(x, 0.0125, weight, 1e-5, f, positions, interleaved)
    check_codes(decode(flat[slots[keep]]), v[keep.numpy()], slack[keep.numpy()])
    rest = torch.ones(len(before), dtype=torch.bool)
    rest[slots[keep]] = False
    assert torch.equal(flat[rest], before[rest])  # rows of other slots stay as they were


def test_parts_may_be_left_out():
    """Without a norm and without a rotation it writes what mla_cache_append writes, byte for
    byte (saturation, infinities, NaN and signed zeros included); each part works alone."""
    g = torch.Generator().manual_seed(5)
    x = (torch.randn(70, 576, generator=g) * 3).bfloat16()
    x[0, :6] = torch.tensor([1e30, -1e30, float("inf"), -float("inf"), -0.0, 0.0]).bfloat16()
    x[1, 5], x[2, 570] = float("nan"), float("nan")
    x = x.to(DEV)
    slots = torch.randperm(128, generator=g)[:70].to(DEV)
    a, b, c, d = (torch.zeros(2, 64, 576, dtype=torch.uint8, device=DEV) for _ in range(4))
    mla.mla_cache_append(a, x, slots, 0.02)
    mla.mla_cache_append_rope(b, x, slots, 0.02)
    assert torch.equal(a, b)
    positions = torch.arange(70, device=DEV)
    rope = mla.mla_rope_init(interleaved=False)
    weight = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    mla.mla_cache_append_rope(c, x, slots, 0.02, rope, positions)
    assert torch.equal(c[..., :512], a[..., :512])
    mla.mla_cache_append_rope(d, x, slots, 0.02, norm_weight=weight)
    assert torch.equal(d[..., 512:], a[..., 512:])
    rows = slots[3:].cpu()
    v, slack = expected(x[3:], 0.02, weight, 1e-6, frequencies(10000.0, 1.0, 0), positions[3:], False)
    check_codes(decode(c.view(-1, 576).cpu()[rows])[:, 512:], v[:, 512:], slack[:, 512:])
    check_codes(decode(d.view(-1, 576).cpu()[rows])[:, :512], v[:, :512], slack[:, :512])


def test_append_rope_bounds_and_zero_rows():
    x = torch.zeros(4, 576, dtype=torch.bfloat16, device=DEV)
    weight = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    pool = torch.full((1, 64, 576), 9, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    slots = torch.tensor([3, 64, 2 ** 40, -1], device=DEV)
    mla.mla_cache_append_rope(pool, x, slots, 0.02, norm_weight=weight, eps=1e-6, status=status)
    assert int(status) == mla.MLA_ERR_BOUNDS
    flat = pool.view(-1, 576)
    assert torch.all(flat[3] == 0) and torch.all(flat[:3] == 9) and torch.all(flat[4:] == 9)


def paged(lens, g, page_size=64, spare=3):
    pages = [-(-n // page_size) for n in lens]
    order = torch.randperm(sum(pages) + spare, generator=g).int()
    table = torch.full((len(lens), max(pages + [1])), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = order[at:at + k]
        at += k
    pool = torch.randint(0, 256, (sum(pages) + spare, page_size, 576), dtype=torch.uint8, generator=g)
    pool[(pool & 0x7F) == 0x7F] = 0  # no NaN codes
    return mla.KVCache(pool.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), 0.0173)


def rows_of(kv, b, lo, hi):
    size = kv.pool.shape[1]
    pos = torch.arange(lo, hi)
    return kv.pool.cpu()[kv.page_table[b].cpu()[pos // size].long(), pos % size]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,starts,page_size", [
    ([1], None, 64), ([64, 65, 63], None, 64), ([100, 0, 7, 300], [99, 0, 0, 5], 64),
    ([5000, 1, 129], [0, 1, 100], 128), ([33] * 70, None, 64)])
def test_gather(lens, starts, page_size, dtype):
    g = torch.Generator().manual_seed(len(lens))
    kv = paged(lens, g, page_size)
    lo = starts or [0] * len(lens)
    cu = np.cumsum([0] + [n - a for n, a in zip(lens, lo)])
    n = int(cu[-1]) + 3  # and rows behind the last sequence
    out = torch.full((n, 576), 5.0, dtype=dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = mla.mla_cache_gather(kv, torch.tensor(cu, device=DEV), n, out=out, status=status,
                               starts=None if starts is None else torch.tensor(lo, dtype=torch.int32, device=DEV))
    assert got is out and int(status) == 0
    want = torch.cat([rows_of(kv, b, a, m) for b, (m, a) in enumerate(zip(lens, lo))])
    want = (want.view(torch.float8_e4m3fn).float() * torch.tensor(0.0173)).to(dtype)  # one product, one rounding
    assert torch.equal(out[:-3].cpu(), want)
    assert torch.all(out[-3:] == 5.0)


def test_gather_reports_bounds():
    """Positions past a sequence, before it, on a page outside the pool: zero rows and a status;
    rows before cu_rows[0] are left alone."""
    kv = paged([100, 200, 64], torch.Generator().manual_seed(9))
    kv.page_table[1, 2] = kv.pool.shape[0]
    cu = torch.tensor([2, 6, 206, 210], device=DEV)
    starts = torch.tensor([98, 0, -2], dtype=torch.int32, device=DEV)
    out = torch.full((212, 576), 5.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.mla_cache_gather(kv, cu, 212, starts=starts, out=out, status=status)
    assert int(status) == mla.MLA_ERR_BOUNDS
    got = out.cpu()
    assert torch.all(got[:2] == 5.0) and torch.all(got[210:] == 5.0)
    value = lambda b, lo, hi: rows_of(kv, b, lo, hi).view(torch.float8_e4m3fn).float() * torch.tensor(0.0173)
    assert torch.equal(got[2:4], value(0, 98, 100)) and torch.all(got[4:6] == 0)
    assert torch.equal(got[6:134], value(1, 0, 128)) and torch.all(got[134:198] == 0)
    assert torch.equal(got[198:206], value(1, 192, 200))
    assert torch.all(got[206:208] == 0) and torch.equal(got[208:210], value(2, 0, 2))


def test_gather_past_32_bit_offsets():
    """Rows whose byte offsets in the pool and in the output pass 2^31 and 2^32."""
    pages = (5 << 30) // (64 * 576)  # a pool of 5 GiB
    pool = torch.zeros(pages, 64, 576, dtype=torch.uint8, device=DEV)
    pool[-1, 63] = 0x38  # 1.0
    pool[-1, 62] = 0x40  # 2.0
    n = 4_000_000
    table = torch.zeros(1, -(-n // 64), dtype=torch.int32, device=DEV)
    table[0, -1] = pages - 1
    kv = mla.KVCache(pool, table, torch.tensor([n], dtype=torch.int32, device=DEV), 1.0)
    out = mla.mla_cache_gather(kv, torch.tensor([0, n], device=DEV), n)
    assert torch.all(out[-1] == 1.0) and torch.all(out[-2] == 2.0) and torch.all(out[-3] == 0.0)


def test_gather_refusals():
    kv = paged([100], torch.Generator().manual_seed(1))
    cu = torch.tensor([0, 100], device=DEV)
    for kw in (dict(cu_rows=cu.int()), dict(cu_rows=torch.zeros(3, dtype=torch.int64, device=DEV)),
               dict(cu_rows=cu, starts=torch.zeros(1, device=DEV)), dict(cu_rows=cu, dtype=torch.float16),
               dict(cu_rows=cu, out=torch.zeros(99, 576, device=DEV)), dict(cu_rows=cu.cpu())):
        with pytest.raises(ValueError):
            mla.mla_cache_gather(kv, n=100, **kw)


def test_written_rows_read_back():
    """The pair: rows written through the norm and the rotation come back as the codes' values."""
    g = torch.Generator().manual_seed(8)
    kv = paged([130, 40], g)
    x = torch.randn(170, 576, generator=g).bfloat16().to(DEV)
    weight = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    positions = torch.cat([torch.arange(130), torch.arange(40)]).to(DEV)
    seq = torch.tensor([0] * 130 + [1] * 40, device=DEV)
    slots = kv.page_table[seq, positions // 64].long() * 64 + positions % 64
    rope = mla.mla_rope_init(interleaved=True)
    mla.mla_cache_append_rope(kv.pool, x, slots, kv.kv_scale, rope, positions, norm_weight=weight)
    out = mla.mla_cache_gather(kv, torch.tensor([0, 130, 170], device=DEV), 170, dtype=torch.float32)
    v, slack = expected(x, 1.0, weight, 1e-6, frequencies(10000.0, 1.0, 0), positions, True)
    check_codes(out.double().cpu().numpy() / kv.kv_scale, v / kv.kv_scale, slack / kv.kv_scale)
