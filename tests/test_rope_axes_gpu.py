"""mla_rope and mla_cache_append_rope for positions with several axes, against the definition in float64.

Tolerances as in test_rope_gpu.py and test_cache_rope_gather_gpu.py: a pair's phase is the product of
one position and one frequency as there, so nothing is added."""
import math

import numpy as np
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from tests.test_cache_rope_gather_gpu import check_codes, decode, expected
from tests.test_rope_gpu import frequencies

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rotate(x, positions, axis, f, amplitude, interleaved):
    """x [n, H, 64] float64 numpy; positions [axes][n] python ints; axis[i] the axis of pair i."""
    n = len(positions[0])
    angle = np.array([[math.fmod(float(positions[axis[i]][t]) * f[i], 2 * math.pi) for i in range(32)] for t in range(n)])
    angle = angle.reshape(n, 32)
    c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None]
    a, b = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    y, size = np.empty_like(x), np.empty_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size * abs(amplitude)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sections,mixed", [([8, 12, 12], False), ([12, 10, 10], True), ([32], False), ([0, 16, 16], True),
                                            ([1, 2, 3, 26], True)])
@pytest.mark.parametrize("n,H,width", [(1, 1, 64), (33, 12, 192), (1700, 12, 576)])
def test_views(n, H, width, sections, mixed, interleaved):
    g = torch.Generator().manual_seed(n + H)
    x = torch.randn(n, H, width, generator=g).bfloat16().to(DEV)
    positions = torch.randint(-100, 200000, (len(sections), n), generator=g)
    axes = mla.mla_rope_axes_init(sections, interleaved=mixed)
    rope = mla.mla_rope_init(10000.0, factor=40.0, original_positions=4096, amplitude=1.25, interleaved=interleaved)
    out = torch.full((n, H, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    part = x[..., width - 64:]
    got = mla.mla_rope(rope, part, positions.to(DEV), out=out[..., 512:], axes=axes)
    assert got.data_ptr() == out[..., 512:].data_ptr()
    ref, size = rotate(part.double().cpu().numpy(), positions.tolist(), list(axes.axis), frequencies(10000.0, 40.0, 4096),
                       1.25, interleaved)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * size + 1e-30)
    assert torch.all(out[..., :512] == 7.0)


def test_equal_axes_are_one_position():
    """Text: every axis the same position turns as a call without axes does, bit for bit; in place too."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(300, 5, 64, generator=g).bfloat16().to(DEV)
    at = torch.randint(0, 10 ** 6, (300,), generator=g).to(DEV)
    for pairs in (False, True):
        rope = mla.mla_rope_init(factor=4.0, interleaved=pairs)
        want = mla.mla_rope(rope, x, at)
        axes = mla.mla_rope_axes_init([10, 11, 11], interleaved=pairs)
        y = x.clone()
        assert mla.mla_rope(rope, y, at.expand(3, 300).contiguous(), out=y, axes=axes) is y
        assert torch.equal(y, want)
        assert torch.equal(mla.mla_rope(rope, x, at[None].contiguous(), axes=mla.mla_rope_axes_init([32])), want)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [1, 37, 9000])
def test_append(n, interleaved):
    g = torch.Generator().manual_seed(n)
    pages = -(-2 * n // 64)
    pool = torch.randint(0, 256, (pages, 64, 576), dtype=torch.uint8, generator=g)
    x = torch.randn(n, 640, generator=g).bfloat16().to(DEV)[:, 64:]
    slots = torch.randperm(pages * 64, generator=g)[:n]
    slots[3::5] = -1
    positions = torch.randint(-100, 150000, (3, n), generator=g)
    weight = torch.randn(512, generator=g).bfloat16().to(DEV)
    rope, axes = mla.mla_rope_init(interleaved=interleaved), mla.mla_rope_axes_init([12, 10, 10], interleaved=True)
    d, status = pool.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.mla_cache_append_rope(d, x, slots.to(DEV), 0.0125, rope, positions.to(DEV), norm_weight=weight, status=status,
                              axes=axes)
    assert int(status) == 0
    keep = slots >= 0
    f = frequencies(10000.0, 1.0, 0)
    v, slack = expected(x, 0.0125, weight, 1e-6, None, None, interleaved)
    y, size = rotate(x[:, None, 512:].double().cpu().numpy(), positions.tolist(), list(axes.axis), f, 1.0, interleaved)
    v[:, 512:], slack[:, 512:] = y[:, 0] / 0.0125, 2.0 ** -19 * size[:, 0] / 0.0125
    flat, before = d.view(-1, 576).cpu(), pool.view(-1, 576)
    check_codes(decode(flat[slots[keep]]), v[keep.numpy()], slack[keep.numpy()])
    rest = torch.ones(len(before), dtype=torch.bool)
    rest[slots[keep]] = False
    assert torch.equal(flat[rest], before[rest])


def test_refusals():
    rope, axes = mla.mla_rope_init(), mla.mla_rope_axes_init([8, 12, 12])
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    at = torch.zeros(3, 4, dtype=torch.int64, device=DEV)
    for bad in (at.int(), at[0], at[:2], at.T.contiguous(), at.T, at.cpu(), at[:, :3]):
        with pytest.raises(ValueError):
            mla.mla_rope(rope, x, bad, axes=axes)
    with pytest.raises(ValueError):
        mla.mla_rope(rope, x, at)  # several axes' positions without their axes
    pool = torch.zeros(1, 64, 576, dtype=torch.uint8, device=DEV)
    rows, slots = torch.zeros(4, 576, dtype=torch.bfloat16, device=DEV), torch.arange(4, device=DEV)
    with pytest.raises(ValueError):
        mla.mla_cache_append_rope(pool, rows, slots, 1.0, axes=axes)
    with pytest.raises(ValueError):
        mla.mla_cache_append_rope(pool, rows, slots, 1.0, rope, at[0], axes=axes)
    assert mla.mla_rope(rope, x[:0], at[:, :0].contiguous(), axes=axes).shape == (0, 2, 64)
