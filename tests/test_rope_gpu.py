"""mla_rope and mla_rope_init against the definition in float64.

Tolerances. The phase is exact up to 2^-64 turns a position (turns holds 53 significant bits:
a further 2^-53 of the angle), its top 32 bits lose 2^-32 turns and their rounding to float32
2^-25 half turns, sincospif adds 2 ulp (2^-22 relative to 1): cos and sin are within 2^-21. An
output is a sum of two products, each operand at most |a|, |b|, rounded three times in float32
and once to bfloat16 (2^-8 of the value): |error| <= 2^-8 |y| + 2^-19 (|a| + |b|) amplitude."""
import math

import numpy as np
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla

pytestmark = pytest.mark.gpu
DEV = "cuda"


def frequencies(base, factor, original, fast=32.0, slow=1.0):
    """Radians per position, pair by pair, from the definition."""
    f = [base ** (-2.0 * i / 64) for i in range(32)]
    if original == 0:
        return [x / factor for x in f]
    # the pair that turns r times over the original positions
    at = lambda r: 32 * math.log(original / (2 * math.pi * r)) / math.log(base)
    low, high = max(0, math.floor(at(fast))), min(63, math.ceil(at(slow)))
    out = []
    for i, x in enumerate(f):
        ramp = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
        out.append(x / factor * ramp + x * (1 - ramp))
    return out


def rotate(x, positions, f, amplitude, interleaved):
    """x [n, H, 64] float64 numpy; positions python ints."""
    angle = np.array([[math.fmod(float(p) * w, 2 * math.pi) for w in f] for p in positions])
    c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None]
    y = np.empty_like(x)
    a, b = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    size = np.empty_like(x)
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size * abs(amplitude)


def check(got, x, positions, f, amplitude, interleaved):
    ref, size = rotate(x.double().cpu().numpy(), positions.tolist(), f, amplitude, interleaved)
    got = got.double().cpu().numpy()
    # the float64 angle of position p is off by p * f * 2^-53 (below 2^-32 for every position here)
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * size + 1e-30)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,H,width", [(1, 1, 64), (3, 12, 192), (33, 16, 576), (257, 5, 192),
                                       (1700, 12, 192), (5000, 1, 64)])
def test_views(n, H, width, interleaved):
    g = torch.Generator().manual_seed(n + H)
    x = torch.randn(n, H, width, generator=g).bfloat16().to(DEV)
    positions = torch.randint(0, 200000, (n,), generator=g).to(DEV)
    out = torch.full((n, H, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    rope = mla.mla_rope_init(10000.0, factor=40.0, original_positions=4096, amplitude=1.25,
                             interleaved=interleaved)
    part = x[..., width - 64:]
    got = mla.mla_rope(rope, part, positions, out=out[..., 512:])
    assert got.data_ptr() == out[..., 512:].data_ptr()
    check(got, part, positions, frequencies(10000.0, 40.0, 4096), 1.25, interleaved)
    assert torch.all(out[..., :512] == 7.0)  # nothing beside the RoPE dims is touched


@pytest.mark.parametrize("base,factor,original", [(10000.0, 1.0, 0), (10000.0, 8.0, 0), (500000.0, 1.0, 0),
                                                  (10000.0, 32.0, 8192), (50000.0, 0.5, 0)])
def test_far_positions(base, factor, original):
    """Angles stay exact where float32 angles are off by radians; positions may be negative."""
    positions = torch.tensor([0, 1, -1, 4095, 4096, 999_983, 2 ** 24 + 1, -(2 ** 24) - 1, 2 ** 31 + 11])
    x = torch.randn(len(positions), 2, 64, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    rope = mla.mla_rope_init(base, factor=factor, original_positions=original, interleaved=False)
    got = mla.mla_rope(rope, x, positions.to(DEV))
    f = frequencies(base, factor, original)
    ref, size = rotate(x.double().cpu().numpy(), positions.tolist(), f, 1.0, False)
    # the oracle's own float64 product: |p f| 2^-53 of an angle; turns rounds likewise
    slack = 2.0 ** -52 * np.abs(positions.numpy())[:, None, None] * size
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * size + slack)


def test_position_zero_is_exact_and_norms_are_kept():
    x = torch.randn(64, 3, 64, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    rope = mla.mla_rope_init()
    zero = torch.zeros(64, dtype=torch.int64, device=DEV)
    assert torch.equal(mla.mla_rope(rope, x, zero), x)
    y = mla.mla_rope(rope, x, torch.arange(64, device=DEV) * 1001).double()
    assert torch.allclose(y.norm(dim=-1), x.double().norm(dim=-1), rtol=2.0 ** -8)


def test_in_place_and_orders():
    """In place gives what a fresh output gives; token and head strides in either order, and one
    row shared by every head (stride 0) read from."""
    g = torch.Generator().manual_seed(3)
    rope = mla.mla_rope_init(interleaved=True)
    base = torch.randn(7, 90, 64, generator=g).bfloat16().to(DEV)  # [H, n, 64] in memory
    x = base.transpose(0, 1)
    positions = torch.randint(0, 5000, (90,), generator=g).to(DEV)
    want = mla.mla_rope(rope, x, positions)
    check(want, x, positions, frequencies(10000.0, 1.0, 0), 1.0, True)
    shared = x[:, :1].expand(90, 4, 64)
    got = mla.mla_rope(rope, shared, positions)
    assert torch.equal(got, want[:, :1].expand(90, 4, 64))
    assert mla.mla_rope(rope, x, positions, out=x) is x
    assert torch.equal(x, want)


def test_one_token_or_head_of_odd_strides():
    """Dimensions of size one have no stride, whatever the tensor says."""
    g = torch.Generator().manual_seed(4)
    rope = mla.mla_rope_init()
    a = torch.randn(3, 5, 72, generator=g).bfloat16().to(DEV)
    one = torch.as_strided(a, (1, 5, 64), (363, 72, 1))
    got = mla.mla_rope(rope, one, torch.tensor([77], device=DEV))
    check(got, one, torch.tensor([77]), frequencies(10000.0, 1.0, 0), 1.0, True)
    head = torch.as_strided(a, (3, 1, 64), (360, 5, 1))
    got = mla.mla_rope(rope, head, torch.tensor([5, 6, 7], device=DEV))
    check(got, head, torch.tensor([5, 6, 7]), frequencies(10000.0, 1.0, 0), 1.0, True)


def test_special_values_stay_in_their_pair():
    x = torch.ones(2, 1, 64).bfloat16()
    x[0, 0, 4] = float("inf")
    x[1, 0, 40] = float("nan")
    rope = mla.mla_rope_init(interleaved=False)
    y = mla.mla_rope(rope, x.to(DEV), torch.tensor([3, 3], device=DEV)).float().cpu()
    bad = ~torch.isfinite(y)
    assert bad[0, 0].nonzero().flatten().tolist() == [4, 36]
    assert bad[1, 0].nonzero().flatten().tolist() == [8, 40]


def test_refusals():
    rope = mla.mla_rope_init()
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    positions = torch.zeros(4, dtype=torch.int64, device=DEV)
    for bad in (x.float(), x[..., :32], x[0], x.cpu(), x.transpose(1, 2)):
        with pytest.raises(ValueError):
            mla.mla_rope(rope, bad, positions)
    for bad in (positions.int(), positions[:3], positions.cpu()):
        with pytest.raises(ValueError):
            mla.mla_rope(rope, x, bad)
    with pytest.raises(ValueError):  # one place for several tokens' outputs
        mla.mla_rope(rope, x, positions, out=x[:1].expand(4, 2, 64))
    wide = torch.zeros(4, 2, 68, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(mla.MlaError):  # 8-byte aligned rows
        mla.mla_rope(rope, wide[..., 4:], positions)
    assert mla.mla_rope(rope, x[:0], positions[:0]).shape == (0, 2, 64)
