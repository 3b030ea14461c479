"""Codes under scales that are no powers of two (kept from elsewhere) are rounded once: scales are
chosen so that quotients and products lie beside a tie of e4m3, within a float32 step of it, where
a float32 quotient, or a product with the reciprocal, lands on the tie or past it. Expected codes in
exact fractions."""
from fractions import Fraction as F

import numpy as np
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla

pytestmark = pytest.mark.gpu
DEV = "cuda"


def eighths(v):
    """A number in [1, 2) in eighths (e4m3's step there), to nearest, ties to even."""
    n, rest = divmod(v * 8, 1)
    return int(n) + (rest > F(1, 2) or (rest == F(1, 2) and n % 2))


def cache(scales):
    """A sequence of two positions for each scale, one block each."""
    B = len(scales)
    s = torch.ones(B, 32)
    s[:, 0] = torch.tensor(scales)
    pool = torch.zeros(B, 64, 576, dtype=torch.uint8)
    return mla.KVCache(pool.to(DEV), torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1),
                       torch.full((B,), 2, dtype=torch.int32, device=DEV), 1.0, scales=s.to(DEV))


def values(kv):
    return kv.pool[:, :2].view(torch.float8_e4m3fn).double()


def test_new_rows_under_a_kept_scale():
    """y / s: y of eight bits, s the float32 beside y / tie."""
    cases = []
    for y in range(128, 256):
        for tie in range(17, 32, 2):
            s = np.float32(float(F(y, 128) / F(tie, 16)))
            exact = F(y, 128) / F(float(s))
            if exact != F(tie, 16):
                cases.append((y / 128, float(s), eighths(exact) / 8))
    wrong = sum(eighths(F(float(np.float32(y) * (np.float32(1) / np.float32(s))))) / 8 != w for y, s, w in cases)
    assert wrong > 300  # (what the reciprocal would get)
    kv = cache([s for _, s, _ in cases])
    x = torch.tensor([y for y, _, _ in cases]).bfloat16()[:, None].repeat(1, 576)
    x[:, 1::2] *= -1
    scales = kv.scales.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.mla_cache_append_scaled(kv, x.to(DEV), torch.arange(len(cases) + 1, device=DEV), status=status)
    assert int(status) == 0 and torch.equal(kv.scales, scales)
    want = torch.tensor([w for _, _, w in cases], dtype=torch.float64, device=DEV)[:, None].repeat(1, 576)
    want[:, 1::2] *= -1
    got = values(kv)
    assert torch.equal(got[:, 1], want) and not bool(got[:, 0].any())


def test_earlier_rows_of_a_block_that_grows():
    """code * s_old / s: s a power of two, s_old the float32 beside tie * s / code."""
    cases = []
    for code in range(8, 16):
        for tie in range(17, 32, 2):
            old = np.float32(float(F(tie, 16) * 8 / F(code, 8)))
            for old in (old, np.nextafter(old, np.float32(0)), np.nextafter(old, np.float32(100))):
                exact = F(code, 8) * F(float(old)) / 8
                if exact != F(tie, 16) and old < 16 and 1 <= exact < 2:
                    cases.append((code, float(old), eighths(exact) / 8))
    wrong = sum(eighths(F(float(np.float32(c / 8) * np.float32(o / 8)))) / 8 != w for c, o, w in cases)
    assert wrong > 20  # (what the rounded product would get)
    kv = cache([o for _, o, _ in cases])
    codes = torch.tensor([c / 8 for c, _, _ in cases]).to(torch.float8_e4m3fn).view(torch.uint8)
    kv.pool[:, 0] = codes.to(DEV)[:, None]
    kv.pool[:, 0, 1::2] |= 0x80
    x = torch.zeros(len(cases), 576, dtype=torch.bfloat16)
    x[:, 5] = 448 * 16
    mla.mla_cache_append_scaled(kv, x.to(DEV), torch.arange(len(cases) + 1, device=DEV))
    assert bool((kv.scales[:, 0] == 16).all())
    want = torch.tensor([w for _, _, w in cases], dtype=torch.float64, device=DEV)[:, None].repeat(1, 576) / 2
    want[:, 1::2] *= -1
    got = values(kv)
    assert torch.equal(got[:, 0], want)
    assert bool((got[:, 1, 5] == 448).all()) and float(got[:, 1].sum()) == 448 * len(cases)


@pytest.mark.parametrize("block", [1, 2, 4, 8, 16, 32, 64])
def test_special_values_under_a_kept_scale(block):
    """As under a power of two: infinities saturate, NaN stays with its entry, zeros and what is far below the
    smallest code are zero. (Blocks of one have no earlier position: their scale is a power of two.)"""
    pool = torch.zeros(1, 64, 576, dtype=torch.uint8, device=DEV)
    kv = mla.KVCache(pool, torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.full((1,), 2, dtype=torch.int32, device=DEV),
                     1.0, scales=torch.full((1, 64 // block), 0.3, device=DEV))
    x = torch.ones(1, 576, dtype=torch.bfloat16)
    x[0, :7] = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 1e-38, -1e-38])
    x[0, 570:573] = torch.tensor([float("inf"), -float("inf"), float("nan")])
    mla.mla_cache_append_scaled(kv, x.to(DEV), torch.tensor([0, 1], device=DEV))
    v = values(kv)[0, 1]
    assert v[[0, 1, 570, 571]].tolist() == [448, -448, 448, -448] and bool(torch.isnan(v[[2, 572]]).all())
    assert not bool(v[3:7].any())
    s = float(kv.scales.view(-1)[1 // block])
    assert s == (2.0 ** -8 if block == 1 else float(np.float32(0.3)))
    assert bool((v[7:570] == (256.0 if block == 1 else 3.25)).all())  # (1 / 0.3 is nearest to 3.25)
