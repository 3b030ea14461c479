"""mla_rope_init and the refusals of the calls around it, without a GPU."""
import ctypes
import math
from fractions import Fraction

import pytest

import mla_latent_kv_attention_gb300 as mla
from tests.test_abi import FAKE, _kv
from tests.test_rope_gpu import frequencies


@pytest.mark.parametrize("base,factor,original", [(10000.0, 1.0, 0), (10000.0, 4.0, 0), (10000.0, 40.0, 4096),
                                                  (500000.0, 8.0, 8192), (10000.0, 0.25, 0), (1.5, 1.0, 0)])
def test_turns(base, factor, original):
    rope = mla.mla_rope_init(base, factor=factor, original_positions=original, amplitude=0.75,
                             interleaved=False)
    assert rope.amplitude == 0.75 and rope.interleaved == 0
    for got, f in zip(rope.turns, frequencies(base, factor, original)):
        turn = Fraction(f) / Fraction(2 * math.pi)  # in float64's pi, like the library
        part = (turn - math.floor(turn)) * 2 ** 64
        # a few roundings of 2^-53 relative to the whole turns a position adds
        assert abs(got - part) <= max(1, Fraction(turn) * 2 ** 64 * Fraction(8, 2 ** 53))


@pytest.mark.parametrize("kw", [dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
                                dict(factor=0.0), dict(factor=-1.0), dict(factor=float("inf")),
                                dict(original_positions=-1), dict(amplitude=float("nan")),
                                dict(original_positions=4096, beta_fast=1.0, beta_slow=1.0),
                                dict(original_positions=4096, beta_slow=0.0)])
def test_init_refusals(kw):
    with pytest.raises(mla.MlaError) as e:
        mla.mla_rope_init(**kw)
    assert e.value.status == mla.MLA_ERR_INVALID_ARG


def test_rope_refusals():
    lib, r = mla.library(), ctypes.byref(mla.mla_rope_init())
    ok = dict(rope=r, x=FAKE, xt=768, xh=64, positions=FAKE, n=3, H=12, out=FAKE, ot=768, oh=64)

    def call(**kw):
        return lib.mla_rope(*dict(ok, **kw).values(), None)

    for kw in (dict(rope=None), dict(x=None), dict(out=None), dict(positions=None), dict(n=-1), dict(H=-1),
               dict(x=FAKE + 8), dict(out=FAKE + 2), dict(positions=FAKE + 4), dict(xt=65), dict(xh=12),
               dict(ot=4), dict(oh=-7)):
        assert call(**kw) == mla.MLA_ERR_INVALID_ARG, kw
    assert call(n=1 << 41, H=1) == mla.MLA_ERR_UNSUPPORTED
    assert call(n=1 << 39, H=1 << 20) == mla.MLA_ERR_UNSUPPORTED
    assert call(n=0) == 0 and call(H=0) == 0
    assert lib.mla_last_launch_count() == 0


def test_append_rope_refusals():
    lib, r = mla.library(), ctypes.byref(mla.mla_rope_init())
    ok = dict(pool=FAKE, pages=4, page_size=64, x=FAKE, stride=576, slots=FAKE, n=3, kv_scale=0.5,
              weight=FAKE, eps=1e-6, rope=r, positions=FAKE, status=None)

    def call(**kw):
        return lib.mla_cache_append_rope(*dict(ok, **kw).values(), None)

    for kw in (dict(n=-1), dict(pages=-1), dict(page_size=0), dict(kv_scale=0.0), dict(kv_scale=float("nan")),
               dict(eps=-1.0), dict(eps=float("nan")), dict(rope=None), dict(positions=None), dict(stride=568),
               dict(stride=580), dict(pool=None), dict(x=None), dict(slots=None), dict(x=FAKE + 8),
               dict(weight=FAKE + 2), dict(positions=FAKE + 4), dict(status=FAKE + 1)):
        assert call(**kw) == mla.MLA_ERR_INVALID_ARG, kw
    assert call(n=0, x=None, slots=None) == 0
    assert lib.mla_last_launch_count() == 0


def test_gather_refusals():
    lib = mla.library()
    kv = _kv()
    ok = dict(kv=ctypes.byref(kv), B=2, starts=None, cu=FAKE, n=5, out=FAKE, f32=0, status=None)

    def call(**kw):
        return lib.mla_cache_gather(*dict(ok, **kw).values(), None)

    for kw in (dict(kv=None), dict(B=-1), dict(n=-1), dict(cu=None), dict(out=None), dict(starts=FAKE + 2),
               dict(cu=FAKE + 4), dict(out=FAKE + 8), dict(status=FAKE + 1),
               dict(kv=ctypes.byref(_kv(pool=None)))):
        assert call(**kw) == mla.MLA_ERR_INVALID_ARG, kw
    assert call(kv=ctypes.byref(_kv(page_size=48))) == mla.MLA_ERR_UNSUPPORTED
    assert call(n=1 << 40) == mla.MLA_ERR_UNSUPPORTED
    assert call(n=0, out=None, cu=None) == 0 and call(B=0) == 0
    assert lib.mla_last_launch_count() == 0


def test_verify_tree_refusals():
    lib = mla.library()
    kv = _kv()
    ok = dict(kv=ctypes.byref(kv), q=FAKE, B=2, n=8, H=12, scale=0.1, mask=FAKE, out=FAKE, lse=FAKE, ws=FAKE,
              ws_bytes=1 << 30)

    def call(**kw):
        return lib.mla_verify_tree(*dict(ok, **kw).values(), None)

    for kw in (dict(kv=None), dict(B=-1), dict(q=None), dict(out=None), dict(mask=None), dict(q=FAKE + 8),
               dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(mask=FAKE + 4)):
        assert call(**kw) == mla.MLA_ERR_INVALID_ARG, kw
    for kw in (dict(n=0), dict(n=65), dict(H=0), dict(H=17), dict(B=1 << 24, n=64, H=16),
               dict(kv=ctypes.byref(_kv(page_size=32)))):
        assert call(**kw) == mla.MLA_ERR_UNSUPPORTED, kw
    assert call(ws=None) == mla.MLA_ERR_WORKSPACE and call(ws=FAKE + 16) == mla.MLA_ERR_WORKSPACE
    assert lib.mla_last_launch_count() == 0
    for args in ((3, 1, 12, 0, 0), (3, 1, 12, 65, 0), (3, 1, 17, 8, 0), (3, -1, 12, 8, 0)):
        assert lib.mla_workspace_size(*args) == 0


def test_accept_refusals():
    lib = mla.library()
    ok = dict(target=FAKE, tokens=FAKE, parents=None, draft=None, u=FAKE, B=2, n=4, V=100, out=FAKE, path=FAKE,
              count=FAKE)

    def call(**kw):
        return lib.mla_accept_drafts(*dict(ok, **kw).values(), None)

    for kw in (dict(B=-1), dict(target=None), dict(tokens=None), dict(u=None), dict(out=None), dict(path=None),
               dict(count=None), dict(target=FAKE + 2), dict(draft=FAKE + 1), dict(parents=FAKE + 2)):
        assert call(**kw) == mla.MLA_ERR_INVALID_ARG, kw
    for kw in (dict(n=0), dict(n=65), dict(V=0), dict(V=(1 << 19) + 1), dict(B=1 << 16),
               dict(parents=FAKE, draft=FAKE)):
        assert call(**kw) == mla.MLA_ERR_UNSUPPORTED, kw
    assert call(B=0, target=None) == 0
    assert lib.mla_last_launch_count() == 0
