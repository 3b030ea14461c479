"""What the calls on a cache with block scales refuse, without a GPU."""
import ctypes

import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from tests.test_abi import FAKE, _kv
from tests.test_kv_cache import OnDevice


def scales(scale=FAKE, block=16):
    return ctypes.byref(mla.mla_scales_t(scale, block))


BAD_SCALES = [(None, mla.MLA_ERR_INVALID_ARG), (scales(None), mla.MLA_ERR_INVALID_ARG),
              (scales(FAKE + 2), mla.MLA_ERR_INVALID_ARG), (scales(block=0), mla.MLA_ERR_UNSUPPORTED),
              (scales(block=-16), mla.MLA_ERR_UNSUPPORTED), (scales(block=24), mla.MLA_ERR_UNSUPPORTED),
              (scales(block=128), mla.MLA_ERR_UNSUPPORTED)]


def test_append():
    lib, r = mla.library(), ctypes.byref(mla.mla_rope_init())
    past = mla.mla_rope_axes_init([16, 16])
    past.axis[5] = 2
    ok = dict(kv=ctypes.byref(_kv()), scales=scales(), x=FAKE, stride=576, cu=FAKE, B=2, n=3, weight=FAKE, eps=1e-6,
              rope=r, axes=None, positions=FAKE, status=None)

    def call(**kw):
        return lib.mla_cache_append_scaled(*dict(ok, **kw).values(), None)

    for s, status in BAD_SCALES:
        assert call(scales=s) == status
    for kw in (dict(kv=None), dict(kv=ctypes.byref(_kv(pool=None))), dict(B=-1), dict(n=-1), dict(eps=-1.0),
               dict(eps=float("nan")), dict(rope=None), dict(positions=None), dict(stride=568), dict(stride=580),
               dict(x=None), dict(cu=None), dict(x=FAKE + 8), dict(cu=FAKE + 4), dict(weight=FAKE + 2),
               dict(positions=FAKE + 4), dict(status=FAKE + 1), dict(axes=past),
               dict(axes=mla.mla_rope_axes_init([32]), rope=None, positions=None)):
        assert call(**kw) == mla.MLA_ERR_INVALID_ARG, kw
    assert call(kv=ctypes.byref(_kv(page_size=48))) == call(n=1 << 31) == call(B=1 << 29) == mla.MLA_ERR_UNSUPPORTED
    assert call(n=0, x=None) == 0 and call(B=0, cu=None) == 0
    assert lib.mla_last_launch_count() == 0


def test_gather():
    lib = mla.library()
    ok = dict(kv=ctypes.byref(_kv()), scales=scales(), B=2, starts=None, cu=FAKE, n=5, out=FAKE, f32=0, status=None)

    def call(**kw):
        return lib.mla_cache_gather_scaled(*dict(ok, **kw).values(), None)

    for s, status in BAD_SCALES:
        assert call(scales=s) == status
    for kw in (dict(kv=None), dict(B=-1), dict(cu=None), dict(out=None), dict(out=FAKE + 8), dict(status=FAKE + 1)):
        assert call(**kw) == mla.MLA_ERR_INVALID_ARG, kw
    assert call(n=0, out=None) == 0
    assert lib.mla_last_launch_count() == 0


def cache(scales, page=64, kv_scale=1.0, device=0):
    tensor = OnDevice(torch.zeros(4, page, 576, dtype=torch.uint8))
    return mla.KVCache(tensor, OnDevice(torch.zeros(2, 3, dtype=torch.int32)), OnDevice(torch.zeros(2, dtype=torch.int32)),
                       kv_scale, scales=None if scales is None else OnDevice(scales, device))


@pytest.mark.parametrize("page,width,block", [(64, 64, 1), (64, 1, 64), (64, 4, 16), (128, 2, 64), (192, 6, 32), (192, 96, 2)])
def test_cache_with_scales(page, width, block):
    c = cache(torch.zeros(4, width), page).c_scales()
    assert c.block == block and c.scale
    assert cache(None, page, 0.5).c_scales() is None


@pytest.mark.parametrize("scales", [torch.zeros(4), torch.zeros(3, 4), torch.zeros(4, 3), torch.zeros(4, 0), torch.zeros(4, 4, 1),
                                    torch.zeros(4, 128), torch.zeros(4, 4, dtype=torch.float64), torch.zeros(4, 8)[:, ::2]])
def test_refused_scales(scales):
    with pytest.raises(ValueError, match="scales"):
        cache(scales).c_scales()


def test_other_refusals():
    with pytest.raises(ValueError, match="scales"):
        cache(torch.zeros(4, 1), page=128).c_scales()  # blocks of 128
    with pytest.raises(ValueError, match="kv_scale"):
        cache(torch.zeros(4, 4), kv_scale=0.5).c_scales()
    with pytest.raises(ValueError, match="device"):
        cache(torch.zeros(4, 4), device=1).c_scales()
