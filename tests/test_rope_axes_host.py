"""mla_rope_axes_init against its definition, and the refusals of the calls that take axes, without a GPU."""
import ctypes

import pytest

import mla_latent_kv_attention_gb300 as mla
from tests.test_abi import FAKE


def in_turn(sections):
    """The axes in turn, each while it has pairs left."""
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


@pytest.mark.parametrize("sections", [[32], [8, 12, 12], [12, 10, 10], [16, 16], [0, 32], [32, 0, 0, 0], [1, 2, 3, 26],
                                      [29, 1, 1, 1], [0, 5, 0, 27]])
def test_assignments(sections):
    axes = mla.mla_rope_axes_init(sections)
    assert axes.n_axes == len(sections)
    assert list(axes.axis) == [a for a, k in enumerate(sections) for _ in range(k)]
    assert list(mla.mla_rope_axes_init(sections, interleaved=True).axis) == in_turn(sections)


@pytest.mark.parametrize("sections", [[], [31], [33], [16, 17], [40, -8], [8] * 5, [2 ** 31 - 1, 1], [16, 16, 0, 0, 0],
                                      [2 ** 32 + 16, 16], [16, 16 - 2 ** 32]])
def test_init_refusals(sections):
    with pytest.raises(mla.MlaError) as e:
        mla.mla_rope_axes_init(sections)
    assert e.value.status == mla.MLA_ERR_INVALID_ARG


def test_init_leaves_a_refused_struct():
    lib = mla.library()
    axes = mla.mla_rope_axes_init([32])
    bad = (ctypes.c_int32 * 2)(30, 3)
    assert lib.mla_rope_axes_init(axes, bad, 2, 0) == mla.MLA_ERR_INVALID_ARG
    assert axes.n_axes == 1 and list(axes.axis) == [0] * 32
    assert lib.mla_rope_axes_init(None, bad, 2, 0) == lib.mla_rope_axes_init(axes, None, 2, 0) == mla.MLA_ERR_INVALID_ARG


def bad_axes():
    past = mla.mla_rope_axes_init([16, 16])
    past.axis[31] = 2
    none, many = mla.mla_rope_axes_init([32]), mla.mla_rope_axes_init([32])
    none.n_axes, many.n_axes = 0, 5
    return [None, past, none, many]


def test_rope_refusals():
    lib, r = mla.library(), ctypes.byref(mla.mla_rope_init())
    ok = dict(rope=r, axes=mla.mla_rope_axes_init([8, 12, 12]), x=FAKE, xt=768, xh=64, positions=FAKE, n=3, H=12,
              out=FAKE, ot=768, oh=64)

    def call(**kw):
        return lib.mla_rope_axes(*dict(ok, **kw).values(), None)

    for axes in bad_axes():
        assert call(axes=axes) == call(axes=axes, n=0) == mla.MLA_ERR_INVALID_ARG
    for kw in (dict(rope=None), dict(x=None), dict(out=None), dict(positions=None), dict(n=-1), dict(H=-1),
               dict(x=FAKE + 8), dict(out=FAKE + 2), dict(positions=FAKE + 4), dict(xt=65), dict(oh=-7)):
        assert call(**kw) == mla.MLA_ERR_INVALID_ARG, kw
    assert call(n=1 << 41, H=1) == mla.MLA_ERR_UNSUPPORTED
    assert call(n=0) == 0 and call(H=0) == 0
    assert lib.mla_last_launch_count() == 0


def test_append_rope_refusals():
    lib, r = mla.library(), ctypes.byref(mla.mla_rope_init())
    ok = dict(pool=FAKE, pages=4, page_size=64, x=FAKE, stride=576, slots=FAKE, n=3, kv_scale=0.5,
              weight=FAKE, eps=1e-6, rope=r, axes=mla.mla_rope_axes_init([8, 12, 12]), positions=FAKE, status=None)

    def call(**kw):
        return lib.mla_cache_append_rope_axes(*dict(ok, **kw).values(), None)

    for axes in bad_axes():
        assert call(axes=axes) == mla.MLA_ERR_INVALID_ARG
    for kw in (dict(n=-1), dict(kv_scale=0.0), dict(eps=-1.0), dict(rope=None), dict(positions=None),
               dict(rope=None, positions=None), dict(stride=568), dict(x=None), dict(positions=FAKE + 4)):
        assert call(**kw) == mla.MLA_ERR_INVALID_ARG, kw
    assert call(n=0, x=None, slots=None) == 0
    assert lib.mla_last_launch_count() == 0
