"""What KVCache accepts, without a GPU: its tensors are stood in for by CPU ones that say they are on
a device. The library reads rows of 576 codes wherever the pool's shape says pages begin."""
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla


class OnDevice:
    """A tensor as KVCache looks at it, on device 0."""

    is_cuda = True

    def __init__(self, t, device=0):
        self.t, self.device_index = t, device

    def get_device(self):
        return self.device_index

    def __getattr__(self, name):
        return getattr(self.t, name)


def cache(pool=(4, 64, 576), table=(2, 3), dtype=torch.uint8, device=0, kv_scale=0.5):
    return mla.KVCache(OnDevice(torch.zeros(pool, dtype=dtype)), OnDevice(torch.zeros(table, dtype=torch.int32)),
                       OnDevice(torch.zeros(table[0], dtype=torch.int32), device), kv_scale)


@pytest.mark.parametrize("pool,pages,size", [((4, 64, 576), 4, 64), ((5, 128, 1, 576), 5, 128), ((0, 64, 576), 0, 64),
                                             ((3, 192, 9, 64), 3, 192)])
def test_accepted(pool, pages, size):
    """Rows of 576 codes in one dimension or more."""
    c = cache(pool).c_struct()
    assert (c.num_pages, c.page_size, c.page_table_stride, c.kv_scale) == (pages, size, 3, 0.5)


@pytest.mark.parametrize("pool", [(4, 64, 512), (4, 64, 640), (4, 64), (4, 64 * 576), (576,), (4, 64, 1, 288), (4, 64, 0)])
def test_pools_of_another_width(pool):
    with pytest.raises(ValueError, match="pool"):
        cache(pool).c_struct()


def test_other_refusals():
    assert cache(table=(2, 3, 1)).c_struct().page_table_stride == 3
    with pytest.raises(ValueError, match="page_table"):
        cache(table=(2, 3, 2)).c_struct()
    with pytest.raises(ValueError, match="page_table"):
        cache(table=(6,)).c_struct()
    with pytest.raises(TypeError):
        cache(dtype=torch.int8).c_struct()
    with pytest.raises(ValueError, match="one device"):
        cache(device=1).c_struct()


@pytest.mark.parametrize("scale", [0.25, 1, torch.tensor(0.5), "0.125"])
def test_scales(scale):
    """Whatever float() takes."""
    assert cache(kv_scale=scale).c_struct().kv_scale == float(scale)
