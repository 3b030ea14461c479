"""mla_cache_append_scaled with an empty x: sequences that say they have new rows are reported, as those with
rows outside any other x are; nothing is written."""
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("block", [1, 2, 16, 64])
@pytest.mark.parametrize("cu,want", [([0, 0, 0, 0], 0), ([0, 1, 1, 4], mla.MLA_ERR_BOUNDS), ([0, 0, 0, 1], mla.MLA_ERR_BOUNDS)])
def test_empty_x(cu, want, block, turned):
    g = torch.Generator().manual_seed(1)
    pool = torch.randint(0, 255, (3, 64, 576), dtype=torch.uint8, generator=g).to(DEV)
    scales = torch.ones(3, 64 // block, device=DEV)
    kv = mla.KVCache(pool, torch.arange(3, dtype=torch.int32, device=DEV).view(3, 1),
                     torch.tensor([5, 0, 64], dtype=torch.int32, device=DEV), 1.0, scales=scales)
    before = pool.clone()
    x = torch.zeros(0, 576, dtype=torch.bfloat16, device=DEV)
    rope = dict(rope=mla.mla_rope_init(), positions=torch.zeros(0, dtype=torch.int64, device=DEV)) if turned else {}
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.mla_cache_append_scaled(kv, x, torch.tensor(cu, device=DEV), status=status, **rope)
    assert int(status) == want and mla.mla_last_launch_count() == 1
    mla.mla_cache_append_scaled(kv, x, torch.tensor(cu, device=DEV), **rope)  # (nowhere to report to)
    assert mla.mla_last_launch_count() == 0
    assert torch.equal(pool, before) and bool((scales == 1).all())


def test_no_sequences():
    kv = mla.KVCache(torch.zeros(1, 64, 576, dtype=torch.uint8, device=DEV), torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                     torch.zeros(1, dtype=torch.int32, device=DEV), 1.0, scales=torch.ones(1, 4, device=DEV))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mla.mla_cache_append_scaled(kv, torch.zeros(3, 576, dtype=torch.bfloat16, device=DEV), torch.tensor([0], device=DEV),
                                status=status)
    assert int(status) == 0 and mla.mla_last_launch_count() == 0
