"""The profiling hook on a cache with block scales: a traced call writes its own stamps (those of a call before
are gone), with the outputs of an untraced one."""
import numpy as np
import pytest
import torch

import mla_latent_kv_attention_gb300 as mla
from mla_latent_kv_attention_gb300 import workloads as W
from tests.test_scaled_attention_gpu import DEV, cache, queries
from tests.test_trace_gpu import WORDS

pytestmark = pytest.mark.gpu
LENS = [5000, 300, 12000, 0, 77]


def traced(call, tiles):
    """call() twice, the second time with the hook on a buffer of old stamps; the tiles it has to count."""
    want = call()
    torch.cuda.synchronize()
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    buffer = torch.full((ctas * WORDS,), 7, dtype=torch.int64, device=DEV)
    lib = mla.library()
    lib.mla_set_trace_buffer(buffer.data_ptr(), buffer.numel() * 8)
    try:
        got = call()
        torch.cuda.synchronize()
    finally:
        lib.mla_set_trace_buffer(None, 0)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    t = buffer.view(ctas, WORDS).cpu().numpy()
    for a, b in ((0, 1), (1, 2), (2, 7)):
        assert np.all(t[:, a] > 7) and np.all(t[:, a] <= t[:, b]), (a, b)
    worked = t[:, 3] != 7  # (a CTA without a tile leaves these words)
    assert worked.any()
    assert np.all(t[worked, 2] <= t[worked, 3]) and np.all(t[worked, 6] <= t[worked, 7])
    assert int((t[worked, 8] >> 32).sum()) >= tiles


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,H", [(1, 12), (2, 12), (4, 12), (4, 16)])
def test_decode_and_verify(n, H, f32):
    kv = cache(LENS, 16, n)
    q = queries(n, len(LENS), n, H)
    call = mla.mla_verify_f32 if f32 else mla.mla_verify
    traced(lambda: call(kv, q, W.SM_SCALE), sum(-(-L // 128) for L in LENS))


def test_prefill():
    T, L, H = 700, 1500, 12
    kv = cache([L], 16, 3)
    q = queries(3, T, H)
    units = -(-T // 4)
    full = units - units % torch.cuda.get_device_properties(0).multi_processor_count
    traced(lambda: mla.mla_prefill(kv, q, W.SM_SCALE), full * ((L - T) // 128))


def test_trees_leave_the_buffer():
    kv = cache(LENS, 16, 5)
    q = queries(5, len(LENS), 3, 12)
    mask = torch.tensor([[1, 3, 5]] * len(LENS), device=DEV)
    buffer = torch.full((1024 * WORDS,), 7, dtype=torch.int64, device=DEV)
    mla.library().mla_set_trace_buffer(buffer.data_ptr(), buffer.numel() * 8)
    try:
        mla.mla_verify_tree(kv, q, mask, W.SM_SCALE)
        torch.cuda.synchronize()
    finally:
        mla.library().mla_set_trace_buffer(None, 0)
    assert bool((buffer == 7).all())
