"""mla_rope_init's whole-number frequencies, without a GPU."""
import pytest

import mla_latent_kv_attention_gb300 as mla


@pytest.mark.parametrize("kw", [dict(factor=1e-320), dict(factor=5e-324, original_positions=4096)])
def test_stretches_past_float64_are_refused(kw):
    """f / factor overflows: no number of turns."""
    with pytest.raises(mla.MlaError) as e:
        mla.mla_rope_init(**kw)
    assert e.value.status == mla.MLA_ERR_INVALID_ARG
