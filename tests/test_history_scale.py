"""The attention's scale: what it is multiplied by inside must leave it finite."""
import pytest

import sparse_dense_interaction_gb300 as sdi
from tests.test_history_abi import BAD, FAKE, OK, _nothing_is_launched, batch, cache, heads, lib, ref  # noqa: F401


@pytest.mark.parametrize("scale,want", [(2.5e38, BAD), (3.0e38, BAD), (3.4e38, BAD), (2.0e38, OK), (1e-38, OK)])
def test_scale_times_log2_e_is_finite(lib, scale, want):  # noqa: F811
    need = sdi.dlrm_kv_attn_workspace_size(2, 0, 8, 4, 64, 4, 60)
    assert lib.dlrm_kv_attn_fwd(ref(heads(n=8)), ref(batch(n=0)), ref(cache()), 64, 2, scale, 1, 0, 4, 60, ref(heads(n=8)),
                                None, FAKE, need, None, None) == want
