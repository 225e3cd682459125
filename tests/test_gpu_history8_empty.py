"""Rows that see nothing, in 8 bits, by the thousand: zeros and -infinity in every
kernel, whatever lies beside them."""
import numpy as np
import pytest
import torch

import sparse_dense_interaction_gb300 as sdi
from tests.test_gpu_history8 import DEV, DT, as64, cache8, flag, randn, tensors8
from tests.test_gpu_history8_edges import _built  # noqa: F401

pytestmark = pytest.mark.gpu


# (new tokens of each, q heads, kv heads, d, dtype): single events; one and two query tiles; wide heads; fp32; chunks
# whose codes are converted; the general kernel
@pytest.mark.parametrize("new,hq,hk,d,dtype", [
    (1, 8, 2, 64, "f16"), (3, 8, 2, 128, "bf16"), (200, 8, 8, 64, "f16"), (200, 8, 8, 64, "bf16"), (120, 8, 2, 64, "bf16"),
    (120, 8, 2, 64, "f16"), (70, 8, 2, 128, "bf16"), (70, 8, 2, 128, "f16"), (40, 4, 1, 96, "bf16"), (50, 8, 2, 256, "bf16"),
    (50, 8, 2, 256, "f16"), (20, 4, 2, 64, "f32"), (400, 8, 2, 128, "bf16"), (600, 8, 2, 64, "f16"), (30, 4, 2, 20, "bf16"),
])
@pytest.mark.parametrize("causal", [False, True])
def test_users_without_a_history(new, hq, hk, d, dtype, causal):
    # all but every eighth user have none; with `causal` those have 3 events, so that most of their rows see nothing too
    S, page = 64, 16
    lengths = [(3 if causal else 70) if s % 8 == 0 else 0 for s in range(S)]
    n, table = S * new, torch.full((S, 5), -1, dtype=torch.int32, device=DEV)
    table[::8] = torch.arange(40, dtype=torch.int32, device=DEV).view(8, 5)
    (kc, ke), (vc, ve) = (tensors8(*cache8(s, 40, page, 8, hk, d)) for s in (61, 62))
    q = randn(63, (n, hq, d), dtype)
    sees = torch.tensor([not causal and length > 0 or causal and i >= new - length for length in lengths
                         for i in range(new)], device=DEV)
    sizes = (S, n, hq, hk, d, new, max(lengths))
    ws = torch.full((sdi.dlrm_kv8_attn_workspace_size(*sizes),), 255, dtype=torch.uint8, device=DEV)
    first = None
    for _ in range(5):
        out, lse, f = torch.full((n, hq, d), 7, dtype=DT[dtype], device=DEV), torch.full((n, hq), 7.0, device=DEV), flag()
        sdi.dlrm_kv8_attn_fwd(q, as64(np.arange(S + 1) * new), as64(lengths), table, kc, vc, ke, ve, out, d ** -0.5, ws,
                              new, max(lengths), causal=causal, lse=lse, err_flag=f)
        assert sdi.dlrm_read_error(f) == 0
        assert (out[~sees] == 0).all() and torch.isneginf(lse[~sees]).all()
        assert torch.isfinite(out).all() and torch.isfinite(lse[sees]).all() and out[sees].abs().sum() > 0
        first = first if first is not None else out
        assert torch.equal(out, first)
