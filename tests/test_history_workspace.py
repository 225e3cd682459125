"""Workspace sizes of the attention over a 16-bit cache: a size that a program was
given once goes on being enough (no GPU needed)."""
import pytest

import sparse_dense_interaction_gb300 as sdi

# (sequences, new tokens, query heads, kv heads, head width, most new, longest), bytes that were enough
ENOUGH = [
    ((5, 2800, 8, 8, 192, 560, 4856), 11279632),
    ((6, 11820, 2, 1, 136, 2224, 4119), 8011024),
    ((27, 1674, 8, 4, 200, 76, 3683), 11746576),
    ((2, 830, 16, 8, 160, 827, 3787), 9411856),
    ((53, 6148, 2, 2, 200, 140, 3659), 11746576),
    ((2, 4226, 2, 1, 256, 2725, 7450), 26065984),
    ((46, 3312, 4, 1, 192, 186, 24832), 40909840),
    ((13, 2249, 8, 2, 256, 260, 7419), 36991568),
    ((64, 64, 16, 4, 256, 1, 2000), 5263376),
    ((1, 1, 16, 4, 256, 1, 262143), 3764752),
    ((4, 8192, 16, 4, 128, 2048, 8192), 7544080),
    ((64, 6400, 8, 8, 64, 200, 2000), 3808528),
    ((256, 256, 16, 4, 128, 1, 8192), 4227088),
]


@pytest.mark.parametrize("sizes,enough", ENOUGH)
def test_workspace_sizes_do_not_grow(sizes, enough):
    assert 0 < sdi.dlrm_kv_attn_workspace_size(*sizes) <= enough
    # the cache in 8 bits has kernels of its own, which may want more
    assert sdi.dlrm_kv8_attn_workspace_size(*sizes) >= sdi.dlrm_kv_attn_workspace_size(*sizes)
