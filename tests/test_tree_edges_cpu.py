"""The entry points of drafted trees without a GPU, further on."""

import pytest

from block_sparse_masked_build_gb300 import _lib
from block_sparse_masked_build_gb300 import build as bsm_build


@pytest.fixture(scope="module")
def lib():
    bsm_build.build()
    return _lib.lib()


def test_selftest_limits(lib):
    for limit in (10, 10 ** 12, -1):
        assert lib.bsm_selftest_tree_timeout(limit, None) == \
            _lib.BSM_ERR_INVALID_ARG


@pytest.mark.parametrize("H,Hkv,T,D,want", [
    # two parts of rows x (D + 2) f32 for each of 160 SMs above 16 rows per K/V
    # head (128 or 256 rows); up to there the kernel of few rows'
    (8, 2, 5, 128, 160 * 2 * 128 * 130 * 4),
    (32, 1, 4, 64, 160 * 2 * 128 * 66 * 4),
    (8, 2, 33, 128, 160 * 2 * 256 * 130 * 4),
    (64, 1, 1024, 64, 160 * 2 * 256 * 66 * 4),
    (8, 2, 4, 128, None), (8, 2, 0, 64, None), (0, 2, 9, 64, None),
    (-8, 2, 4, 128, 0), (8, 0, 4, 128, 0), (8, -1, 4, 128, 0),
    (8, 2, -1, 128, 0)])
def test_workspace_bytes(lib, H, Hkv, T, D, want):
    if want is None:
        want = lib.bsm_paged_attention_workspace_bytes()
    assert lib.bsm_paged_attention_tree_workspace_bytes(H, Hkv, T, D) == want
