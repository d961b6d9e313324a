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
