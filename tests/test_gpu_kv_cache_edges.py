"""The paged cache at its edges: error records beside others."""

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import kv_cache_ref as ref

pytestmark = pytest.mark.gpu


def test_a_bad_page_beside_a_timeout_is_reported_too():
    """Each status call reports one of two pending records; the append that
    left tokens unwritten is not forgotten for the timeout's sake."""
    assert bsm.bsm_device_status()[0] == 0
    page, D = 16, 64
    cache = bsm.KVCache(*[t.cuda() for t in ref.random_cache(4, 1, page, D, 1)])
    table = torch.tensor([[99]], dtype=torch.int32).cuda()  # no such page
    lens = torch.zeros(1, dtype=torch.int32).cuda()
    x = torch.ones(1, 1, 2, D, dtype=torch.bfloat16).cuda()
    bsm.kv_append(cache, table, lens, x, x)
    bsm.bsm_selftest_wait_timeout(1_000_000)  # 1 ms, nothing ever arrives
    st, detail = bsm.bsm_device_status()
    assert st == -4 and detail[0] == 1
    st, detail = bsm.bsm_device_status()
    assert st == -1 and detail == [2, 0, 0, 99]
    assert bsm.bsm_device_status()[0] == 0
