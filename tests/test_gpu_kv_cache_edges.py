"""The paged cache at its edges: error records beside others, scales at the
ends of their range, many sequences.  Tolerances as in test_gpu_kv_cache."""

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import kv_cache_ref as ref
from test_gpu_kv_cache import _attend, check, status

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


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("D", [64, 128])
def test_key_and_value_scales_at_the_ends_of_their_range(D, T):
    """2^-40 and 2^40 side by side: logits that a cap holds, and values whose
    largest outweigh the others by 2^80."""
    lens, page = [400, 77, 16], 16
    k, v, ks, vs = ref.random_cache(40, 2, page, D, 7, spread=0, centre=0)
    g = torch.Generator().manual_seed(8)
    for s in (ks, vs):
        s.copy_(torch.where(torch.rand(s.shape, generator=g) < 0.5,
                            2.0 ** -40, 2.0 ** 40))
    vs[::3] = 1.0
    table = ref.random_table(lens, page, 26, 40, 9)
    out, lse, want = _attend(lens, page, D, 2, 3, T, 10, softcap=6.0,
                             host=(k, v, ks, vs), table=table)
    assert status()[0] == 0
    check(out, lse, want)


@pytest.mark.parametrize("T", [1, 3])
def test_many_more_sequences_than_ctas(T):
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 70, (3000,), generator=g).tolist()
    out, lse, want = _attend(lens, 16, 64, 1, 2, T, 12, softcap=9.0)
    assert status()[0] == 0
    check(out, lse, want)
