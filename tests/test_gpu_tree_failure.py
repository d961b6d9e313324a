"""The bounded waits of the drafted trees' kernel: its roles, whose work is not
dealt out, give up after a short limit, return and leave a record; the context
and the kernel stay usable."""

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
from block_sparse_masked_build_gb300 import _lib
from test_gpu_kv_cache import check, status
from test_gpu_tree import CASES, _case, _ints, _run, _want

pytestmark = pytest.mark.gpu

LIMIT = 1_000_000  # 1 ms


def _is_the_trees(detail):
    # block 0; loader, MMA, converter or score, for its first step
    return detail[0] == 1 and detail[1] == 0 and detail[2] in (2, 3, 4, 5) \
        and detail[3] == 9


def test_roles_give_up_and_report():
    assert status()[0] == 0
    for stream in (None, torch.cuda.Stream()):
        bsm.bsm_selftest_tree_timeout(LIMIT, stream)
        st, detail = status()
        assert st == _lib.BSM_ERR_DEVICE_TIMEOUT and _is_the_trees(detail)
        assert status()[0] == 0  # read once
    for case in (CASES[9], CASES[10]):  # two tiles, one
        d = _case(*case)
        check(*_run(d), _want(d))
    assert status()[0] == 0


def test_no_record_is_lost():
    """Each call of bsm_device_status reports one: timeouts, then what was out
    of range."""
    d = _case(64, 128, 8, 2, 40, [300, 200], [40, 40], 0, 0.0, False, True)
    cache = bsm.KVCache(*[t.cuda() for t in d["host"]])
    bsm.paged_attention(d["q"].cuda(), cache, d["table"].cuda(),
                        _ints([300, -5]), n_new=_ints([40, 0]))
    bsm.bsm_selftest_tree_timeout(LIMIT)
    bsm.bsm_selftest_wait_timeout(LIMIT)
    seen = [status() for _ in range(4)]
    timeout = _lib.BSM_ERR_DEVICE_TIMEOUT
    assert [s for s, _ in seen] == [timeout, timeout,
                                    _lib.BSM_ERR_INVALID_ARG, 0]
    assert seen[0][1][3] == 7 and _is_the_trees(seen[1][1])
    assert seen[2][1] == [2, 1, -1, -5]
