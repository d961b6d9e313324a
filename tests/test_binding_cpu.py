"""The Python side of the bindings without a GPU: what the checks refuse."""

import ctypes

import pytest
import torch

from block_sparse_masked_build_gb300 import _lib, api
from block_sparse_masked_build_gb300 import build as bsm_build

BF = torch.bfloat16


def _t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def test_operands():
    q, k = _t(2, 4, 10, 64), _t(2, 2, 12, 64)
    api._check_operands(q, k, k)
    api._check_operands(q, k.view(torch.int16), k.view(torch.uint16))
    api._check_operands(q, _t(3, 2, 12, 64), _t(2, 2, 30, 64))
    for bad in ((q.half(), k, k), (q, k.float(), k), (q, k, k[:, :, :11]),
                (q, k, k[:, :1]), (q, k[:1], k[:1]),
                (q, k[..., :32], k[..., :32]), (q[0], k, k),
                (q.transpose(2, 3), k, k), (q, k.to("meta"), k)):
        with pytest.raises(ValueError):
            api._check_operands(*bad)


def test_outputs():
    q = _t(2, 4, 10, 64)
    api._check_like(None, q, "out")
    api._check_like(_t(2, 4, 20, 64), q, "out")
    for bad in (q.float(), q[:1], q[:, :, :9], q[..., :8], q[0],
                q.to("meta")):
        with pytest.raises(ValueError, match="out must be"):
            api._check_like(bad, q, "out")
    api._check_lse(None, q)
    api._check_lse(_t(8, 10, dtype=torch.float32), q)
    for bad in (_t(8, 10), _t(8, 9, dtype=torch.float32),
                _t(8, 20, dtype=torch.float32)[:, ::2]):
        with pytest.raises(ValueError, match="lse must be"):
            api._check_lse(bad, q)


def test_segment_ids():
    cpu = torch.device("cpu")
    good = _t(2, 10, dtype=torch.int32)
    for t in (None, good, good.view(20), good.view(torch.uint32)):
        api._check_ids(t, 2, 10, cpu, "q_segment_ids")
    for bad in (good.long(), good[:, :9], good[:1], good[:1].expand(2, 10),
                good.to("meta")):
        with pytest.raises(ValueError, match="q_segment_ids must be"):
            api._check_ids(bad, 2, 10, cpu, "q_segment_ids")


@pytest.mark.parametrize("fast", [False, True])
def test_mask_info_inputs(fast, monkeypatch):
    """Ids and mask words that the kernels would read past are refused before
    anything touches a device."""
    if fast and not api._fast():
        pytest.skip("the tensor binding is not built")
    if not fast:
        monkeypatch.setattr(api, "_fast", lambda: False)
        # no GPU: the checks come before the buffer's contents matter
        monkeypatch.setattr(api, "_CUDA", torch.device("cpu"))
    SEG, DN = api.MASK_SEGMENT, api.MASK_DENSE
    good = _t(2, 40, dtype=torch.int32)
    for bad in (good.long(), good[:1], good[:, :39], good[:1].expand(2, 40),
                good[:, ::2]):
        for a, b in ((bad, good), (good, bad)):
            with pytest.raises(ValueError, match="of 80 elements"):
                api.build_mask_info(SEG, 2, 40, 40, q_segment_ids=a,
                                    kv_segment_ids=b)
    words = _t(40, 2, dtype=torch.int32)
    for bad in (words[:39], words[:, :1]):
        with pytest.raises(ValueError, match="Sq rows"):
            api.build_mask_info(DN, 1, 40, 40, dense_bits=bad)
    with pytest.raises(ValueError, match="must be CUDA tensors"):
        api.build_mask_info(SEG, 2, 40, 40, q_segment_ids=good,
                            kv_segment_ids=good)
    with pytest.raises(ValueError, match="on a CUDA device"):
        api.build_mask_info(api.MASK_CAUSAL, 1, 40, 40, device="cpu")


def test_a_module_that_does_not_load_leaves_ctypes(monkeypatch, tmp_path):
    bsm_build.build()
    _lib.lib()
    (tmp_path / "_bsm_torch.so").write_bytes(b"built for another machine")
    monkeypatch.setattr(_lib, "HERE", str(tmp_path))
    monkeypatch.setattr(_lib, "_fast", None)
    with pytest.warns(RuntimeWarning, match="does not load"):
        assert _lib.fast(api._check) is False
    assert _lib.fast(api._check) is False  # without another attempt


def test_an_older_library_is_named(monkeypatch):
    bsm_build.build()
    none = ctypes.CDLL(None)  # has none of the entry points
    monkeypatch.setattr(_lib, "_lib", None)
    monkeypatch.setattr(_lib.ctypes, "CDLL", lambda path: none)
    with pytest.raises(RuntimeError, match="rebuild the library"):
        _lib.lib()
