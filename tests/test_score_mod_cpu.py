"""Modified softmax scores, without a GPU: the refusals of the entry points
and the fp64 reference's own gradients."""

import ctypes
import math

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import score_mod_ref as ref
from block_sparse_masked_build_gb300 import _lib
from block_sparse_masked_build_gb300 import build as bsm_build
from block_sparse_masked_build_gb300._lib import (I64x3, MaskInfoStruct,
                                                  ScoreMod, TensorView)

INVALID = _lib.BSM_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    bsm_build.build()
    return _lib.lib()


def _info():
    i = MaskInfoStruct()
    i.flags, i.window, i.num_tables = 1, 0, 1
    i.Sq = i.Skv = 256
    i.block_q = i.block_kv = 128
    i.nq = i.nk = 2
    i.num_super = 1
    i.block_mask = 0x50000
    return i


def _fwd(lib, mod, scale=0.125, score=0, B=1):
    s = I64x3(2 * 256 * 128, 256 * 128, 128)
    return lib.bsm_splash_fwd_mod(
        0x10000, 0x20000, 0x30000, s, s, s, s, B, 2, 2, 256, 256, 128,
        ctypes.byref(_info()), None, None, scale, score,
        None if mod is None else ctypes.byref(mod), 0x40000, None, 0x70000,
        256 + 256 * 2 * 3 * 2048 * 2, None)


def _bwd(lib, mod, scale=0.125, score=0, B=1):
    t = TensorView(0x10000, I64x3(2 * 256 * 128, 256 * 128, 128))
    r = ctypes.byref(t)
    return lib.bsm_splash_bwd_mod(
        r, r, r, r, 0x60000, r, B, 2, 2, 256, 256, 128,
        ctypes.byref(_info()), None, None, scale, score,
        None if mod is None else ctypes.byref(mod), r, r, r, 0x70000, 1 << 20,
        None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_mod_refusals(lib, call):
    # every refusal comes before anything touches the device
    for cap in (-1.0, float("nan"), float("inf"), float("-inf")):
        assert call(lib, ScoreMod(cap, None)) == INVALID
        assert "softcap" in _lib.last_error()
    assert call(lib, ScoreMod(1e-30, None), scale=1e20) == INVALID
    assert "softcap" in _lib.last_error()
    assert call(lib, ScoreMod(3e38, None)) == INVALID
    assert call(lib, ScoreMod(5.0, None), score=1) == INVALID
    assert "softmax" in _lib.last_error()
    assert call(lib, ScoreMod(0.0, 0x1000), score=1) == INVALID
    assert call(lib, ScoreMod(0.0, 0x1002)) == INVALID
    assert "aligned" in _lib.last_error()


def test_empty_input_is_a_no_op(lib):
    assert _fwd(lib, ScoreMod(5.0, 0x1000), B=0) == 0
    assert _bwd(lib, ScoreMod(5.0, 0x1000), B=0) == 0


def test_slopes_are_checked():
    from block_sparse_masked_build_gb300.api import _score_mod
    cpu = torch.device("cpu")
    assert _score_mod(0.0, None, 4, cpu) is None
    assert _score_mod(30.0, None, 4, cpu).softcap == 30.0
    good = torch.zeros(4)
    assert _score_mod(0.0, good, 4, cpu).alibi_slopes == good.data_ptr()
    for bad in (torch.zeros(3), torch.zeros(4, dtype=torch.float64),
                torch.zeros(4, 1), torch.zeros(8)[::2],
                torch.zeros(4, device="meta")):
        with pytest.raises(ValueError, match="alibi_slopes"):
            _score_mod(0.0, bad, 4, cpu)


@pytest.mark.parametrize("softcap,biased", [(0.0, False), (3.0, False),
                                            (0.0, True), (3.0, True)])
def test_reference_gradients(softcap, biased):
    # the formulas against automatic differentiation and central differences
    g = torch.Generator().manual_seed(5)
    q = torch.randn(1, 4, 9, 8, generator=g).double()
    k = torch.randn(1, 2, 7, 8, generator=g).double()
    v = torch.randn(1, 2, 7, 8, generator=g).double()
    do = torch.randn(1, 4, 9, 8, generator=g).double()
    slopes = torch.tensor([0.5, 0.25, 0.125, -0.1]) if biased else None
    vis = ref.visible(bsm.MASK_CAUSAL, 0, 9, 7, 1)
    got = ref.backward(q, k, v, do, vis, 0.7, softcap, slopes)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    out = ref.forward(*leaves, vis, 0.7, softcap, slopes)[0]
    auto = torch.autograd.grad(out, leaves, do)
    for a, b in zip(got, auto):
        torch.testing.assert_close(a, b, rtol=1e-9, atol=1e-11)
    for n in range(3):
        u = torch.randn((q, k, v)[n].shape, generator=g).double()
        h, f = 1e-5, []
        for sign in (1, -1):
            x = [q, k, v]
            x[n] = x[n] + sign * h * u
            f.append((ref.forward(*x, vis, 0.7, softcap, slopes)[0]
                      * do).sum())
        diff = (f[0] - f[1]) / (2 * h)
        # third-order term h^2 and cancellation 2^-52 / h, both below 1e-8
        assert math.isclose(float((got[n] * u).sum()), float(diff),
                            rel_tol=1e-6, abs_tol=1e-7)
