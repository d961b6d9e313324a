"""Rotations without a GPU: copies of a Rope, the turns it holds, what it refuses,
and results in place of their inputs."""

import copy
import ctypes
import gc
import pickle
from decimal import Decimal, localcontext

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
from block_sparse_masked_build_gb300 import _lib, api
from block_sparse_masked_build_gb300._lib import I64x3, RopeStruct, TensorView


@pytest.mark.parametrize("again", [
    copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))])
def test_copies_stand_alone(again):
    """The table that a copy's calls read is the copy's own, also when the Rope
    that it was made from is gone."""
    rope = bsm.Rope(64, 1e6, axes=[0, 1] * 16, interleaved=True)
    want = bytes(rope._struct)
    other = again(rope)
    del rope
    gc.collect()
    assert (other.dim, other.axes, other.interleaved) == (64, 2, True)
    at = api._rope_address(other)
    assert at == ctypes.addressof(other._struct)
    assert bytes(RopeStruct.from_address(at)) == want


# 1 / (2 pi) to 79 digits
INV_TURN = Decimal("0.1591549430918953357688837633725143620344596457404564"
                   "48747667344058896797634226535")


@pytest.mark.parametrize("freq", [
    1.0, -1.0, 0.8058421877614819, 63.7, 64.0, -63.9, 0.5, 1e-7, -1e-7, 2.0 ** -70,
    -2.0 ** -70, 0.0, 6.283185307179586, 50.26548245743669, 1e4 ** (-62 / 64)])
def test_steps_to_their_last_bit(freq):
    """Turns per position in units of 2^-64, rounded to the nearest: what
    keeps far positions' angles (2^31 times half a unit is 2^-34 turns)."""
    with localcontext() as c:
        c.prec = 100
        want = Decimal(freq) * INV_TURN * 2 ** 64
        got = bsm.Rope(16, inv_freq=[freq] * 8)._struct.step[3]
        off = abs((Decimal(got) - want) % 2 ** 64)
        off = min(off, 2 ** 64 - off)
    assert off <= Decimal("0.5001"), off


def _view(data, *strides):
    return ctypes.byref(TensorView(data, I64x3(*strides)))


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("backward", [False, True])
def test_in_place_needs_the_inputs_strides(which, backward):
    """Rows written over an input that lies otherwise in the same memory would
    be read again."""
    lib = _lib.lib()
    rope = bsm.Rope(64)._struct
    # [B, S, H, D] and [B, H, S, D] in one memory; the others apart
    a, b = (4096, 64, 512), (4096, 512, 64)
    kw = dict(q=_view(0x500000, *a), qo=_view(0x600000, *a),
              k=_view(0x700000, *a), ko=_view(0x800000, *a))
    kw[which] = _view(0x900000, *a)
    kw[which + "o"] = _view(0x900000, *b)

    def call(B=2, H=8, S=8):
        more = (B, H, H, S, 64, None, rope, None)
        if backward:
            return lib.bsm_norm_rope_bwd(
                kw["q"], kw["k"], None, None, *more, kw["qo"], kw["ko"], None,
                None, None, 0, None)
        return lib.bsm_norm_rope(kw["q"], kw["k"], *more, kw["qo"], kw["ko"],
                                 None)

    assert call() == _lib.BSM_ERR_INVALID_ARG
    assert "strides" in _lib.last_error() and "in place" in _lib.last_error()
    kw[which + "o"] = _view(0x900000, 4096, 64, 1024)
    assert call() == _lib.BSM_ERR_INVALID_ARG and "place" in _lib.last_error()
    assert call(S=0) == 0


@pytest.mark.parametrize("args", [
    dict(dim=1 << 40), dict(dim=-64), dict(dim=0), dict(dim=144),
    dict(dim=64.5), dict(dim=64, axes=[0.5] * 32),
    dict(dim=64, axes=[0, 1.25] * 16), dict(dim=64, axes=[1 << 32] * 32),
    dict(dim=64, axes=[-1] * 32)])
def test_sizes_and_axes_that_are_none(args):
    """Refused before anything of that size is made, and not cut to whole
    numbers."""
    with pytest.raises((ValueError, bsm.BsmError)):
        bsm.Rope(**args)


def test_whole_numbers_of_any_type():
    r = bsm.Rope(64.0, axes=torch.tensor([0.0, 1.0] * 16))
    assert (r.dim, r.axes) == (64, 2)
    assert bytes(r._struct) == bytes(bsm.Rope(64, axes=[0, 1] * 16)._struct)
