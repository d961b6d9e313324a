"""Rotations without a GPU: copies of a Rope, and the turns it holds."""

import copy
import ctypes
import gc
import pickle
from decimal import Decimal, localcontext

import pytest

import block_sparse_masked_build_gb300 as bsm
from block_sparse_masked_build_gb300 import api
from block_sparse_masked_build_gb300._lib import RopeStruct


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
