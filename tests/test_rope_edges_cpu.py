"""Rotations without a GPU: copies of a Rope."""

import copy
import ctypes
import gc
import pickle

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
