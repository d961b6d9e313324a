"""The paged 8-bit cache without a GPU: refusals of its entry points, and the
fp64 reference's rounding."""

import ctypes

import numpy as np
import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import kv_cache_ref as ref
from block_sparse_masked_build_gb300 import _lib
from block_sparse_masked_build_gb300 import build as bsm_build
from block_sparse_masked_build_gb300._lib import (I64x3, KVCacheStruct,
                                                  ScoreMod, TensorView)

INVALID, UNSUPPORTED = _lib.BSM_ERR_INVALID_ARG, _lib.BSM_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    bsm_build.build()
    return _lib.lib()


def _cache(**kw):
    d = dict(k=0x100000, v=0x200000, k_scale=0x300000, v_scale=0x400000,
             num_pages=8, H_kv=2, page_size=64, D=128)
    d.update(kw)
    return KVCacheStruct(*[d[n] for n, _ in KVCacheStruct._fields_])


def _view(data=0x500000, strides=(4 * 128, 128, 128)):
    return ctypes.byref(TensorView(data, I64x3(*strides)))


def _append(lib, cache=None, table=0x600000, stride=4, max_pages=4,
            lens=0x700000, n_new=None, k=None, v=None, B=2, T=2, **kw):
    c = _cache(**kw) if cache is None else cache
    return lib.bsm_kv_append(
        None if c == "null" else ctypes.byref(c), table, stride, max_pages,
        lens, n_new, _view() if k is None else k, _view() if v is None else v,
        B, T, None)


def _attend(lib, table=0x600000, stride=4, max_pages=4, lens=0x700000,
            q=None, out=None, lse=None, B=2, H=4, T=2, scale=0.1, window=0,
            mod=None, ws=0x900000, wsb=None, **kw):
    if wsb is None:
        wsb = 1 << 40
    return lib.bsm_paged_attention(
        _view() if q is None else q, ctypes.byref(_cache(**kw)), table,
        stride, max_pages, lens, B, H, T, scale, window,
        None if mod is None else ctypes.byref(mod),
        _view(0x800000) if out is None else out, lse, ws, wsb, None)


@pytest.mark.parametrize("call", [_append, _attend])
def test_shared_refusals(lib, call):
    # found before anything touches the device
    assert call(lib, D=96) == UNSUPPORTED
    assert call(lib, page_size=48) == UNSUPPORTED
    assert call(lib, page_size=256) == UNSUPPORTED
    assert call(lib, num_pages=-1) == INVALID
    assert call(lib, B=-1) == INVALID
    assert call(lib, T=-1) == INVALID
    assert call(lib, max_pages=-1) == INVALID
    assert call(lib, stride=3) == INVALID
    assert "table_stride" in _lib.last_error()
    assert call(lib, B=70000) == UNSUPPORTED
    assert call(lib, max_pages=1 << 25, stride=1 << 25) == UNSUPPORTED
    assert call(lib, lens=None) == INVALID
    assert call(lib, lens=0x700002) == INVALID
    assert call(lib, table=None) == INVALID
    assert call(lib, table=0x600001) == INVALID
    assert call(lib, k_scale=None) == INVALID
    assert call(lib, v_scale=0x400002) == INVALID
    for n in ("v",):
        assert call(lib, **{"num_pages": 8, "H_kv": 2}, D=128,
                    page_size=64, v_scale=None) == INVALID
    assert call(lib, B=0, lens=None, table=None) == 0
    assert call(lib, T=0, lens=None, table=None) == 0


def test_append_refusals(lib):
    assert _append(lib, cache="null") == INVALID
    assert _append(lib, cache=_cache(k=0x100008)) == INVALID
    assert _append(lib, cache=_cache(v=None)) == INVALID
    assert _append(lib, n_new=0x700001) == INVALID
    assert _append(lib, k=_view(0x500004)) == INVALID
    assert _append(lib, v=_view(None)) == INVALID
    assert "v_new" in _lib.last_error()
    assert _append(lib, k=_view(strides=(512, 130, 128))) == INVALID
    assert _append(lib, k=_view(strides=(512, 128, -128))) == INVALID
    assert "multiples of 8" in _lib.last_error()


def test_attention_refusals(lib):
    assert _attend(lib, H=3) == INVALID
    assert _attend(lib, H=-2) == INVALID
    assert _attend(lib, scale=float("nan")) == INVALID
    assert _attend(lib, window=-1) == INVALID
    assert _attend(lib, mod=ScoreMod(-1.0, None)) == INVALID
    assert _attend(lib, mod=ScoreMod(float("nan"), None)) == INVALID
    assert _attend(lib, mod=ScoreMod(1e-30, None), scale=1e20) == INVALID
    assert _attend(lib, mod=ScoreMod(0.0, 0x1002)) == INVALID
    assert _attend(lib, q=_view(0x500002)) == INVALID
    assert _attend(lib, out=_view(None)) == INVALID
    assert _attend(lib, lse=0x700002) == INVALID
    assert _attend(lib, H=0, q=_view(None)) == 0
    need = lib.bsm_paged_attention_workspace_bytes()
    assert _attend(lib, wsb=need - 1) == INVALID
    assert _attend(lib, ws=None) == INVALID
    assert _attend(lib, ws=0x900008) == INVALID
    assert "workspace" in _lib.last_error()


@pytest.mark.parametrize("binding", ["tensors", "ctypes"])
def test_python_checks(binding, lib, monkeypatch):
    # the module that calls the library from tensors, and ctypes alone
    if binding == "ctypes":
        monkeypatch.setattr(bsm.api, "_fast", lambda: False)
    else:
        assert bsm.api._fast()
    k, v, ks, vs = ref.random_cache(3, 2, 16, 64, 1)
    cache = bsm.KVCache(k, v, ks, vs)
    assert cache.struct.num_pages == 3 and cache.struct.page_size == 16
    with pytest.raises(ValueError):
        bsm.KVCache(k.float(), v, ks, vs)
    with pytest.raises(ValueError):
        bsm.KVCache(k, v[:2], ks, vs)
    with pytest.raises(ValueError):
        bsm.KVCache(k.transpose(1, 2), v.transpose(1, 2), ks, vs)
    with pytest.raises(ValueError):
        bsm.KVCache(k, v, ks.double(), vs)
    table = torch.zeros(1, 3, dtype=torch.int32)
    lens = torch.zeros(1, dtype=torch.int32)
    new = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    bad = [
        (table.long(), lens, new), (table[0], lens, new),
        (table.repeat(2, 1), lens, new), (table, lens.long(), new),
        (table, lens.repeat(2), new), (table, lens, new.float()),
        (table, lens, new[:, :1]), (table, lens, new[..., :32]),
        (table.repeat(1, 2)[:, ::2], lens, new)]
    for t, n, x in bad:
        with pytest.raises(ValueError):
            bsm.kv_append(cache, t, n, x, x)
    with pytest.raises(ValueError):
        bsm.kv_append(cache, table, lens, new, new, n_new=lens.float())
    for t, n, x in ((table.long(), lens, q), (table, lens.long(), q),
                    (table, lens, q.float()), (table, lens, q[..., :32])):
        with pytest.raises(ValueError):
            bsm.paged_attention(x, cache, t, n)
    with pytest.raises(ValueError):
        bsm.paged_attention(q, cache, table, lens,
                            alibi_slopes=torch.zeros(3))
    with pytest.raises(ValueError):
        bsm.paged_attention(q, cache, table, lens,
                            lse=torch.zeros(1, 4, 1, dtype=torch.float64))
    # right in every way but that it lies on the host
    with pytest.raises(ValueError, match="CUDA"):
        bsm.paged_attention(q, cache, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        bsm.kv_append(cache, table, lens, new, new)


def test_a_cache_keeps_the_tensors_it_checked():
    cache = bsm.KVCache(*ref.random_cache(3, 2, 16, 64, 1))
    for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name))


def test_reference_rounding():
    # every e4m3 value is itself; midpoints go to the even neighbour
    codes = torch.arange(0, 0x7f, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(ref.e4m3(vals), vals)
    assert np.array_equal(ref.e4m3(-vals), -vals)
    mid = (vals[:-1] + vals[1:]) / 2
    want = np.where(np.arange(len(mid)) % 2 == 0, vals[:-1], vals[1:])
    assert np.array_equal(ref.e4m3(mid), want)
    assert ref.e4m3(np.array([1e9, -np.inf])).tolist() == [448.0, -448.0]
    assert np.isnan(ref.e4m3(np.array([np.nan])))[0]
    assert ref.block_scale(np.array([448.0])) == 1.0
    assert ref.block_scale(np.array([449.0])) == 2.0
    assert ref.block_scale(np.array([0.0, np.nan, np.inf])) == 2.0 ** -40
    assert ref.block_scale(np.array([1e30])) == 2.0 ** 40
