"""Norm and rotation without a GPU: refusals of the entry points and bindings,
the rotation's table, and the fp64 reference's gradient."""

import ctypes
import math

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import rope_ref as ref
from block_sparse_masked_build_gb300 import _lib, api
from block_sparse_masked_build_gb300 import build as bsm_build
from block_sparse_masked_build_gb300._lib import (HeadNorm, I64x3,
                                                  KVCacheStruct, Positions,
                                                  RopeStruct, TensorView)

INVALID, UNSUPPORTED = _lib.BSM_ERR_INVALID_ARG, _lib.BSM_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    bsm_build.build()
    return _lib.lib()


def _init(lib, dim=64, freq=None, axis=None, axes=1):
    half = max(dim // 2, 1)
    freq = [0.5] * half if freq is None else freq
    r = RopeStruct()
    st = lib.bsm_rope_init(
        r, dim, 0, (ctypes.c_double * half)(*freq),
        None if axis is None else (ctypes.c_int32 * half)(*axis), axes)
    return st, r


def test_rope_init(lib):
    st, r = _init(lib, 16, [2 * math.pi * f for f in
                            (0.25, 0.5, 1.0, 1.25, -0.25, 0.0, 3.5, 2 ** -20)],
                  [0, 1, 2, 3, 0, 1, 2, 3], 4)
    assert st == 0 and list(r.axis[:8]) == [0, 1, 2, 3] * 2
    want = [0.25, 0.5, 0.0, 0.25, 0.75, 0.0, 0.5, 2 ** -20]
    for got, w in zip(r.step[:8], want):
        d = (got / 2.0 ** 64 - w) % 1.0
        assert min(d, 1 - d) < 2.0 ** -50
    assert list(r.step[8:]) == [0] * 56
    for bad in (dict(dim=0), dict(dim=8), dict(dim=24), dict(dim=144),
                dict(axes=0), dict(axes=5), dict(freq=[float("nan")] * 32),
                dict(freq=[65.0] * 32), dict(axis=[1] * 32),
                dict(axis=[-1] * 32, axes=2)):
        assert _init(lib, **bad)[0] == INVALID, bad
    assert lib.bsm_rope_init(None, 64, 0, None, None, 1) == INVALID


def test_rope_class():
    r = bsm.Rope(64, 1e6, interleaved=True)
    assert (r.dim, r.axes, r.interleaved) == (64, 1, True)
    assert bsm.Rope(32, axes=[0, 2] * 8).axes == 3
    for bad in (dict(dim=20), dict(dim=64, inv_freq=[1.0] * 31),
                dict(dim=64, axes=[0] * 33), dict(dim=64, axes=[4] * 32)):
        with pytest.raises((ValueError, bsm.BsmError)):
            bsm.Rope(**bad)


def _view(data=0x500000, strides=(4096, 128, 256)):
    return ctypes.byref(TensorView(data, I64x3(*strides)))


def _norm(q=0x1000, k=0x2000, bf16=0, eps=1e-6):
    return HeadNorm(q, k, bf16, eps)


def _pos(data=0x3000):
    return Positions(data, (ctypes.c_int64 * 3)(0, 1, 1))


def _fwd(lib, B=1, H=2, Hkv=2, S=4, D=128, norm=None, rope=None, pos=None,
         q=None, k=None, qo=None, ko=None):
    v = _view()
    return lib.bsm_norm_rope(q or v, k or v, B, H, Hkv, S, D, norm, rope, pos,
                             qo or v, ko or v, None)


def _bwd(lib, B=1, H=2, Hkv=2, S=4, D=128, norm=None, rope=None, pos=None,
         dqw=None, dkw=None, ws=0x900000, wsb=1 << 30, q=None, **kw):
    v = _view()
    return lib.bsm_norm_rope_bwd(v, v, q or v, v, B, H, Hkv, S, D, norm, rope,
                                 pos, v, v, dqw, dkw, ws, wsb, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_refusals(lib, call):
    rope = _init(lib)[1]
    assert call(lib) == INVALID and "neither" in _lib.last_error()
    assert call(lib, rope=rope, D=96) == UNSUPPORTED
    assert call(lib, rope=rope, B=-1) == INVALID
    assert call(lib, rope=rope, B=1 << 20, S=1 << 20) == UNSUPPORTED
    assert call(lib, rope=_init(lib, 128)[1], D=64) == INVALID
    assert call(lib, rope=RopeStruct()) == INVALID
    bad = _init(lib)[1]
    bad.axis[3] = 1
    assert call(lib, rope=bad) == INVALID
    assert call(lib, norm=_norm(eps=-1.0)) == INVALID
    assert call(lib, norm=_norm(eps=float("nan"))) == INVALID
    assert call(lib, norm=_norm(q=0x1001)) == INVALID
    assert call(lib, norm=_norm(k=0x1002)) == INVALID
    assert call(lib, norm=_norm(), pos=_pos()) == INVALID
    assert call(lib, rope=rope, pos=_pos(0x3002)) == INVALID
    for v in (_view(0), _view(0x500008), _view(strides=(4096, 100, 256)),
              _view(strides=(4096, 0, 256)), _view(strides=(4096, 128, -8))):
        assert call(lib, norm=_norm(), q=v) == INVALID
    assert call(lib, rope=rope, S=0) == 0  # nothing to do


def test_backward_refusals(lib):
    rope = _init(lib)[1]
    assert _bwd(lib, rope=rope, dqw=0x1000) == INVALID
    assert "without a norm" in _lib.last_error()
    assert _bwd(lib, norm=_norm(), dqw=0x1002) == INVALID
    assert _bwd(lib, norm=_norm(), dqw=0x1000, ws=None) == INVALID
    assert _bwd(lib, norm=_norm(), dkw=0x1000, ws=0x900004) == INVALID
    assert _bwd(lib, norm=_norm(), dkw=0x1000, wsb=16) == INVALID
    v = _view()
    assert lib.bsm_norm_rope_bwd(v, v, None, v, 1, 2, 2, 4, 128, _norm(), rope,
                                 None, v, v, None, None, None, 0,
                                 None) == INVALID


def test_append_refusals(lib):
    c = KVCacheStruct(0x100000, 0x200000, 0x300000, 0x400000, 8, 2, 64, 64)

    def call(norm=None, rope=None, pos=None, cache=c):
        return lib.bsm_kv_append_rope(cache, 0x600000, 4, 4, 0x700000, None,
                                      _view(), _view(), 2, 2, norm, rope, pos,
                                      None)

    assert call() == INVALID and "neither" in _lib.last_error()
    assert call(rope=_init(lib, 128)[1]) == INVALID
    assert call(norm=_norm(), pos=_pos()) == INVALID
    assert call(norm=_norm(), cache=None) == INVALID
    c.page_size = 48
    assert call(norm=_norm()) == UNSUPPORTED


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("fast", [False, True])
def test_binding_refusals(fast, monkeypatch):
    if fast and not api._fast():
        pytest.skip("the tensor binding is not built")
    if not fast:
        monkeypatch.setattr(api, "_fast", lambda: False)
    rope, q = bsm.Rope(64), _t(1, 2, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        bsm.norm_rope(q, rope=rope)
    with pytest.raises(ValueError, match="CUDA"):
        bsm.norm_rope_bwd(q, rope=rope)
    for bad in (q.float(), q[0], q.transpose(2, 3)):
        with pytest.raises(ValueError):
            bsm.norm_rope(bad, rope=rope)
    with pytest.raises(ValueError):
        bsm.norm_rope(q, q[:, :, :3], rope=rope)
    with pytest.raises(TypeError):
        bsm.norm_rope(q, rope=3)


def test_turn_refusals():
    cpu, rope = torch.device("cpu"), bsm.Rope(64)
    three = bsm.Rope(64, axes=[0, 1, 2, 0] * 8)
    pos = _t(2, 5, dtype=torch.int32)
    api._turn(rope, pos, None, None, None, 2, 5, 64, cpu)
    api._turn(rope, pos[None], None, None, 1e-6, 2, 5, 64, cpu)
    api._turn(three, pos.expand(3, 2, 5), _t(64), _t(64), 1e-6, 2, 5, 64, cpu)
    for a in ((None, None, None, None, None), (None, pos, None, None, 1e-6),
              (rope, pos.long(), None, None, None),
              (rope, pos[:, :4], None, None, None),
              (rope, pos[:1], None, None, None), (rope, pos[0], None, None, None),
              (three, pos, None, None, None),
              (rope, pos.expand(3, 2, 5), None, None, None),
              (rope, pos.to("meta"), None, None, None),
              (rope, None, _t(64), None, None),
              (rope, None, _t(32), None, 1e-6),
              (rope, None, _t(64).half(), None, 1e-6),
              (rope, None, _t(64), _t(64).float(), 1e-6),
              (rope, None, _t(128)[::2], None, 1e-6)):
        with pytest.raises(ValueError):
            api._turn(*a, 2, 5, 64, cpu)


@pytest.mark.parametrize("inter", [False, True])
def test_reference_gradient(inter):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(2, 3, 5, 64, generator=g, dtype=torch.float64)
    w = torch.randn(64, generator=g, dtype=torch.float64)
    gr = torch.randn(2, 3, 5, 64, generator=g, dtype=torch.float64)
    pos = torch.randint(0, 900, (2, 2, 5), generator=g)
    angle = ref.angles(pos, ref.frequencies(48, 1e4), [0, 1] * 12)
    x.requires_grad_()
    w.requires_grad_()
    n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-3) * w
    want = torch.autograd.grad(ref.turn(n, angle, inter), (x, w), gr)
    dx, _, dw, _ = ref.backward(gr, x.detach(), w.detach(), 1e-3, angle, inter)
    assert torch.allclose(dx, want[0]) and torch.allclose(dw, want[1])
