"""Attention of drafted tokens without a GPU: refusals of the entry point and
bindings, the workspace's size, and the fp64 reference against the plain
cache's."""

import ctypes

import pytest
import torch

import block_sparse_masked_build_gb300 as bsm
import kv_cache_ref
import tree_ref as ref
from block_sparse_masked_build_gb300 import _lib, api
from block_sparse_masked_build_gb300 import build as bsm_build
from block_sparse_masked_build_gb300._lib import (I64x3, KVCacheStruct,
                                                  ScoreMod, TensorView)

INVALID, UNSUPPORTED = _lib.BSM_ERR_INVALID_ARG, _lib.BSM_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    bsm_build.build()
    return _lib.lib()


def _view(data=0x500000, strides=(1 << 20, 1 << 16, 128)):
    return ctypes.byref(TensorView(data, I64x3(*strides)))


def _attend(lib, n_new=0xa00000, tree=0xb00000, sb=64, st=4, B=2, H=4, T=40,
            scale=0.1, window=0, mod=None, q=None, out=None, lse=None,
            ws=0x900000, wsb=1 << 40, lens=0x700000, **kw):
    d = dict(k=0x100000, v=0x200000, k_scale=0x300000, v_scale=0x400000,
             num_pages=8, H_kv=2, page_size=64, D=128)
    d.update(kw)
    c = KVCacheStruct(*[d[n] for n, _ in KVCacheStruct._fields_])
    return lib.bsm_paged_attention_tree(
        q or _view(), ctypes.byref(c), 0x600000, 4, 4, lens, n_new, tree, sb,
        st, B, H, T, scale, window, mod, out or _view(0x800000), lse, ws, wsb,
        None)


def test_refusals(lib):
    # found before anything touches the device
    for bad in (dict(n_new=0xa00002), dict(tree=0xb00001), dict(sb=-1),
                dict(st=-4), dict(scale=float("nan")), dict(window=-1),
                dict(H=3), dict(T=-1), dict(B=-1), dict(lens=None),
                dict(lse=0x1002), dict(ws=None), dict(ws=0x900008),
                dict(wsb=64), dict(q=_view(0)), dict(q=_view(0x500008)),
                dict(out=_view(strides=(8, 8, 12))),
                dict(mod=ctypes.byref(ScoreMod(-1.0, None)))):
        assert _attend(lib, **bad) == INVALID, bad
    for bad in (dict(T=1025), dict(D=96), dict(page_size=48),
                dict(T=1024, H=2048)):
        assert _attend(lib, **bad) == UNSUPPORTED, bad
    for nothing in (dict(B=0), dict(T=0), dict(H=0, H_kv=0)):
        assert _attend(lib, **nothing) == 0, nothing


@pytest.mark.parametrize("T", [1, 4, 5, 32, 33, 64, 65, 1024])
def test_workspace(lib, T):
    need = lib.bsm_paged_attention_tree_workspace_bytes(8, 2, T, 128)
    assert 0 < need < 1 << 30 and need % 16 == 0
    assert _attend(lib, T=T, H=8, st=32, wsb=need - 1) == INVALID
    assert "_tree_workspace_bytes" in _lib.last_error()


def test_workspace_of_nothing(lib):
    f = lib.bsm_paged_attention_tree_workspace_bytes
    for a in ((0, 0, 4, 128), (8, 0, 4, 128), (8, 3, 4, 128), (8, 2, 0, 128),
              (8, 2, -1, 128), (-8, 2, 4, 128), (8, 2, 4, 96)):
        assert f(*a) >= 0, a  # (an answer, not an abort)


def _t(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


def test_tree_argument():
    cpu = torch.device("cpu")
    for good in (None, _t(2, 40, 2), _t(40, 2), _t(40, 7), _t(40, 7)[:, 2:4],
                 _t(2, 40, 2).view(torch.uint32), _t(1, 40, 2).expand(2, 40, 2)):
        api._check_tree(good, 2, 40, cpu)
    for bad in (_t(2, 40, 1), _t(2, 39, 2), _t(3, 40, 2), _t(40, 4)[:, ::2],
                _t(40), _t(1, 2, 40, 2), _t(40, 2).long(), _t(40, 2).bool(),
                _t(40, 2).to("meta")):
        with pytest.raises(ValueError, match="tree"):
            api._check_tree(bad, 2, 40, cpu)


@pytest.mark.parametrize("fast", [False, True])
def test_binding_refusals(fast, monkeypatch):
    if fast and not api._fast():
        pytest.skip("the tensor binding is not built")
    if not fast:
        monkeypatch.setattr(api, "_fast", lambda: False)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    cache = bsm.KVCache(z(4, 2, 32, 64).to(torch.float8_e4m3fn),
                        z(4, 2, 32, 64).to(torch.float8_e4m3fn),
                        z(4, 2, dtype=torch.float32),
                        z(4, 2, dtype=torch.float32))
    q, table, lens = z(2, 4, 40, 64), _t(2, 2), _t(2)

    def call(q=q, tree=None, n_new=lens):
        return bsm.paged_attention(q, cache, table, lens, tree=tree,
                                   n_new=n_new)

    with pytest.raises(ValueError, match="CUDA"):
        call(tree=_t(2, 40, 2))
    for bad in (dict(tree=_t(2, 40, 1)), dict(tree=_t(40, 4)[:, ::2]),
                dict(tree=_t(2, 40, 2).long()), dict(n_new=_t(3)),
                dict(n_new=_t(2).long()), dict(q=q[0]), dict(q=q.float())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises((TypeError, AttributeError)):
        call(tree=3)


def test_pack():
    bits = ref.random_tree(2, 70, 5, empty=0.1)
    words = ref.pack(bits)
    assert words.shape == (2, 70, 3) and words.dtype == torch.int32
    w = words.numpy().view("uint32")
    for b, t, j in ((0, 3, 3), (1, 69, 64), (1, 40, 31), (0, 69, 0)):
        assert (int(w[b, t, j // 32]) >> (j % 32) & 1) == int(bits[b, t, j])


@pytest.mark.parametrize("window,softcap,bias",
                         [(0, 0.0, False), (7, 3.0, False), (40, 0.0, True)])
def test_reference_is_the_caches_for_a_chain(window, softcap, bias):
    H, Hkv, D, T, P = 4, 2, 64, 6, 16
    lens = [50, 6, 33]
    pages = kv_cache_ref.random_cache(16, Hkv, P, D, 3)
    table = kv_cache_ref.random_table(lens, P, 5, 16, 4)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(3, H, T, D, generator=g).bfloat16()
    slopes = [0.1, 0.02, 0.5, 0.3] if bias else None
    more = (D ** -0.5, window, softcap, slopes)
    want = kv_cache_ref.attention(q, *pages, table, lens, *more)
    lower = torch.ones(T, T, dtype=torch.bool).tril().expand(3, T, T)
    for bits in (None, lower):
        got = ref.attention(q, *pages, table, lens, [T] * 3, bits, *more)
        assert all(torch.allclose(a, b) for a, b in zip(got, want))
