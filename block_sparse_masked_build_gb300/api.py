"""Python binding of the C ABI (same names as include/bsm.h) plus two thin
conveniences that allocate with torch and call it.

Every step of the computation runs in the CUDA kernels of libbsm.so; this
module only marshals arguments (pointers, strides, the stream) and uses
torch for device memory, pinned host memory and streams.
"""

from __future__ import annotations

import ctypes
import functools
import math
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import I64x3, KVCacheStruct, MaskInfoStruct, MaskSpec, ScoreMod

MASK_CAUSAL = 1
MASK_LOCAL = 2
MASK_SEGMENT = 4
MASK_BAND = 8  # with MASK_LOCAL: |q - k| < window
MASK_DENSE = 16  # arbitrary mask, bit-packed uint32 words per query row
SCORE_SOFTMAX = 0
SCORE_POINTWISE = 1
_INT32 = (torch.int32, torch.uint32)  # of segment ids


class BsmError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        name = _lib.STATUS_NAMES.get(status, str(status))
        super().__init__(f"{name}: {message}")


def _check(status: int) -> None:
    if status != _lib.BSM_OK:
        raise BsmError(status, _lib.last_error())


# The current device and its current stream as plain numbers (making a
# torch.cuda.Stream object costs several microseconds of every call).
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream) -> int | None:
    if stream is None:
        if _current_stream is not None and torch.cuda.is_initialized():
            return _current_stream(_current_device())
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _elsewhere(dev) -> bool:
    """Whether dev is a CUDA device other than the current one (launches and
    the current stream go by that one)."""
    return dev.index is not None and dev.type == "cuda" and \
        dev.index != torch.cuda.current_device()


def _fast():
    """The module that calls the library straight from tensors, or False."""
    return _lib._fast or _lib.fast(_check)


def _fast_stream(stream) -> int | None:
    """A given stream's handle; None leaves the choice (the tensors' device's
    current stream) to the call."""
    return None if stream is None else _stream_handle(stream)


def _other_stream(stream, dev):
    """A given stream that is not dev's current one, as a torch stream; else
    None."""
    if stream is None:
        return None
    handle = _stream_handle(stream)
    if handle == torch.cuda.current_stream(dev).cuda_stream:
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return (torch.cuda.ExternalStream(handle, device=dev) if handle
            else torch.cuda.default_stream(dev))


def _run_on(s, call):
    """call() with stream s current, so that what it allocates is s's memory:
    scratch is not used again before s has run the call, and the tensors it
    returns not before the caller's stream, too, is done with them."""
    caller = torch.cuda.current_stream(s.device)
    with torch.cuda.stream(s):
        result = call()
    for t in result:
        if t is not None and t.is_cuda:
            t.record_stream(caller)
    return result


def _scratch(nbytes: int, dev, stream, kept: dict | None = None):
    """Device memory for a call on `stream` (allocated there: see _run_on).
    With `kept`, one per (device, stream), as calls on one stream run in
    order; a captured call gets one of its own, from the graph's memory, as
    graphs captured on one stream may run at once."""
    s = _other_stream(stream, dev)
    if s is not None:
        with torch.cuda.stream(s):
            return _scratch(nbytes, dev, None, kept)
    if kept is None or torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    key = (dev, torch.cuda.current_stream(dev).cuda_stream)
    if key not in kept:
        kept[key] = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return kept[key]


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


# --------------------------------------------------------------- C ABI names

def bsm_version() -> int:
    return int(_lib.lib().bsm_version())


def bsm_last_error() -> str:
    return _lib.last_error()


def bsm_mask_info_bytes(flags: int, window: int, B: int, Sq: int, Skv: int,
                        block_q: int, block_kv: int) -> int:
    spec = MaskSpec(flags, window)
    return int(_lib.lib().bsm_mask_info_bytes(ctypes.byref(spec), B, Sq, Skv,
                                              block_q, block_kv))


@dataclass
class MaskInfo:
    """Mask-info tables living in ``buffer`` (a CUDA uint8 tensor)."""

    struct: MaskInfoStruct
    buffer: torch.Tensor
    dense_bits: object = None  # keeps a MASK_DENSE mask alive with the info

    def _view(self, ptr: int, dtype, count: int) -> torch.Tensor:
        off = ptr - self.buffer.data_ptr()
        nbytes = count * torch.empty((), dtype=dtype).element_size()
        return self.buffer[off:off + nbytes].view(dtype)

    @property
    def num_tables(self) -> int:
        return self.struct.num_tables

    @property
    def nq(self) -> int:
        return self.struct.nq

    @property
    def nk(self) -> int:
        return self.struct.nk

    @property
    def block_mask(self) -> torch.Tensor:
        s = self.struct
        return self._view(s.block_mask, torch.int8,
                          s.num_tables * s.nq * s.nk).view(
                              s.num_tables, s.nq, s.nk)

    @property
    def data_next(self) -> torch.Tensor:
        s = self.struct
        return self._view(s.data_next, torch.int32,
                          s.num_tables * s.nq * s.nk).view(
                              s.num_tables, s.nq, s.nk)

    @property
    def row_ptr(self) -> torch.Tensor:
        s = self.struct
        return self._view(s.row_ptr, torch.int32, s.num_tables * s.nq + 1)

    @property
    def seg_range(self) -> torch.Tensor:
        """[B, Sq, 2] first/last key with the row's segment id (SEGMENT)."""
        s = self.struct
        return self._view(s.seg_range, torch.int32,
                          s.num_tables * s.Sq * 2).view(s.num_tables, s.Sq, 2)

    @property
    def seg_flags(self) -> torch.Tensor:
        return self._view(self.struct.seg_flags, torch.int32, 1)

    @property
    def super_order(self):
        """[num_tables * num_super] longest-first (table, 256-row super-tile)
        pairs as table * num_super + super_tile, or None when not built."""
        s = self.struct
        if not s.super_order:
            return None
        return self._view(s.super_order, torch.int32,
                          s.num_tables * s.num_super)

    def kv_lists(self) -> tuple[torch.Tensor, torch.Tensor]:
        """(kv_idx, kv_cls) trimmed to row_ptr[-1] entries (synchronises)."""
        s = self.struct
        nnz = int(self.row_ptr[-1].item())
        idx = self._view(s.kv_idx, torch.int32, s.num_tables * s.nq * s.nk)
        cls = self._view(s.kv_cls, torch.int8, s.num_tables * s.nq * s.nk)
        return idx[:nnz], cls[:nnz]


def _check_mask_inputs(flags: int, q_seg, kv_seg, B: int, Sq: int, Skv: int,
                       dense_bits, dev) -> None:
    """What the mask-info kernels will read."""
    if flags & MASK_SEGMENT:
        for name, t, n in (("q_segment_ids", q_seg, B * Sq),
                           ("kv_segment_ids", kv_seg, B * Skv)):
            if t is not None and (t.dtype not in _INT32 or t.numel() < n
                                  or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous int32 tensor "
                                 f"of {n} elements or more")
    if flags & MASK_DENSE and dense_bits is not None and (
            dense_bits.shape[0] < Sq
            or dense_bits.shape[1] < (Skv + 31) // 32):
        raise ValueError("dense_bits must have Sq rows of ceil(Skv / 32) "
                         "words")
    given = [t for t in (q_seg, kv_seg, dense_bits) if t is not None]
    if not all(t.is_cuda for t in given):
        raise ValueError("segment ids and dense_bits must be CUDA tensors")
    if dev.type != "cuda":
        raise ValueError("the mask info must be on a CUDA device")
    if any(t.device != dev for t in given):
        raise ValueError(f"segment ids and dense_bits must be on {dev}")


def bsm_build_mask_info(flags: int, window: int, q_segment_ids, kv_segment_ids,
                        B: int, Sq: int, Skv: int, block_q: int, block_kv: int,
                        buffer: torch.Tensor, stream=None,
                        dense_bits=None) -> MaskInfo:
    """dense_bits: with MASK_DENSE, a device int32/uint32-bits tensor
    [Sq, W] (W >= ceil(Skv / 32), row-major); it must stay alive while the
    mask info is used, since the forward reads it too."""
    spec = MaskSpec(flags, window)
    if dense_bits is not None:
        if dense_bits.dim() != 2 or dense_bits.stride(1) != 1 or \
                dense_bits.element_size() != 4:
            raise ValueError("dense_bits must be a [Sq, W] 32-bit tensor with "
                             "contiguous rows")
        spec.dense_bits = dense_bits.data_ptr()
        spec.dense_row_words = dense_bits.stride(0)
    _check_mask_inputs(flags, q_segment_ids, kv_segment_ids, B, Sq, Skv,
                       dense_bits, buffer.device)
    info = MaskInfoStruct()
    _check(_lib.lib().bsm_build_mask_info(
        ctypes.byref(spec), _ptr(q_segment_ids), _ptr(kv_segment_ids), B, Sq,
        Skv, block_q, block_kv, buffer.data_ptr(),
        buffer.numel() * buffer.element_size(), ctypes.byref(info),
        _stream_handle(stream)))
    return MaskInfo(info, buffer, dense_bits)


def _strides3(t: torch.Tensor):
    st = t.stride()
    if len(st) != 4 or st[3] != 1:
        raise ValueError("tensors must be 4-D [B, H, S, D] views with a "
                         "contiguous head dimension")
    return I64x3(st[0], st[1], st[2])


def bsm_splash_fwd_workspace_bytes() -> int:
    return int(_lib.lib().bsm_splash_fwd_workspace_bytes())


_workspaces: dict = {}


def _score_mod(softcap: float, alibi_slopes, H: int, device):
    """bsm_score_mod of a cap and per-head slopes, or None for neither."""
    if alibi_slopes is not None:
        if (alibi_slopes.dtype != torch.float32
                or alibi_slopes.shape != (H,)
                or not alibi_slopes.is_contiguous()
                or alibi_slopes.device != device):
            raise ValueError("alibi_slopes must be a contiguous float32 "
                             f"tensor [{H}] on {device}")
    elif softcap == 0:
        return None
    return ScoreMod(float(softcap), _ptr(alibi_slopes))


def bsm_splash_fwd(q, k, v, mask_info: MaskInfo, q_segment_ids,
                   kv_segment_ids, scale: float, score: int, out,
                   lse=None, stream=None, workspace=None,
                   softcap: float = 0.0, alibi_slopes=None) -> None:
    """q [B,H,Sq,D], k/v [B,H_kv,Skv,D], out [B,H,Sq,D] (bf16, CUDA).
    softcap, alibi_slopes: modified softmax scores (bsm_splash_fwd_mod)."""
    B, H, Sq, D = q.shape
    H_kv, Skv = k.shape[1], k.shape[2]
    sh = _stream_handle(stream)
    mod = _score_mod(softcap, alibi_slopes, H, q.device)
    if workspace is None:
        workspace = _scratch(bsm_splash_fwd_workspace_bytes(), q.device,
                             stream, _workspaces)
    views, at = _views(q, k, v, out)  # strides are behind the pointers
    _check(_lib.lib().bsm_splash_fwd_mod(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), at + 8, at + 40, at + 72,
        at + 104, B, H, H_kv, Sq, Skv, D, mask_info.struct,
        _ptr(q_segment_ids), _ptr(kv_segment_ids), float(scale), int(score),
        mod, out.data_ptr(), _ptr(lse), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), sh))


def bsm_splash_fwd_host_bytes(flags: int, window: int, B: int, H: int,
                              H_kv: int, Sq: int, Skv: int, D: int,
                              block_q: int, block_kv: int, score: int) -> int:
    spec = MaskSpec(flags, window)
    return int(_lib.lib().bsm_splash_fwd_host_bytes(
        ctypes.byref(spec), B, H, H_kv, Sq, Skv, D, block_q, block_kv, score))


def bsm_splash_fwd_host(flags: int, window: int, q, k, v, q_segment_ids,
                        kv_segment_ids, block_q: int, block_kv: int,
                        scale: float, score: int, out, lse, device_buffer,
                        n_chunks: int = 0, stream=None) -> None:
    """The forward on contiguous CPU tensors (pinned for overlap): q
    [B,H,Sq,D], k/v [B,H_kv,Skv,D] bf16, segment ids int32 [B,S], out
    [B,H,Sq,D] bf16 and lse [B,H,Sq] f32 (or None); device_buffer a CUDA
    uint8 tensor of bsm_splash_fwd_host_bytes(...) bytes.  Enqueued on
    `stream`; out and lse are ready once it is synchronised."""
    B, H, Sq, D = q.shape
    H_kv, Skv = k.shape[1], k.shape[2]
    spec = MaskSpec(flags, window)
    _check(_lib.lib().bsm_splash_fwd_host(
        ctypes.byref(spec), q.data_ptr(), k.data_ptr(), v.data_ptr(),
        _ptr(q_segment_ids), _ptr(kv_segment_ids), B, H, H_kv, Sq, Skv, D,
        block_q, block_kv, float(scale), int(score), out.data_ptr(),
        _ptr(lse), device_buffer.data_ptr(),
        device_buffer.numel() * device_buffer.element_size(), int(n_chunks),
        _stream_handle(stream)))


def bsm_splash_fwd_noalloc(q, k, v, mask_info: MaskInfo, q_segment_ids,
                           kv_segment_ids, scale: float, score: int, out,
                           lse=None, stream=None) -> None:
    """bsm_splash_fwd using the library's own device scratch (allocates
    nothing; calls that overlap on the GPU must not be issued)."""
    B, H, Sq, D = q.shape
    H_kv, Skv = k.shape[1], k.shape[2]
    _check(_lib.lib().bsm_splash_fwd_noalloc(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _strides3(q), _strides3(k),
        _strides3(v), _strides3(out), B, H, H_kv, Sq, Skv, D,
        ctypes.byref(mask_info.struct), _ptr(q_segment_ids),
        _ptr(kv_segment_ids), float(scale), int(score), out.data_ptr(),
        _ptr(lse), _stream_handle(stream)))


def _views(*tensors):
    """bsm_tensor structs (32 bytes each) of 4-D [B, heads, S, D] tensor
    views, in one array: (array, its address); None leaves zeros."""
    flat = []
    for t in tensors:
        if t is None:
            flat += (0, 0, 0, 0)
            continue
        st = t.stride()
        if len(st) != 4 or st[3] != 1:
            raise ValueError("tensors must be 4-D [B, H, S, D] views with a "
                             "contiguous head dimension")
        flat += (t.data_ptr(), st[0], st[1], st[2])
    array = _views_type(len(flat))(*flat)
    return array, ctypes.addressof(array)


@functools.lru_cache(maxsize=None)
def _views_type(n: int):
    return ctypes.c_int64 * n


def bsm_splash_bwd_workspace_bytes(B: int, H: int, Sq: int,
                                   score: int) -> int:
    return int(_lib.lib().bsm_splash_bwd_workspace_bytes(B, H, Sq, score))


def bsm_splash_bwd_mod_workspace_bytes(B: int, H: int, H_kv: int, Sq: int,
                                       Skv: int, D: int) -> int:
    return int(_lib.lib().bsm_splash_bwd_mod_workspace_bytes(B, H, H_kv, Sq,
                                                             Skv, D))


def bsm_splash_bwd(q, k, v, out, lse, dout, mask_info: MaskInfo,
                   q_segment_ids, kv_segment_ids, scale: float, score: int,
                   dq, dk, dv, stream=None, workspace=None,
                   softcap: float = 0.0, alibi_slopes=None) -> None:
    """Gradients of sum(dout * out): dq [B,H,Sq,D], dk/dv [B,H_kv,Skv,D]
    (bf16, CUDA), from the forward's q, k, v and (softmax) out and lse.
    softcap, alibi_slopes: as given to the forward."""
    B, H, Sq, D = q.shape
    H_kv, Skv = k.shape[1], k.shape[2]
    sh = _stream_handle(stream)
    mod = _score_mod(softcap, alibi_slopes, H, q.device)
    need = bsm_splash_bwd_workspace_bytes(B, H, Sq, score) if mod is None \
        else bsm_splash_bwd_mod_workspace_bytes(B, H, H_kv, Sq, Skv, D)
    if workspace is None and need > 0:
        workspace = _scratch(need, q.device, stream)
    views, at = _views(q, k, v, out, dout, dq, dk, dv)
    _check(_lib.lib().bsm_splash_bwd_mod(
        at, at + 32, at + 64, None if out is None else at + 96, _ptr(lse),
        at + 128, B, H, H_kv, Sq, Skv, D, mask_info.struct,
        _ptr(q_segment_ids), _ptr(kv_segment_ids), float(scale), int(score),
        mod, at + 160, at + 192, at + 224, _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        sh))


_BF16_BITS = (torch.bfloat16, torch.int16, torch.uint16)


def _covers(t, sizes) -> bool:
    """Whether t holds the first `sizes` (a larger buffer may serve)."""
    return t.dim() == len(sizes) and all(
        n >= m for n, m in zip(t.shape, sizes))


def _check_operands(q, k, v) -> None:
    """The checks of the tensor binding on a forward's operands, which hold
    what their pointers will be read with."""
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != 4 or t.stride(3) != 1:
            raise ValueError("tensors must be 4-D [B, H, S, D] views with a "
                             "contiguous head dimension")
        if t.dtype not in _BF16_BITS or t.device != dev:
            raise ValueError(f"{name} must be a bfloat16 tensor on {dev}")
    need = (q.shape[0], k.shape[1], k.shape[2], q.shape[3])
    if not _covers(k, need) or not _covers(v, need):
        raise ValueError("k and v must be [B, H_kv, Skv, D] for q's B and D")


def _check_like(t, like, name: str) -> None:
    if t is not None and (t.dtype not in _BF16_BITS
                          or not _covers(t, like.shape)
                          or t.device != like.device):
        raise ValueError(f"{name} must be a bfloat16 tensor of q's shape and "
                         "device")


def _check_lse(t, q) -> None:
    if t is not None and (t.dtype != torch.float32
                          or t.numel() < math.prod(q.shape[:3])
                          or not t.is_contiguous() or t.device != q.device):
        raise ValueError("lse must be a contiguous float32 tensor of B H Sq "
                         "elements or more on q's device")


def _check_ids(t, B: int, S: int, dev, name: str) -> None:
    if t is not None and (t.dtype not in _INT32 or t.numel() < B * S
                          or not t.is_contiguous() or t.device != dev):
        raise ValueError(f"{name} must be a contiguous int32 tensor of B S "
                         f"elements or more on {dev}")


def _check_both_ids(q_seg, kv_seg, q, k) -> None:
    _check_ids(q_seg, q.shape[0], q.shape[2], q.device, "q_segment_ids")
    _check_ids(kv_seg, q.shape[0], k.shape[2], q.device, "kv_segment_ids")


def _check_cache(k_pages, v_pages, k_scale, v_scale) -> None:
    shape, dev = k_pages.shape, k_pages.device
    for t in (k_pages, v_pages):
        if (t.dtype != torch.float8_e4m3fn or t.dim() != 4
                or t.shape != shape or not t.is_contiguous()
                or t.device != dev):
            raise ValueError("k_pages and v_pages must be contiguous "
                             "float8_e4m3fn tensors of one shape "
                             "[num_pages, H_kv, page_size, D] on one device")
    for t in (k_scale, v_scale):
        if (t.dtype != torch.float32 or t.shape != shape[:2]
                or not t.is_contiguous() or t.device != dev):
            raise ValueError("k_scale and v_scale must be contiguous float32 "
                             "tensors [num_pages, H_kv] beside the pages")


class KVCache:
    """A paged 8-bit key/value cache over four CUDA tensors, which it keeps:
    k_pages, v_pages [num_pages, H_kv, page_size, D] (float8_e4m3fn) and
    k_scale, v_scale [num_pages, H_kv] (float32), all contiguous.  An element
    is its code times the scale of its page and head, which lies between 2^-40
    and 2^40 wherever a page holds tokens."""

    __slots__ = ("_tensors",)

    def __init__(self, k_pages, v_pages, k_scale, v_scale):
        fast = _fast()
        if fast:
            fast.check_cache(k_pages, v_pages, k_scale, v_scale)
        else:
            _check_cache(k_pages, v_pages, k_scale, v_scale)
        self._tensors = (k_pages, v_pages, k_scale, v_scale)

    # read only: calls rely on the checks made above
    k_pages = property(lambda self: self._tensors[0])
    v_pages = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    @property
    def device(self) -> torch.device:
        return self._tensors[0].device

    @property
    def struct(self) -> KVCacheStruct:
        """bsm_kv_cache, for the C ABI."""
        return KVCacheStruct(*[t.data_ptr() for t in self._tensors],
                             *self.k_pages.shape)

    @classmethod
    def empty(cls, num_pages: int, H_kv: int, page_size: int, D: int,
              device="cuda") -> "KVCache":
        """A cache of unwritten pages."""
        pages = [torch.empty((num_pages, H_kv, page_size, D),
                             dtype=torch.float8_e4m3fn, device=device)
                 for _ in range(2)]
        scales = [torch.ones((num_pages, H_kv), device=device)
                  for _ in range(2)]
        return cls(*pages, *scales)


def _check_table(dev, page_table, B: int, lens, n_new=None) -> None:
    if (page_table.dtype != torch.int32 or page_table.dim() != 2
            or page_table.shape[0] != B or page_table.device != dev
            or (page_table.shape[1] > 1 and page_table.stride(1) != 1)):
        raise ValueError("page_table must be an int32 tensor [B, max_pages] "
                         "with contiguous rows, beside the cache")
    for name, t in (("lens", lens), ("n_new", n_new)):
        if t is not None and (t.dtype != torch.int32 or t.shape != (B,)
                              or not t.is_contiguous() or t.device != dev):
            raise ValueError(f"{name} must be a contiguous int32 tensor [B] "
                             "beside the cache")


def _check_tokens(t, shape, dev, name: str) -> None:
    if (t.dtype != torch.bfloat16 or t.shape != shape or t.device != dev
            or t.stride(3) != 1):
        raise ValueError(f"{name} must be a bfloat16 tensor {list(shape)} "
                         "with a contiguous head dimension, beside the cache")


def bsm_kv_append(cache: KVCache, page_table, lens, k_new, v_new, n_new=None,
                  stream=None) -> None:
    """Append k_new, v_new [B,H_kv,T,D] (bf16, any strides that are multiples
    of 8) to sequences of lens [B] tokens, n_new [B] of them each (None: T).
    page_table int32 [B, max_pages]; lens is left as it is."""
    dev = cache.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return bsm_kv_append(cache, page_table, lens, k_new, v_new, n_new,
                                 stream)
    s = cache.struct
    if k_new.dim() != 4:
        raise ValueError("k_new must be [B, H_kv, T, D]")
    B, _, T, _ = k_new.shape
    _check_table(dev, page_table, B, lens, n_new)
    shape = (B, s.H_kv, T, s.D)
    _check_tokens(k_new, shape, dev, "k_new")
    _check_tokens(v_new, shape, dev, "v_new")
    if dev.type != "cuda":
        raise ValueError("the cache must be on a CUDA device")
    views, at = _views(k_new, v_new)
    _check(_lib.lib().bsm_kv_append(
        s, page_table.data_ptr(), page_table.stride(0), page_table.shape[1],
        lens.data_ptr(), None if n_new is None else n_new.data_ptr(), at,
        at + 32, B, T, _stream_handle(stream)))


def bsm_paged_attention_workspace_bytes() -> int:
    return int(_lib.lib().bsm_paged_attention_workspace_bytes())


_paged_workspaces: dict = {}


def bsm_paged_attention(q, cache: KVCache, page_table, lens, scale: float,
                        out, lse=None, window: int = 0, softcap: float = 0.0,
                        alibi_slopes=None, stream=None,
                        workspace=None) -> None:
    """q, out [B,H,T,D] (bf16): the last T of each sequence's lens [B]
    tokens attend to the cache; lse [B,H,T] (f32, contiguous) or None."""
    dev = cache.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return bsm_paged_attention(q, cache, page_table, lens, scale, out,
                                       lse, window, softcap, alibi_slopes,
                                       stream, workspace)
    s = cache.struct
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, D]")
    B, H, T, D = q.shape
    _check_table(dev, page_table, B, lens)
    shape = (B, H, T, s.D)
    _check_tokens(q, shape, dev, "q")
    _check_tokens(out, shape, dev, "out")
    if lse is not None and (lse.dtype != torch.float32
                            or lse.shape != (B, H, T) or lse.device != dev
                            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 tensor [B, H, T] "
                         "beside the cache")
    mod = _score_mod(softcap, alibi_slopes, H, dev)
    if dev.type != "cuda":
        raise ValueError("the cache must be on a CUDA device")
    if window >= 2 ** 31:
        raise ValueError("integer out of range")
    sh = _stream_handle(stream)
    if workspace is None:
        workspace = _scratch(bsm_paged_attention_workspace_bytes(), dev,
                             stream, _paged_workspaces)
    views, at = _views(q, out)
    _check(_lib.lib().bsm_paged_attention(
        at, s, page_table.data_ptr(), page_table.stride(0),
        page_table.shape[1], lens.data_ptr(), B, H, T, scale, window, mod,
        at + 32, None if lse is None else lse.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        sh))


def bsm_device_status(stream=None) -> tuple[int, list[int]]:
    detail = (ctypes.c_int32 * 4)()
    st = _lib.lib().bsm_device_status(_stream_handle(stream), detail)
    return int(st), list(detail)


def bsm_selftest_wait_timeout(timeout_ns: int, stream=None) -> None:
    _check(_lib.lib().bsm_selftest_wait_timeout(int(timeout_ns),
                                                _stream_handle(stream)))


def bsm_debug_set_trace(buffer) -> None:
    """Trace the following forward launches into ``buffer`` (a CUDA tensor,
    16-byte aligned) or switch tracing off with None."""
    if buffer is None:
        _check(_lib.lib().bsm_debug_set_trace(None, 0))
    else:
        _check(_lib.lib().bsm_debug_set_trace(
            buffer.data_ptr(), buffer.numel() * buffer.element_size()))


def bsm_debug_fwd_grid(B: int, H: int, Sq: int) -> int:
    return int(_lib.lib().bsm_debug_fwd_grid(B, H, Sq))


def decode_trace(buffer, grid: int):
    """Records of a trace buffer as a list per CTA of
    (t_ns, role, event, tile, entry, unit), sorted by time."""
    raw = buffer.cpu().numpy().view("<u8").reshape(-1, 2)
    per = raw.shape[0] // grid
    region = (per - 2) // 6
    out = []
    for c in range(grid):
        blk = raw[c * per:(c + 1) * per]
        counts = blk[0:2].reshape(-1).view("<u4")[:6]
        recs = []
        for r, n in enumerate(counts):
            for i in range(int(n)):
                row = blk[2 + r * region + i]
                a = int(row[1] & 0xFFFFFFFF)
                recs.append((int(row[0]), a >> 28, (a >> 24) & 15,
                             (a >> 20) & 15, a & 0xFFFFF, int(row[1] >> 32)))
        recs.sort()
        out.append(recs)
    return out


# ------------------------------------------------------------ conveniences

_CUDA = torch.device("cuda")


def build_mask_info(flags: int, B: int, Sq: int, Skv: int, block_q: int = 128,
                    block_kv: int = 128, window: int = 0, q_segment_ids=None,
                    kv_segment_ids=None, device=None, stream=None,
                    dense_bits=None) -> MaskInfo:
    """Allocate the mask-info buffer with torch and build the tables."""
    if stream is not None:
        dev = torch.device(device) if device is not None else \
            _CUDA if q_segment_ids is None else q_segment_ids.device
        s = _other_stream(stream, dev) if dev.type == "cuda" else None
        if s is not None:
            made = []

            def build():
                made.append(build_mask_info(
                    flags, B, Sq, Skv, block_q, block_kv, window,
                    q_segment_ids, kv_segment_ids, device, None, dense_bits))
                return [made[0].buffer]

            _run_on(s, build)
            return made[0]
    if device is not None and torch.device(device).type != "cuda":
        raise ValueError("the mask info must be on a CUDA device")
    fast = _fast()
    if fast:
        if device is None:
            index = None if q_segment_ids is None else \
                q_segment_ids.device.index
        else:
            index = torch.device(device).index
        info = MaskInfoStruct()
        buf = fast.build_mask_info(
            ctypes.addressof(info), flags, window, q_segment_ids,
            kv_segment_ids, B, Sq, Skv, block_q, block_kv, index, dense_bits,
            _fast_stream(stream))
        if buf is None:
            raise BsmError(_lib.BSM_ERR_INVALID_ARG, bsm_last_error())
        return MaskInfo(info, buf, dense_bits)
    nbytes = bsm_mask_info_bytes(flags, window, B, Sq, Skv, block_q, block_kv)
    if nbytes == 0:
        raise BsmError(_lib.BSM_ERR_INVALID_ARG, bsm_last_error())
    if device is None:
        device = (q_segment_ids.device if q_segment_ids is not None
                  else _CUDA)
    buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return bsm_build_mask_info(flags, window, q_segment_ids, kv_segment_ids, B,
                               Sq, Skv, block_q, block_kv, buf, stream,
                               dense_bits)


def bsm_pack_dense_mask(mask: torch.Tensor, words: torch.Tensor,
                        stream=None) -> None:
    """Bit-pack a boolean CUDA mask [Sq, Skv] (rows contiguous) into the
    int32/uint32 CUDA tensor words [Sq, W], W >= ceil(Skv / 32): bit k % 32
    of word k // 32 of row q is mask[q, k] (the layout MASK_DENSE reads)."""
    if not (mask.is_cuda and words.is_cuda):
        raise ValueError("mask and words must be CUDA tensors")
    if mask.dim() != 2 or mask.stride(1) != 1 or mask.element_size() != 1:
        raise ValueError("mask must be a [Sq, Skv] bool/uint8 tensor with "
                         "contiguous rows")
    if words.dim() != 2 or words.stride(1) != 1 or words.element_size() != 4:
        raise ValueError("words must be a [Sq, W] 32-bit tensor with "
                         "contiguous rows")
    Sq, Skv = mask.shape
    if words.shape[0] != Sq:
        raise ValueError("words must have one row per mask row")
    _check(_lib.lib().bsm_pack_dense_mask(
        mask.data_ptr(), mask.stride(0), Sq, Skv, words.data_ptr(),
        words.stride(0), _stream_handle(stream)))


def pack_dense_mask(mask: torch.Tensor, stream=None) -> torch.Tensor:
    """bsm_pack_dense_mask into a new int32 tensor [Sq, ceil(Skv / 32)]."""
    Sq, Skv = mask.shape
    if mask.dtype != torch.bool and mask.dtype != torch.uint8:
        mask = mask != 0
    mask = mask.contiguous()
    words = torch.empty((Sq, (Skv + 31) // 32), dtype=torch.int32,
                        device=mask.device)
    bsm_pack_dense_mask(mask, words, stream)
    return words


def kv_append(cache: KVCache, page_table, lens, k_new, v_new, *, n_new=None,
              stream=None) -> None:
    """Append new tokens' keys and values (bf16 [B, H_kv, T, D]) to the 8-bit
    cache: sequence b, which holds lens[b] tokens, gets its first n_new[b]
    (None: all T).  One scale per page and head, a power of two; a page that
    already holds tokens keeps or raises its scale (include/bsm.h has the
    rule).  A page that the call writes belongs to one sequence only; pages
    that sequences share are full ones.  ``lens`` is not changed: advance it
    before attending."""
    fast = _fast()
    if fast:
        return fast.kv_append(
            *cache._tensors, page_table, lens, k_new, v_new, n_new,
            _fast_stream(stream))
    bsm_kv_append(cache, page_table, lens, k_new, v_new, n_new, stream)


def paged_attention(q, cache: KVCache, page_table, lens, *,
                    scale: float | None = None, window: int = 0,
                    softcap: float = 0.0, alibi_slopes=None,
                    return_lse: bool = True, out=None, lse=None, stream=None):
    """Causal attention of q [B, H, T, D] (bf16), the last T tokens of each
    sequence, over the cache's lens[b] tokens (the queries' own among them).

    ``window`` > 0 keeps the last ``window`` keys of each query; scale,
    ``softcap`` and ``alibi_slopes`` as in :func:`splash_attention`.  Rows
    that see no key are 0 with logsumexp -inf.  Returns (out, lse)."""
    s = _other_stream(stream, cache.device) \
        if cache.device.type == "cuda" else None
    if s is not None:
        return _run_on(s, lambda: paged_attention(
            q, cache, page_table, lens, scale=scale, window=window,
            softcap=softcap, alibi_slopes=alibi_slopes, return_lse=return_lse,
            out=out, lse=lse))
    fast = _fast()
    if fast:
        return fast.paged_attention(
            *cache._tensors, page_table, lens, q, scale, window, softcap,
            alibi_slopes, out, lse, return_lse, _fast_stream(stream))
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, D]")
    B, H, T, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((B, H, T, D), dtype=torch.bfloat16, device=q.device)
    if not return_lse:
        lse = None
    elif lse is None:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    bsm_paged_attention(q, cache, page_table, lens, scale, out, lse, window,
                        softcap, alibi_slopes, stream)
    return out, lse


def splash_attention_bwd(q, k, v, out, lse, dout, *,
                         mask_flags: int = MASK_CAUSAL, window: int = 0,
                         q_segment_ids=None, kv_segment_ids=None,
                         scale: float | None = None,
                         score: int = SCORE_SOFTMAX, block_q: int = 128,
                         block_kv: int = 128,
                         mask_info: MaskInfo | None = None, stream=None,
                         dense_mask=None, softcap: float = 0.0,
                         alibi_slopes=None):
    """Backward of :func:`splash_attention` on CUDA tensors: returns
    (dq, dk, dv) for the gradient ``dout`` of the output.  ``out`` and
    ``lse`` are the forward's (softmax path; ignored for the pointwise
    path); ``softcap`` and ``alibi_slopes`` as given to it (the slopes are
    constants and get no gradient)."""
    s = _other_stream(stream, q.device) if q.is_cuda else None
    if s is not None:
        return _run_on(s, lambda: splash_attention_bwd(
            q, k, v, out, lse, dout, mask_flags=mask_flags, window=window,
            q_segment_ids=q_segment_ids, kv_segment_ids=kv_segment_ids,
            scale=scale, score=score, block_q=block_q, block_kv=block_kv,
            mask_info=mask_info, dense_mask=dense_mask, softcap=softcap,
            alibi_slopes=alibi_slopes))
    B, H, Sq, D = q.shape
    Skv = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if mask_info is None:
        bits = None
        if dense_mask is not None:
            bits = pack_dense_mask(dense_mask.to(q.device))
        mask_info = build_mask_info(mask_flags, B, Sq, Skv, block_q, block_kv,
                                    window, q_segment_ids, kv_segment_ids,
                                    device=q.device, stream=stream,
                                    dense_bits=bits)
    sm = score == SCORE_SOFTMAX
    fast = _fast()
    if fast:
        return fast.splash_bwd(
            q, k, v, out if sm else None, lse if sm else None, dout,
            ctypes.addressof(mask_info.struct), q_segment_ids, kv_segment_ids,
            scale, score, softcap, alibi_slopes, _fast_stream(stream))
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    _check_operands(q, k, v)
    _check_like(out if sm else None, q, "out")
    _check_like(dout, q, "dout")
    _check_lse(lse if sm else None, q)
    _check_both_ids(q_segment_ids, kv_segment_ids, q, k)
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    bsm_splash_bwd(q, k, v, out if sm else None, lse if sm else None, dout,
                   mask_info, q_segment_ids, kv_segment_ids, scale, score, dq,
                   dk, dv, stream, softcap=softcap, alibi_slopes=alibi_slopes)
    return dq, dk, dv


def _can_pipeline(q, k, v, out, lse, q_seg, kv_seg, stream, mask_info,
                  dense_mask):
    """Host inputs go through bsm_splash_fwd_host (chunked copies that
    overlap the forward when the memory is pinned) when they and any given
    outputs are contiguous CPU tensors, and no prebuilt mask info or
    arbitrary mask is involved."""
    ts = [q, k, v] + [t for t in (out, lse, q_seg, kv_seg) if t is not None]
    return (all(t.device.type == "cpu" and t.is_contiguous() for t in ts)
            and mask_info is None and dense_mask is None
            and (stream is None or isinstance(stream, torch.cuda.Stream))
            and k.shape[1] > 0 and q.shape[1] % k.shape[1] == 0)


def _splash_host_pipelined(q, k, v, flags, window, q_seg, kv_seg, scale,
                           score, block_q, block_kv, want_lse, out, lse,
                           stream, dev):
    """Host tensors through bsm_splash_fwd_host: one call that copies in,
    builds the mask info, runs the forward and copies out, pipelined over
    ranges of heads on the library's copy streams."""
    B, H, Sq, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    comp = torch.cuda.current_stream(dev) if stream is None else stream
    nbytes = bsm_splash_fwd_host_bytes(flags, window, B, H, Hkv, Sq, Skv, D,
                                       block_q, block_kv, score)
    if nbytes == 0:
        raise BsmError(_lib.BSM_ERR_INVALID_ARG,
                       "bsm_splash_fwd_host_bytes: bad arguments")
    with torch.cuda.stream(comp):
        buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty((B, H, Sq, D), dtype=torch.bfloat16,
                          pin_memory=True)
    if want_lse and lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, pin_memory=True)
    qs = None if q_seg is None else q_seg.to(torch.int32).contiguous()
    ks = None if kv_seg is None else kv_seg.to(torch.int32).contiguous()
    bsm_splash_fwd_host(flags, window, q, k, v, qs, ks, block_q, block_kv,
                        scale, score, out, lse if want_lse else None, buf,
                        0, comp)
    comp.synchronize()
    return out, (lse if want_lse else None)


def splash_attention(q, k, v, *, mask_flags: int = MASK_CAUSAL,
                     window: int = 0, q_segment_ids=None, kv_segment_ids=None,
                     scale: float | None = None, score: int = SCORE_SOFTMAX,
                     block_q: int = 128, block_kv: int = 128,
                     mask_info: MaskInfo | None = None,
                     return_lse: bool = True, out=None, lse=None,
                     stream=None, dense_mask=None, softcap: float = 0.0,
                     alibi_slopes=None):
    """Block-sparse masked attention forward, q/k/v [B, H, S, D] bf16.

    Defaults follow hstu_ops ``pointwise_splash_attention``: scale =
    1/sqrt(D).  With CUDA inputs everything stays on the device.  With CPU
    inputs (ideally pinned) the inputs are copied to the current device,
    the kernels run there, and ``out``/``lse`` are copied back into host
    tensors (``out``/``lse`` may be given, pinned, to be reused).
    Returns (out, lse); lse is None for the pointwise path or when
    ``return_lse`` is False.  ``dense_mask`` (with MASK_DENSE) is a boolean
    [Sq, Skv] tensor, an arbitrary mask shared by every batch row and head;
    it is bit-packed on the device here.

    Modified softmax scores: with x = scale * q.k, ``softcap`` = c > 0 makes
    the score c * tanh(x / c), and ``alibi_slopes`` (float32 [H], contiguous,
    on the compute device, or on the host with host inputs) subtracts
    slopes[h] * |q - k|; the mask comes after both.
    """
    B, H, Sq, D = q.shape
    Skv = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    host = q.is_cpu
    dev = torch.device("cuda", torch.cuda.current_device()) if host \
        else q.device
    want_lse = return_lse and score == SCORE_SOFTMAX
    modified = softcap != 0 or alibi_slopes is not None
    if host and not modified and _can_pipeline(
            q, k, v, out, lse, q_segment_ids, kv_segment_ids, stream,
            mask_info, dense_mask):
        return _splash_host_pipelined(
            q, k, v, mask_flags, window, q_segment_ids, kv_segment_ids,
            scale, score, block_q, block_kv, want_lse, out, lse, stream, dev)
    s = _other_stream(stream, dev)
    if s is not None:
        return _run_on(s, lambda: splash_attention(
            q, k, v, mask_flags=mask_flags, window=window,
            q_segment_ids=q_segment_ids, kv_segment_ids=kv_segment_ids,
            scale=scale, score=score, block_q=block_q, block_kv=block_kv,
            mask_info=mask_info, return_lse=return_lse, out=out, lse=lse,
            dense_mask=dense_mask, softcap=softcap,
            alibi_slopes=alibi_slopes))
    if host:
        nb = q.is_pinned()
        qd = q.to(dev, non_blocking=nb)
        kd = k.to(dev, non_blocking=nb)
        vd = v.to(dev, non_blocking=nb)
        qs = None if q_segment_ids is None else \
            q_segment_ids.to(dev, non_blocking=nb)
        ks = None if kv_segment_ids is None else \
            kv_segment_ids.to(dev, non_blocking=nb)
        if alibi_slopes is not None:
            alibi_slopes = alibi_slopes.to(dev)
    else:
        qd, kd, vd, qs, ks = q, k, v, q_segment_ids, kv_segment_ids
    if mask_info is None:
        bits = None
        if dense_mask is not None:
            bits = pack_dense_mask(dense_mask.to(dev))
        mask_info = build_mask_info(mask_flags, B, Sq, Skv, block_q, block_kv,
                                    window, qs, ks, device=dev, stream=stream,
                                    dense_bits=bits)
    fast = _fast()
    if fast and not host:
        return fast.splash_fwd(
            q, k, v, ctypes.addressof(mask_info.struct), qs, ks, scale, score,
            softcap, alibi_slopes, out, lse, want_lse, _fast_stream(stream))
    _check_operands(qd, kd, vd)
    _check_both_ids(qs, ks, qd, kd)
    _score_mod(softcap, alibi_slopes, H, dev)
    od = torch.empty((B, H, Sq, D), dtype=torch.bfloat16, device=dev) \
        if (host or out is None) else out
    _check_like(od, qd, "out")
    ld = None
    if want_lse:
        ld = torch.empty((B, H, Sq), dtype=torch.float32, device=dev) \
            if (host or lse is None) else lse
        _check_lse(ld, qd)
    bsm_splash_fwd(qd, kd, vd, mask_info, qs, ks, scale, score, od, ld,
                   stream, softcap=softcap, alibi_slopes=alibi_slopes)
    if not host:
        return od, ld
    if out is None:
        out = torch.empty((B, H, Sq, D), dtype=torch.bfloat16,
                          pin_memory=True)
    out.copy_(od, non_blocking=True)
    if want_lse:
        if lse is None:
            lse = torch.empty((B, H, Sq), dtype=torch.float32,
                              pin_memory=True)
        lse.copy_(ld, non_blocking=True)
    torch.cuda.current_stream(dev).synchronize()  # (another: see _run_on)
    return out, (lse if want_lse else None)
