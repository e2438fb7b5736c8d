"""Python entry points of scored attention and rotary positions.

``fwd_scored`` / ``bwd_scored`` and ``fwd_paged_scored`` are ``fwd`` / ``bwd``
and ``fwd_paged`` with scores that are capped, biased by distance and
restricted to a range of keys per query (``key_ranges``); ``rotary`` turns q
and k by their positions before them, ``rotary_bwd`` takes the gradients back,
and ``rotary_and_cache`` also writes the paged cache.  As in :mod:`.api`,
these check tensor metadata, allocate outputs and call the C ABI; the
arithmetic is in libfa.so.  Calls run on the device of their tensors, on
``stream`` or that device's current stream; with ``stream``, it is the caller
who orders that stream behind the inputs' work and before the results' use.
"""

from __future__ import annotations

import math
import struct
from typing import Optional, Sequence, Tuple

import torch

from . import _native
from .api import _check_input, _dtype_code, _empty_on, _shape, _workspace


# A call of the smallest sizes is bound by this module, not by its kernel, so
# the device and stream are asked for as plain numbers (a torch.cuda.Stream
# costs 2 us, its raw handle 0.1) and tensors are compared by device index.
# Builds of torch that lack these bindings take the public way.
def _public_raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_raw_stream)


def _stream(device: int, stream: Optional[torch.cuda.Stream]) -> int:
    """Handle of ``stream``, or of the device's current stream."""
    if stream is None:
        return _raw_stream(device)
    if stream.device.index != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{device}")
    return stream.cuda_stream


def _elsewhere(t: torch.Tensor) -> bool:
    """Whether ``t`` is on another device than the current one: the call then
    runs again with that one current (a launch goes to the current device)."""
    return t.get_device() not in (_current_device(), -1)


_HALF, _BF16 = torch.float16, torch.bfloat16


def _plain_qkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
    """(Z, H, Hkv, Nq, Nk, D), as ``api._shape`` checks them; that one is asked
    (and names what is wrong) only where the quick look finds something."""
    if type(q) is type(k) is type(v) is torch.Tensor:
        dt = q.dtype
        if (dt is _HALF or dt is _BF16) and k.dtype is dt and v.dtype is dt and q.is_cuda and q.is_contiguous() \
                and k.is_contiguous() and v.is_contiguous() and k.is_cuda and v.is_cuda:
            qs, ks = q.shape, k.shape
            if len(qs) == 4 and len(ks) == 4 and v.shape == ks:
                Z, H, Nq, D = qs
                Zk, Hkv, Nk, Dk = ks
                if Z == Zk and D == Dk and Hkv > 0 and H % Hkv == 0:
                    return Z, H, Hkv, Nq, Nk, D
    return _shape(q, k, v)


def _same_device(q: torch.Tensor, *tensors: Optional[torch.Tensor]) -> int:
    """Checks that every tensor (or None) is on q's device; its index."""
    device = q.get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"a tensor of shape {tuple(t.shape)} is on {t.device}, q on {q.device}")
    return device


def _check_int(name: str, t: torch.Tensor, dtype: torch.dtype, shape: Tuple[int, ...]) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _check_slopes(slopes: Optional[torch.Tensor], H: int) -> int:
    if slopes is None:
        return 0
    if not slopes.is_cuda or slopes.dtype != torch.float32 or slopes.shape != (H,) or not slopes.is_contiguous():
        raise ValueError(f"slopes must be a contiguous float32 CUDA tensor [{H}], one per query head")
    return slopes.data_ptr()


def _check_out(out, like, names) -> None:
    for name, t, x in zip(names, out, like):
        if t.shape != x[0] or t.dtype != x[1] or not t.is_contiguous():
            raise ValueError(f"out: {name} must be contiguous {x[1]} {tuple(x[0])}")


_INT_MAX = 0x7fffffff
_FLOAT_MIN = 2.0 ** -149  # the smallest fp32 above 0


def _c_int(n: int) -> int:
    """n as a C int, which ctypes would cut to its low 32 bits: a larger window
    hides no key either, and what is out of range is refused there all the same."""
    return n if -_INT_MAX <= n <= _INT_MAX else (_INT_MAX if n > 0 else -_INT_MAX)


def _c_cap(softcap: float) -> float:
    """softcap as a C float: a cap (or a negative one) too small for it must not
    become 0, which means no cap."""
    return softcap if softcap == 0.0 or not -_FLOAT_MIN < softcap < _FLOAT_MIN else math.copysign(_FLOAT_MIN, softcap)


class KeyRanges:
    """The keys that each query of a [Z, H, Nq, D] x [Z, Hkv, Nk, D] attention
    may see, as :func:`key_ranges` builds them: ``rows`` is the int32
    [Z, Nq, 2] view of (first, one past the last) key of each query ((0, 0):
    none), followed in ``buffer`` by the tables the kernels go by.  Built once
    per batch, it serves every layer's forward and backward."""

    __slots__ = ("buffer", "Z", "Nq", "Nk")

    def __init__(self, buffer: torch.Tensor, Z: int, Nq: int, Nk: int):
        self.buffer, self.Z, self.Nq, self.Nk = buffer, Z, Nq, Nk

    @property
    def rows(self) -> torch.Tensor:
        return self.buffer[: 2 * self.Z * self.Nq].view(self.Z, self.Nq, 2)


def key_ranges(Nq: int, Nk: int, doc_ids: Optional[torch.Tensor] = None, prefix_lens: Optional[torch.Tensor] = None,
               ranges: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> KeyRanges:
    """Key ranges from exactly one of: ``doc_ids`` int32 [Z, Nk] (a query sees
    the run of equal ids its position lies in; use with ``causal=True`` for
    packed causal documents), ``prefix_lens`` int32 [Z] (a query sees the keys
    up to its position and the first prefix_lens[z] keys; use with
    ``causal=False``), or ``ranges`` int32 [Z, Nq, 2] (keys lo <= j < hi; lo
    >= hi: none).  The queries are the last Nq of Nk positions."""
    given = [t for t in (doc_ids, prefix_lens, ranges) if t is not None]
    if len(given) != 1:
        raise ValueError("give exactly one of doc_ids, prefix_lens and ranges")
    t = given[0]
    if not isinstance(t, torch.Tensor) or t.dim() < 1:
        raise ValueError("doc_ids, prefix_lens and ranges are tensors with a sequence dimension")
    Z = t.shape[0]
    if Z < 1 or Nq < 1 or Nk < 1:
        raise ValueError("key_ranges needs at least one sequence, query and key")
    if doc_ids is not None:
        _check_int("doc_ids", doc_ids, torch.int32, (Z, Nk))
    elif prefix_lens is not None:
        _check_int("prefix_lens", prefix_lens, torch.int32, (Z,))
    else:
        _check_int("ranges", ranges, torch.int32, (Z, Nq, 2))
    return _key_ranges(t, doc_ids, prefix_lens, ranges, Z, Nq, Nk, stream)


def _key_ranges(t, doc_ids, prefix_lens, ranges, Z, Nq, Nk, stream) -> KeyRanges:
    if _elsewhere(t):
        with torch.cuda.device(t.device):
            return _key_ranges(t, doc_ids, prefix_lens, ranges, Z, Nq, Nk, stream)
    lib = _native.lib()
    need = lib.fa_key_ranges_size(Z, Nq, Nk)
    handle = _stream(t.get_device(), stream)
    buffer, = _empty_on(stream, t.device, (need // 4, torch.int32))
    rc = lib.fa_key_ranges(doc_ids.data_ptr() if doc_ids is not None else None,
                           prefix_lens.data_ptr() if prefix_lens is not None else None,
                           ranges.data_ptr() if ranges is not None else None, buffer.data_ptr(), need, Z, Nq, Nk, handle)
    _native.check(rc, "fa_key_ranges")
    return KeyRanges(buffer, Z, Nq, Nk)


def _mask_args(key_ranges: Optional[KeyRanges], q: torch.Tensor, Z: int, Nq: int, Nk: int):
    if key_ranges is None:
        return None, 0
    if not isinstance(key_ranges, KeyRanges):
        raise TypeError("key_ranges must come from key_ranges()")
    if (key_ranges.Z, key_ranges.Nq, key_ranges.Nk) != (Z, Nq, Nk):
        raise ValueError(f"key_ranges are for Z, Nq, Nk = {key_ranges.Z}, {key_ranges.Nq}, {key_ranges.Nk}; "
                         f"the call has {Z}, {Nq}, {Nk}")
    _same_device(q, key_ranges.buffer)
    return key_ranges.buffer.data_ptr(), key_ranges.buffer.numel() * 4


def fwd_scored(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
               scale: Optional[float] = None, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
               window: int = 0, key_ranges: Optional[KeyRanges] = None,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
               stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention forward with scored keys.  Shapes, types, ``causal`` and
    ``scale`` as for :func:`~.api.fwd`.  ``softcap`` > 0 caps scores to
    softcap * tanh(x / softcap), softcap at most 4096; ``slopes`` (float32
    [H]) subtracts slopes[h] times the distance between query and key;
    ``window`` > 0 (needs causal) hides keys more than window - 1 positions
    before the query;
    ``key_ranges`` hides keys outside each query's range.  Returns ``(o,
    lse)``; a query that sees no key gets o = 0 and lse = -inf."""
    Z, H, Hkv, Nq, Nk, D = _plain_qkv(q, k, v)
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return fwd_scored(q, k, v, causal, scale, softcap, slopes, window, key_ranges, out, stream)
    handle = _stream(_same_device(q, k, v, slopes), stream)
    slopes_ptr = _check_slopes(slopes, H)
    mask, mask_bytes = _mask_args(key_ranges, q, Z, Nq, Nk)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None and stream is None:
        o, lse = torch.empty_like(q), torch.empty((Z, H, Nq), dtype=torch.float32, device=q.device)
    elif out is None:
        o, lse = _empty_on(stream, q.device, (q.shape, q.dtype), ((Z, H, Nq), torch.float32))
    else:
        o, lse = out
        _check_out(out, ((q.shape, q.dtype), ((Z, H, Nq), torch.float32)), ("o", "lse"))
        _same_device(q, o, lse)
    rc = _native.lib().fa_fwd_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), Z, H, Hkv,
                                     Nq, Nk, D, 1 if causal else 0, scale, _c_cap(softcap), slopes_ptr,
                                     _c_int(window), mask, mask_bytes, _dtype_code(q), handle)
    _native.check(rc, "fa_fwd_scored")
    return o, lse


def bwd_scored(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, do: torch.Tensor,
               lse: torch.Tensor, causal: bool = False, scale: Optional[float] = None, softcap: float = 0.0,
               slopes: Optional[torch.Tensor] = None, window: int = 0, key_ranges: Optional[KeyRanges] = None,
               workspace: Optional[torch.Tensor] = None, out=None, stream: Optional[torch.cuda.Stream] = None
               ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Backward of :func:`fwd_scored` with the same scoring arguments: ``(dq,
    dk, dv)`` shaped like q, k, v.  ``workspace`` as for :func:`~.api.bwd`
    (``bwd_workspace_size`` bytes).  slopes have no gradient."""
    Z, H, Hkv, Nq, Nk, D = _plain_qkv(q, k, v)
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return bwd_scored(q, k, v, o, do, lse, causal, scale, softcap, slopes, window, key_ranges, workspace, out,
                              stream)
    for name, t in (("o", o), ("do", do)):
        _check_input(name, t, q.dtype)
        if t.shape != q.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(q.shape)}")
    if lse.dtype != torch.float32 or lse.shape != (Z, H, Nq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [Z, H, Nq] tensor")
    handle = _stream(_same_device(q, k, v, o, do, lse, slopes, workspace), stream)
    slopes_ptr = _check_slopes(slopes, H)
    mask, mask_bytes = _mask_args(key_ranges, q, Z, Nq, Nk)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    lib = _native.lib()
    if workspace is None:
        need = lib.fa_bwd_ex_workspace_size(Z, H, Hkv, Nq, Nk, D, 1 if causal else 0)
        workspace, = _empty_on(stream, q.device, (max(need, 1), torch.uint8), result=False)
    if out is None and stream is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    elif out is None:
        dq, dk, dv = _empty_on(stream, q.device, *((t.shape, q.dtype) for t in (q, k, v)))
    else:
        dq, dk, dv = out
        _check_out(out, tuple((t.shape, q.dtype) for t in (q, k, v)), ("dq", "dk", "dv"))
        _same_device(q, dq, dk, dv)
    rc = lib.fa_bwd_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                           dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *_workspace(workspace), Z, H, Hkv, Nq, Nk, D,
                           1 if causal else 0, scale, _c_cap(softcap), slopes_ptr, _c_int(window), mask, mask_bytes,
                           _dtype_code(q), handle)
    _native.check(rc, "fa_bwd_scored")
    return dq, dk, dv


def fwd_paged_scored(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                     context_lens: torch.Tensor, q_lens: Optional[torch.Tensor] = None, causal: bool = True,
                     scale: Optional[float] = None, softcap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                     window: int = 0, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                     stream: Optional[torch.cuda.Stream] = None, splits: int = 0,
                     workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Scored attention of a chunk of new tokens per sequence over a paged
    cache.  q [B, H, Nq, D]; caches, block_table and context_lens as for
    :func:`~.api.fwd_paged`; ``q_lens`` int32 [B]: sequence b's first
    q_lens[b] rows are its new tokens, the last of its context (None: all Nq);
    rows behind them, and rows before position 0, get o = 0 and lse = -inf.  Scoring arguments as for
    :func:`fwd_scored`; ``splits`` and ``workspace`` as for ``fwd_paged``
    (0: the library chooses)."""
    _check_input("q", q)
    _check_input("k_cache", k_cache, q.dtype)
    _check_input("v_cache", v_cache, q.dtype)
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return fwd_paged_scored(q, k_cache, v_cache, block_table, context_lens, q_lens, causal, scale, softcap,
                                    slopes, window, out, stream, splits, workspace)
    B, H, Nq, D = q.shape
    num_pages, page_size, Hkv, Dk = k_cache.shape
    if Dk != D or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, Hkv, D] with q's D")
    if Hkv < 1 or H % Hkv != 0:
        raise ValueError(f"q's {H} heads are not a multiple of the cache's {Hkv} heads")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    max_pages = block_table.shape[1]
    _check_int("block_table", block_table, torch.int32, (B, max_pages))
    _check_int("context_lens", context_lens, torch.int32, (B,))
    if q_lens is not None:
        _check_int("q_lens", q_lens, torch.int32, (B,))
    handle = _stream(_same_device(q, k_cache, v_cache, block_table, context_lens, q_lens, slopes, workspace), stream)
    slopes_ptr = _check_slopes(slopes, H)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    lib = _native.lib()
    causal_flag = 1 if causal else 0
    if out is None and stream is None:
        o, lse = torch.empty_like(q), torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    elif out is None:
        o, lse = _empty_on(stream, q.device, (q.shape, q.dtype), ((B, H, Nq), torch.float32))
    else:
        o, lse = out
        _check_out(out, ((q.shape, q.dtype), ((B, H, Nq), torch.float32)), ("o", "lse"))
        _same_device(q, o, lse)
    if splits == 0:
        splits = lib.fa_fwd_paged_scored_split_count(B, H, Hkv, Nq, D, page_size, max_pages, causal_flag)
    splits = _c_int(splits)
    ws_ptr, ws_bytes = None, 0
    if splits != 1:
        if workspace is None:
            need = lib.fa_fwd_paged_split_workspace_size(B, H, Nq, D, splits)
            workspace, = _empty_on(stream, q.device, (max(need, 1), torch.uint8), result=False)
        ws_ptr, ws_bytes = _workspace(workspace)
    rc = lib.fa_fwd_paged_scored(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                                 context_lens.data_ptr(), q_lens.data_ptr() if q_lens is not None else None,
                                 o.data_ptr(), lse.data_ptr(), ws_ptr, ws_bytes, B, H, Hkv, Nq, D, num_pages,
                                 page_size, max_pages, splits, causal_flag, scale, _c_cap(softcap), slopes_ptr,
                                 _c_int(window), _dtype_code(q), handle)
    _native.check(rc, "fa_fwd_paged_scored")
    return o, lse


# ------------------------------------------------------------------ rotary

_pack3 = struct.Struct("3q").pack


def _strides(t: torch.Tensor) -> bytes:
    """The C ABI's array of (sequence, head, token) strides."""
    return _pack3(*t.stride()[:3])


def _check_strided(name: str, t: torch.Tensor, like: Optional[torch.Tensor] = None) -> None:
    if type(t) is torch.Tensor and t.is_cuda and t.dim() == 4 and t.stride(3) == 1:  # the usual case
        if like is not None:
            if t.dtype is like.dtype and t.get_device() == like.get_device():
                return
        elif t.dtype is _HALF or t.dtype is _BF16:
            return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"{name} must be a float16 or bfloat16 CUDA tensor")
    if t.dim() != 4 or (t.stride(3) != 1 and t.numel() > 0):
        raise ValueError(f"{name} must be [Z, heads, N, D] with contiguous rows (any other strides)")
    if like is not None and (t.dtype != like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {like.dtype} on {like.device}")


def _written(name: str, t: torch.Tensor) -> None:
    """An output may not write one value twice: every stride reaches past what
    the smaller ones span."""
    span = 0
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if stride <= span and t.numel() > 0:
            raise ValueError(f"{name} overlaps itself (strides {t.stride()}): an output needs memory of its own for every "
                             "value")
        span += stride * (size - 1)


def _positions(positions: torch.Tensor, q: torch.Tensor) -> int:
    """Checks positions int64 [Z, N] or [N]; returns their sequence stride."""
    Z, _, N, _ = q.shape
    if positions.shape == (N,):
        _check_int("positions", positions, torch.int64, (N,))
        stride = 0
    else:
        _check_int("positions", positions, torch.int64, (Z, N))
        stride = N
    return stride


def _check_freqs(freqs: torch.Tensor, q: torch.Tensor) -> int:
    """Checks freqs; returns the number of values turned."""
    if not isinstance(freqs, torch.Tensor) or freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_cuda \
            or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous float64 CUDA tensor [rot / 2], radians per position")
    rot = 2 * freqs.shape[0]
    if not 0 < rot <= q.shape[3]:
        raise ValueError(f"freqs turn {rot} of a head's {q.shape[3]} values")
    return rot


def _rotary(q, k, positions, freqs, interleaved, mscale, inverse, out, stream):
    _check_strided("q", q)
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return _rotary(q, k, positions, freqs, interleaved, mscale, inverse, out, stream)
    Z, H, N, D = q.shape
    if k is not None:
        _check_strided("k", k, q)
        if (k.shape[0], k.shape[2], k.shape[3]) != (Z, N, D):
            raise ValueError(f"k {tuple(k.shape)} must be [Z, Hkv, N, D] with q's Z, N and D {(Z, N, D)}")
    pos_stride = _positions(positions, q)
    rot = _check_freqs(freqs, q)
    handle = _stream(_same_device(q, positions, freqs), stream)
    if out is None and stream is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        k_out = torch.empty(k.shape, dtype=q.dtype, device=q.device) if k is not None else None
    elif out is None:
        q_out, k_out = (_empty_on(stream, q.device, *((t.shape, q.dtype) for t in (q, k) if t is not None)) + [None])[:2]
    else:
        q_out, k_out = out if k is not None else (out[0] if isinstance(out, Sequence) else out, None)
        for name, t, x in (("out: q", q_out, q), ("out: k", k_out, k)):
            if x is not None:
                _check_strided(name, t, q)
                _written(name, t)
                if t.shape != x.shape:
                    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(x.shape)}")
    has_k = k is not None and k.shape[1] > 0
    rc = _native.lib().fa_rotary(q.data_ptr(), _strides(q), q_out.data_ptr(), _strides(q_out),
                                 k.data_ptr() if has_k else None, _strides(k) if has_k else None,
                                 k_out.data_ptr() if has_k else None, _strides(k_out) if has_k else None,
                                 positions.data_ptr(), pos_stride, freqs.data_ptr(), Z, H, k.shape[1] if has_k else 0,
                                 N, D, rot, 1 if interleaved else 0, 1 if inverse else 0, mscale, _dtype_code(q),
                                 handle)
    _native.check(rc, "fa_rotary")
    return q_out if k is None else (q_out, k_out)


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, freqs: torch.Tensor,
           interleaved: bool = False, mscale: float = 1.0, out=None, stream: Optional[torch.cuda.Stream] = None):
    """Turn q [Z, H, N, D] and k [Z, Hkv, N, D] (or None) by their rotary
    positions.  Both may have any strides with contiguous rows (views of a
    projection's [Z, N, heads, D] output); the results are new contiguous
    tensors, or ``out`` (any strides; the inputs themselves are allowed).
    ``positions`` int64 [Z, N] or [N]; ``freqs`` float64 [rot / 2] (see
    :func:`rotary_freqs`); pairs are (j, j + rot / 2), or (2 j, 2 j + 1) when
    ``interleaved``; values past rot are copied; turned values are multiplied
    by ``mscale``.  Returns ``(q, k)``, or q alone for k None."""
    return _rotary(q, k, positions, freqs, interleaved, mscale, False, out, stream)


def rotary_bwd(dq: torch.Tensor, dk: Optional[torch.Tensor], positions: torch.Tensor, freqs: torch.Tensor,
               interleaved: bool = False, mscale: float = 1.0, out=None,
               stream: Optional[torch.cuda.Stream] = None):
    """Gradients of :func:`rotary`'s inputs from those of its outputs, with
    the same arguments: the turn by the opposite angle."""
    return _rotary(dq, dk, positions, freqs, interleaved, mscale, True, out, stream)


def rotary_and_cache(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, positions: torch.Tensor,
                     freqs: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     interleaved: bool = False, mscale: float = 1.0, out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """:func:`rotary` of q [B, H, N, D] (returned, or written to ``out``), and
    in the same launch the new tokens' turned keys and their values
    ([B, Hkv, N, D], any strides with contiguous rows) into the paged caches
    [num_pages, page_size, Hkv, D] at the slots of ``slot_mapping`` (int64
    [B, N]; negative slots and slots past the cache are skipped; a slot given
    twice ends up with parts of either token)."""
    _check_strided("q", q)
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return rotary_and_cache(q, k_new, v_new, positions, freqs, slot_mapping, k_cache, v_cache, interleaved,
                                    mscale, out, stream)
    B, H, N, D = q.shape
    _check_strided("k_new", k_new, q)
    _check_strided("v_new", v_new, q)
    Bk, Hkv, Nk, Dk = k_new.shape
    if v_new.shape != k_new.shape or Bk != B or Nk != N or Dk != D:
        raise ValueError(f"k_new {tuple(k_new.shape)} and v_new {tuple(v_new.shape)} must be [B, Hkv, N, D] with q's B, "
                         f"N and D {(B, N, D)}")
    _check_input("k_cache", k_cache, q.dtype)
    _check_input("v_cache", v_cache, q.dtype)
    num_pages, page_size, Hc, Dc = k_cache.shape
    if v_cache.shape != k_cache.shape or Hc != Hkv or Dc != D:
        raise ValueError(f"k_cache and v_cache must be [num_pages, page_size, {Hkv}, {D}]")
    pos_stride = _positions(positions, q)
    rot = _check_freqs(freqs, q)
    _check_int("slot_mapping", slot_mapping, torch.int64, (B, N))
    handle = _stream(_same_device(q, k_cache, v_cache, positions, freqs, slot_mapping), stream)
    if out is None and stream is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out is None:
        out, = _empty_on(stream, q.device, (q.shape, q.dtype))
    else:
        _check_strided("out", out, q)
        _written("out", out)
        if out.shape != q.shape:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(q.shape)}")
    rc = _native.lib().fa_rotary_and_cache(q.data_ptr(), _strides(q), out.data_ptr(), _strides(out), k_new.data_ptr(),
                                           _strides(k_new), v_new.data_ptr(), _strides(v_new), positions.data_ptr(),
                                           pos_stride, freqs.data_ptr(), slot_mapping.data_ptr(), k_cache.data_ptr(),
                                           v_cache.data_ptr(), B, H, Hkv, N, D, rot, 1 if interleaved else 0, mscale,
                                           num_pages, page_size, _dtype_code(q), handle)
    _native.check(rc, "fa_rotary_and_cache")
    return out


def rotary_freqs(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                 original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 device="cuda") -> Tuple[torch.Tensor, float]:
    """``(freqs, mscale)`` for :func:`rotary`: freqs[j] = base^(-2 j / rot),
    float64, scaled for contexts ``factor`` times the trained ones:

    * None: unscaled;
    * "linear": every frequency divided by factor;
    * "ntk": base multiplied by factor^(rot / (rot - 2)), which divides the
      lowest frequency by factor and leaves the highest;
    * "yarn": frequencies that turn less than beta_slow times within
      ``original_len`` positions are divided by factor, those that turn more
      than beta_fast times are kept, with a linear ramp over j in between;
      mscale = 0.1 ln(factor) + 1.

    mscale is 1 for the others."""
    if rot <= 0 or rot % 2 != 0 or not base > 1.0 or not factor >= 1.0:
        raise ValueError("rotary_freqs needs an even rot > 0, base > 1 and factor >= 1")
    if scaling == "ntk":
        if rot < 4:
            raise ValueError("ntk scaling needs rot >= 4")
        base = base * factor ** (rot / (rot - 2))
    j = torch.arange(0, rot, 2, dtype=torch.float64)
    freqs = torch.pow(torch.tensor(base, dtype=torch.float64), -j / rot)
    mscale = 1.0
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "yarn":
        if original_len <= 0:
            raise ValueError("yarn scaling needs original_len")

        def pair_of(turns: float) -> float:  # the (fractional) pair that turns so often within original_len
            return rot * math.log(original_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        # the ramp's ends; the last may lie behind the last pair, which is on the ramp then
        low, high = max(math.floor(pair_of(beta_fast)), 0), math.ceil(pair_of(beta_slow))
        pair = torch.arange(rot // 2, dtype=torch.float64)
        ramp = ((pair - low) / (high - low)).clamp(0.0, 1.0) if high > low else (pair >= high).double()
        freqs = freqs * (1.0 - ramp) + freqs / factor * ramp
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}: None, 'linear', 'ntk' or 'yarn'")
    return freqs.to(device), mscale
