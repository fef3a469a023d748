"""Python binding of libattn_b200.so (exact, IO-aware attention on B200).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of the shared library.  PyTorch supplies device memory and streams.
There is no fallback: if the library is missing or a call fails, an
exception is raised.

Entry points mirror include/attn.h:

    attn_fwd(q, k, v, ...)            prefill, [B, N, H, d] tensors
    attn_decode(q, k_cache, v_cache, seqlens, ...)
    attn_decode_multi(q, k_cache, v_cache, seqlens, ...)
    attn_bwd(q, k, v, o, lse, dout, ...)
    key_stats(k), attn_fwd_bound(q, k, v, kbar, radius, ...)
    rope(q, k, positions, axes, freq, ...)
    kv4_pool(...), kv4_append(k, v, pool, table, seqlens, ...), kv4_read(...)
    attn_decode_kv4(q, pool, table, seqlens, ...)
    copy_pages(pool, src, dst)
    frame_block_map(n_frames, frame_len)
    classify(mask_kind, block_map, Nq, Nkv, tq, tk)
    plan(mask_kind, block_map, Nq, Nkv)
    sync_status(stream=None)

Above these: exact_io_aware_sm_b200.autograd.attention (the differentiable op,
attn_fwd forward and attn_bwd backward; rope there is differentiable too),
exact_io_aware_sm_b200.kv4_cache (the pages of a 4-bit cache: sequences added,
extended, forked, freed and compacted) and exact_io_aware_sm_b200.ulysses
(sequence-parallel forward, backward and differentiable op over
torch.distributed).

The C ABI takes plain pointers and cannot see buffer sizes, so every tensor
and block map is checked here (device, contiguity, dtype, shape) before a
pointer is passed: a mis-shaped output or map raises ValueError instead of
being written or read past its end.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libattn_b200.so")

ATTN_OK = 0
STATUS_NAMES = {
    0: "ATTN_OK", 1: "ATTN_ERR_NULL", 2: "ATTN_ERR_SHAPE", 3: "ATTN_ERR_ALIGN",
    4: "ATTN_ERR_UNSUPPORTED", 5: "ATTN_ERR_MASK", 6: "ATTN_ERR_CUDA",
    7: "ATTN_ERR_DEVICE_TIMEOUT", 8: "ATTN_ERR_WORKSPACE", 9: "ATTN_ERR_DEVICE_ARG",
}
MASK_NONE, MASK_CAUSAL, MASK_BLOCK = 0, 1, 2
BF16, F32 = 0, 1

_lib = None


class AttnError(RuntimeError):
    def __init__(self, code: int, detail: str):
        self.code = code
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {detail}")


def lib() -> ctypes.CDLL:
    """Load libattn_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m exact_io_aware_sm_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, P, I, P]
        L.attn_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, P]
        L.attn_decode_multi.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, P]
        L.attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, P]
        L.attn_frame_block_map.argtypes = [I, I, P]
        L.attn_classify.argtypes = [I, P, I, I, I, I, P]
        L.attn_plan.argtypes = [I, P, I, I, P, I, P, I, P, P]
        L.attn_sync_status.argtypes = [P]
        L.attn_last_error_detail.argtypes = [ctypes.c_char_p, I]
        L.attn_shutdown.argtypes = []
        L.attn_debug_fault.argtypes = [I]
        L.attn_key_stats.argtypes = [P, P, P, I, I, I, I, P]
        L.attn_fwd_bound.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, P, P, P, P, P]
        D = ctypes.c_int64
        L.attn_rope.argtypes = [P] * 8 + [I] * 10 + [P]
        L.attn_kv4_append.argtypes = [P] * 7 + [I] * 7 + [P]
        L.attn_kv4_read.argtypes = [P] * 6 + [I] * 7 + [P]
        L.attn_decode_kv4.argtypes = [P] * 7 + [D] + [I] * 8 + [F, P]
        L.attn_decode_kv4_workspace.argtypes = [I] * 7
        L.attn_decode_kv4_workspace.restype = D
        L.attn_copy_pages.argtypes = [P, D, I, P, P, I, P]
        L.attn_version.restype = ctypes.c_char_p
        for fn in (L.attn_fwd, L.attn_decode, L.attn_decode_multi, L.attn_bwd, L.attn_frame_block_map,
                   L.attn_classify, L.attn_plan, L.attn_key_stats, L.attn_fwd_bound, L.attn_rope,
                   L.attn_kv4_append, L.attn_kv4_read, L.attn_decode_kv4, L.attn_copy_pages,
                   L.attn_sync_status, L.attn_last_error_detail, L.attn_shutdown, L.attn_debug_fault):
            fn.restype = I
        _lib = L
    return _lib


def last_error() -> str:
    buf = ctypes.create_string_buffer(512)
    lib().attn_last_error_detail(buf, 512)
    return buf.value.decode()


def _check(rc: int) -> None:
    if rc != ATTN_OK:
        raise AttnError(rc, last_error())


def _np_ptr(a):
    return None if a is None else a.ctypes.data_as(ctypes.c_void_p)


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _bm(block_map, Nq=None, Nkv=None):
    """The block map as a contiguous uint8 array of ceil(Nq/16) x ceil(Nkv/16)
    (the size the library reads), or None."""
    if block_map is None:
        return None
    bm = np.ascontiguousarray(block_map, dtype=np.uint8)
    if Nq is not None:
        want = ((Nq + 15) // 16, (Nkv + 15) // 16)
        if bm.shape != want:
            raise ValueError(f"block_map has shape {bm.shape}; Nq={Nq}, Nkv={Nkv} need {want}")
    return bm


def _need(t, name, shape, dtypes, device=None):
    """Check a tensor handed to the library: a contiguous CUDA tensor of one
    of the given dtypes whose shape matches `shape` (None entries match any
    size), on `device` if given, else (the call's first tensor) on the
    current CUDA device, where the library launches."""
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}; expected {' or '.join(str(d) for d in dtypes)}")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        want = tuple("*" if w is None else w for w in shape)
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {want}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}; expected {device}")
    if device is None:  # the call's first tensor: the library runs on the current device
        import torch
        cur = torch.cuda.current_device()
        if t.device.index is not None and t.device.index != cur:
            raise ValueError(f"{name} is on {t.device} but the current CUDA device is {cur}; "
                             f"call inside torch.cuda.device({t.device.index})")


def attn_fwd(q, k, v, o=None, lse=None, scale=None, mask_kind=MASK_NONE, block_map=None,
             stream=None, want_lse=True):
    """Prefill attention.  q [B,Nq,Hq,d], k/v [B,Nkv,Hkv,d] CUDA tensors
    (bf16, or fp32 for the exact fp32 path).  Returns (o, lse) with o like q
    and lse fp32 [B,Hq,Nq] (None if want_lse is False and lse is None)."""
    import torch
    _need(q, "q", (None,) * 4, (torch.bfloat16, torch.float32))
    B, Nq, Hq, d = q.shape
    _need(k, "k", (B, None, None, d), (q.dtype,), q.device)
    Nkv, Hkv = k.shape[1], k.shape[2]
    _need(v, "v", k.shape, (q.dtype,), q.device)
    dt = BF16 if q.dtype == torch.bfloat16 else F32
    if o is None:
        o = torch.empty_like(q)
    _need(o, "o", q.shape, (q.dtype,), q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", (B, Hq, Nq), (torch.float32,), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    bm = _bm(block_map, Nq, Nkv)
    _check(lib().attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                          None if lse is None else lse.data_ptr(), B, Hq, Hkv, Nq, Nkv, d,
                          float(scale), mask_kind, _np_ptr(bm), dt, _stream_ptr(stream)))
    return o, lse


def key_stats(k, kbar=None, radius=None, stream=None):
    """Key statistics for the bound-based softmax: kbar fp32 [B,Hkv,d] (mean
    key) and radius fp32 [B,Hkv] (largest centred key norm) of a bf16
    k [B,Nkv,Hkv,d] CUDA tensor."""
    import torch
    _need(k, "k", (None,) * 4, (torch.bfloat16,))
    B, Nkv, Hkv, d = k.shape
    if kbar is None:
        kbar = torch.empty((B, Hkv, d), dtype=torch.float32, device=k.device)
    if radius is None:
        radius = torch.empty((B, Hkv), dtype=torch.float32, device=k.device)
    _need(kbar, "kbar", (B, Hkv, d), (torch.float32,), k.device)
    _need(radius, "radius", (B, Hkv), (torch.float32,), k.device)
    _check(lib().attn_key_stats(k.data_ptr(), kbar.data_ptr(), radius.data_ptr(), B, Nkv, Hkv, d,
                                _stream_ptr(stream)))
    return kbar, radius


def attn_fwd_bound(q, k, v, kbar, radius, o=None, lse=None, scale=None, mask_kind=MASK_NONE, block_map=None,
                   n_fallback=None, stream=None):
    """attn_fwd (bf16) with the bound-based softmax; kbar, radius from
    key_stats(k).  n_fallback: optional int32 CUDA tensor of one element to
    which the number of rows that kept the running max is added.
    Returns (o, lse)."""
    import torch
    _need(q, "q", (None,) * 4, (torch.bfloat16,))
    B, Nq, Hq, d = q.shape
    _need(k, "k", (B, None, None, d), (torch.bfloat16,), q.device)
    Nkv, Hkv = k.shape[1], k.shape[2]
    _need(v, "v", k.shape, (torch.bfloat16,), q.device)
    _need(kbar, "kbar", (B, Hkv, d), (torch.float32,), q.device)
    _need(radius, "radius", (B, Hkv), (torch.float32,), q.device)
    if n_fallback is not None:
        _need(n_fallback, "n_fallback", (1,), (torch.int32,), q.device)
    if o is None:
        o = torch.empty_like(q)
    _need(o, "o", q.shape, (torch.bfloat16,), q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    _need(lse, "lse", (B, Hq, Nq), (torch.float32,), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    bm = _bm(block_map, Nq, Nkv)
    _check(lib().attn_fwd_bound(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hkv,
                                Nq, Nkv, d, float(scale), mask_kind, _np_ptr(bm), kbar.data_ptr(), radius.data_ptr(),
                                None if n_fallback is None else n_fallback.data_ptr(), _stream_ptr(stream)))
    return o, lse


def _check_cache(k_cache, v_cache, seqlens, B, d, device):
    import torch
    _need(k_cache, "k_cache", (B, None, None, d),
          (torch.bfloat16,), device)
    _need(v_cache, "v_cache", k_cache.shape, (torch.bfloat16,), device)
    _need(seqlens, "seqlens", (B,), (torch.int32,), device)


def attn_decode(q, k_cache, v_cache, seqlens, o=None, lse=None, scale=None, stream=None,
                want_lse=True):
    """Single-token decode.  q [B,Hq,d] bf16; caches [B,Lmax,Hkv,d] bf16;
    seqlens int32 [B] on the device."""
    import torch
    _need(q, "q", (None,) * 3, (torch.bfloat16,))
    B, Hq, d = q.shape
    _check_cache(k_cache, v_cache, seqlens, B, d, q.device)
    Lmax, Hkv = k_cache.shape[1], k_cache.shape[2]
    if o is None:
        o = torch.empty_like(q)
    _need(o, "o", q.shape, (torch.bfloat16,), q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", (B, Hq), (torch.float32,), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(lib().attn_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), seqlens.data_ptr(),
                             o.data_ptr(), None if lse is None else lse.data_ptr(), B, Hq, Hkv, Lmax,
                             d, float(scale), _stream_ptr(stream)))
    return o, lse


def attn_decode_multi(q, k_cache, v_cache, seqlens, o=None, lse=None, scale=None, stream=None,
                      want_lse=True):
    """Decode of the Sq newest tokens per sequence.  q [B,Sq,Hq,d] bf16;
    caches [B,Lmax,Hkv,d] bf16; seqlens int32 [B] on the device (including
    the Sq new tokens).  Returns o [B,Sq,Hq,d] and lse [B,Hq,Sq]."""
    import torch
    _need(q, "q", (None,) * 4, (torch.bfloat16,))
    B, Sq, Hq, d = q.shape
    _check_cache(k_cache, v_cache, seqlens, B, d, q.device)
    Lmax, Hkv = k_cache.shape[1], k_cache.shape[2]
    if o is None:
        o = torch.empty_like(q)
    _need(o, "o", q.shape, (torch.bfloat16,), q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", (B, Hq, Sq), (torch.float32,), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(lib().attn_decode_multi(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), seqlens.data_ptr(),
                                   o.data_ptr(), None if lse is None else lse.data_ptr(), B, Sq, Hq, Hkv,
                                   Lmax, d, float(scale), _stream_ptr(stream)))
    return o, lse


def _on(stream):
    """The context that makes `stream` the current one, so that a call's outputs and workspace
    belong to the stream it runs on (their memory is not reused while it runs)."""
    import torch
    if stream.device_index != torch.cuda.current_device():
        raise ValueError(f"stream is on device {stream.device_index} but the current CUDA device is "
                         f"{torch.cuda.current_device()}")
    return torch.cuda.stream(stream)


def _stream_here(device):
    """The current stream of the current device as an integer handle."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device)


def _is(t, shape, dtype, device):
    """Whether a tensor is what the library takes; the calls below ask this first and _need, which
    says what is wrong, only where it is not (small calls are bound by the host)."""
    return t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device


def _device_of(t, name):
    """The current device, on which the call's first tensor has to be."""
    import torch
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a CUDA tensor")
    device, cur = t.get_device(), torch.cuda.current_device()
    if device != cur:
        raise ValueError(f"{name} is on {t.device} but the current CUDA device is {cur}; "
                         f"call inside torch.cuda.device({device})")
    return device


def _rows(t, name, shape, dtype, device):
    """Check a [B, N, H, d] tensor whose heads and channels are contiguous but whose batch and
    token strides are free (a part of a fused projection); returns those two strides (0 for
    dimensions of one element)."""
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}; expected cuda:{device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}; expected {dtype}")
    if t.dim() != 4 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape or ('*',) * 4)}")
    B, N, H, d = t.shape
    sb, sn, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (H > 1 and sh != d):
        raise ValueError(f"{name} must have contiguous heads and channels (strides {t.stride()})")
    return (sb if B > 1 else 0), (sn if N > 1 else 0)


def _extent(t):
    """First and one-past-last byte address of a tensor's elements."""
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _apart(out, name, others):
    """Refuse an output [B,N,H,d] that repeats its own rows, or that overlaps one of
    `others` (tensor, may it be that very tensor).  Rows of one fused buffer, side by side
    at the same strides, do not overlap."""
    B, N, H, d = out.shape
    e, row = out.element_size(), H * d
    dims = sorted((s, n) for s, n in ((out.stride(0), B), (out.stride(1), N)) if n > 1)
    span = row
    for s, n in dims:
        if s < span:
            raise ValueError(f"{name} must not repeat elements (strides {out.stride()})")
        span = (n - 1) * s + span
    lo, hi = _extent(out)
    for t, same in others:
        if same and t.data_ptr() == out.data_ptr() and t.shape == out.shape and t.stride() == out.stride():
            continue
        a, b = _extent(t)
        if a >= hi or lo >= b:
            continue
        if dims and t.dim() == 4 and t.shape[:2] == out.shape[:2] and t.stride()[:2] == out.stride()[:2]:
            step = dims[0][0] * e
            r = (a - lo) % step
            if all(s * e % step == 0 for s, _ in dims) and r >= row * e and step - r >= t.shape[2] * d * e:
                continue
        raise ValueError(f"{name} overlaps another tensor of the call")


def _like(t):
    """A contiguous tensor of t's shape and type."""
    import torch
    return torch.empty_like(t) if t.is_contiguous() else torch.empty_like(t, memory_format=torch.contiguous_format)


def _axes(axes):
    """Axis numbers as a uint8 array, refused where that would change them."""
    axes = np.asarray(axes)
    if axes.dtype == np.uint8:
        return axes
    if axes.size and (not np.issubdtype(axes.dtype, np.integer) or axes.min() < 0 or axes.max() > 255):
        raise ValueError(f"axes must be axis numbers, got {axes.dtype} from {axes.min()} to {axes.max()}")
    return axes.astype(np.uint8)


_PACK10, _PACK4 = struct.Struct("10q").pack, struct.Struct("4q").pack  # strides, as the library reads them


def rope(q, k, positions, axes, freq, interleaved=False, inverse=False, q_out=None, k_out=None, stream=None):
    """Rotary positions with several axes.  q [B,N,Hq,d], k [B,N,Hk,d] (or None), bf16 or
    fp32; positions int32 [B,N,A] (or [N,A] for every sequence); axes and freq: host
    arrays of n <= d/2 entries, pair p turning by positions[..., axes[p]] * freq[p].
    Pair p is channels (p, p + d/2), or (2p, 2p + 1) if interleaved; channels without an
    entry are copied.  inverse rotates back.  q and k may have any batch and token
    strides of whole 16 bytes; q_out may be q, and k_out k.  Returns (q_out, k_out)."""
    import torch
    if stream is not None:
        with _on(stream):
            return rope(q, k, positions, axes, freq, interleaved, inverse, q_out, k_out)
    dev, dtype = _device_of(q, "q"), q.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"q has dtype {dtype}; expected torch.bfloat16 or torch.float32")
    qb, qn = _rows(q, "q", None, dtype, dev)
    B, N, Hq, d = q.shape
    kb = kn = kob = kon = Hk = 0
    if k is not None:
        Hk = k.shape[2] if k.dim() == 4 else 0
        kb, kn = _rows(k, "k", (B, N, Hk, d), dtype, dev)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if not q.numel() or (k is not None and not Hk):
        raise ValueError(f"q and k must not be empty, got {tuple(q.shape)}" + ("" if k is None else f" and {tuple(k.shape)}"))
    axes = _axes(axes)
    freq = np.asarray(freq, dtype=np.float64)
    if axes.ndim != 1 or axes.shape != freq.shape:
        raise ValueError(f"axes and freq must be vectors of one length, got {axes.shape} and {freq.shape}")
    if not (getattr(positions, "is_cuda", False) and positions.dtype is torch.int32 and positions.get_device() == dev):
        raise ValueError(f"positions must be an int32 tensor on cuda:{dev}")
    if positions.dim() == 2:
        positions = positions.expand(B, *positions.shape)
    if positions.dim() != 3 or positions.shape[0] != B or positions.shape[1] != N:
        raise ValueError(f"positions has shape {tuple(positions.shape)}; expected ({B}, {N}, *) or ({N}, *)")
    A = positions.shape[2]
    pb, pn, pa = positions.stride()
    if A > 1 and pa != 1:
        raise ValueError("positions must be contiguous in its last dimension")
    if q_out is None:
        q_out = _like(q)
        qob, qon = N * Hq * d, Hq * d
    else:
        qob, qon = _rows(q_out, "q_out", (B, N, Hq, d), dtype, dev)
        _apart(q_out, "q_out", [(q, True), (positions, False)] + ([] if k is None else [(k, False)]))
    if k is not None:
        if k_out is None:
            k_out = _like(k)
            kob, kon = N * Hk * d, Hk * d
        else:
            kob, kon = _rows(k_out, "k_out", (B, N, Hk, d), dtype, dev)
            _apart(k_out, "k_out", [(k, True), (q, False), (q_out, False), (positions, False)])
    strides = _PACK10(qb, qn, kb, kn, qob, qon, kob, kon, pb if B > 1 else 0, pn if N > 1 else 0)
    rc = lib().attn_rope(q.data_ptr(), None if k is None else k.data_ptr(), q_out.data_ptr(),
                         None if k is None else k_out.data_ptr(), positions.data_ptr(), axes.tobytes(),
                         freq.tobytes(), strides, B, N, Hq, Hk, d, A, len(axes), bool(interleaved), bool(inverse),
                         BF16 if dtype is torch.bfloat16 else F32, _stream_here(dev))
    if rc:
        _check(rc)
    return q_out, k_out


def kv4_page_bytes(page, Hkv, d):
    """Bytes of a page of `page` tokens (16, 32, 64, 128 or 256): K and V codes and scales of every KV head."""
    if page not in (16, 32, 64, 128, 256) or d not in (64, 128):
        raise ValueError(f"page must be 16, 32, 64, 128 or 256 (got {page}) and d 64 or 128 (got {d})")
    return page // 16 * 18 * d * Hkv


def kv4_pool(n_pages, Hkv, d, page=64, device=None):
    """An empty pool of a 4-bit cache: uint8 [n_pages, Hkv, page/16 * 18 d] (uninitialised)."""
    import torch
    return torch.empty((n_pages, Hkv, kv4_page_bytes(page, 1, d)), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def _kv4(pool, table, seqlens, B, Hkv, d, device):
    """Check a pool, page table and lengths; returns (n_pages, Hkv, page, max_pages)."""
    import torch
    u8, i32 = torch.uint8, torch.int32
    if pool.dim() == 3 and table.dim() == 2:
        n_pages, heads, nbytes = pool.shape
        rows, max_pages = table.shape
        ok = (_is(pool, (n_pages, heads, nbytes), u8, device) and _is(table, (rows, max_pages), i32, device)
              and _is(seqlens, (rows,), i32, device))
    if pool.dim() != 3 or table.dim() != 2 or not ok or (B or rows) != rows or (Hkv or heads) != heads:
        dev = torch.device("cuda", device)
        _need(pool, "pool", (None, Hkv, None), (u8,), dev)
        _need(table, "table", (B, None), (i32,), dev)
        _need(seqlens, "seqlens", (table.shape[0],), (i32,), dev)
    if d not in (64, 128):
        raise ValueError(f"the 4-bit cache needs d in (64, 128), got {d}")
    page = nbytes // (18 * d) * 16
    if page not in (16, 32, 64, 128, 256) or nbytes != page // 16 * 18 * d:
        raise ValueError(f"pool has {nbytes} bytes a page and head: no page of 16, 32, 64, 128 or 256 tokens at d = {d}")
    return n_pages, heads, page, max_pages


def _counts(t, name, B, device):
    """The address of an optional int32 [B] on the device."""
    import torch
    if t is None:
        return None
    if not _is(t, (B,), torch.int32, device):
        _need(t, name, (B,), (torch.int32,), torch.device("cuda", device))
    return t.data_ptr()


def kv4_append(k, v, pool, table, seqlens, n_new=None, stream=None):
    """Quantise k, v [B,N,Hkv,d] bf16 (any batch and token strides of whole 16 bytes) and
    write them into the pages of pool (kv4_pool) that table int32 [B,max_pages] names, as
    tokens seqlens[b] - n_new[b] .. seqlens[b] - 1; n_new int32 [B] (None: N each), rows
    behind it are padding.  Nothing else in the pool changes.  The page size follows from the
    pool's bytes and d, so d has to be the pool's (Kv4Cache checks it).  Returns pool."""
    import torch
    if stream is not None:
        with _on(stream):
            return kv4_append(k, v, pool, table, seqlens, n_new)
    dev = _device_of(k, "k")
    kb, kn = _rows(k, "k", None, torch.bfloat16, dev)
    B, N, Hkv, d = k.shape
    vb, vn = _rows(v, "v", (B, N, Hkv, d), torch.bfloat16, dev)
    n_pages, _, page, max_pages = _kv4(pool, table, seqlens, B, Hkv, d, dev)
    rc = lib().attn_kv4_append(k.data_ptr(), v.data_ptr(), pool.data_ptr(), table.data_ptr(), seqlens.data_ptr(),
                               _counts(n_new, "n_new", B, dev), _PACK4(kb, kn, vb, vn), B, N, Hkv, d, n_pages, page,
                               max_pages, _stream_here(dev))
    if rc:
        _check(rc)
    return pool


def kv4_read(pool, table, seqlens, N, d, start=None, k=None, v=None, stream=None):
    """Tokens start[b] .. start[b] + N - 1 (start int32 [B]; None: 0) of each sequence of a
    4-bit cache as bf16 k, v [B,N,Hkv,d]; rows at and past seqlens[b] are zeros."""
    import torch
    if stream is not None:
        with _on(stream):
            return kv4_read(pool, table, seqlens, N, d, start, k, v)
    dev = _device_of(pool, "pool")
    n_pages, Hkv, page, max_pages = _kv4(pool, table, seqlens, None, None, d, dev)
    B = table.shape[0]
    shape, bf16 = (B, N, Hkv, d), torch.bfloat16
    if k is None:
        k = pool.new_empty(shape, dtype=bf16)
    elif not _is(k, shape, bf16, dev):
        _need(k, "k", shape, (bf16,), pool.device)
    if v is None:
        v = torch.empty_like(k)
    elif not _is(v, shape, bf16, dev):
        _need(v, "v", shape, (bf16,), pool.device)
    rc = lib().attn_kv4_read(k.data_ptr(), v.data_ptr(), pool.data_ptr(), table.data_ptr(), seqlens.data_ptr(),
                             _counts(start, "start", B, dev), B, N, Hkv, d, n_pages, page, max_pages,
                             _stream_here(dev))
    if rc:
        _check(rc)
    return k, v


@functools.lru_cache(maxsize=256)
def _decode_kv4_workspace(*sizes):
    return max(0, lib().attn_decode_kv4_workspace(*sizes))  # -1: refused sizes, which the call itself reports


def attn_decode_kv4(q, pool, table, seqlens, o=None, lse=None, scale=None, stream=None, want_lse=True):
    """Decode of the Sq newest tokens per sequence over a 4-bit paged cache.  q
    [B,Sq,Hq,d] bf16; pool from kv4_pool; table int32 [B,max_pages]; seqlens int32 [B]
    on the device (including the Sq new tokens).  Returns o [B,Sq,Hq,d] and lse [B,Hq,Sq]."""
    import torch
    if stream is not None:
        with _on(stream):
            return attn_decode_kv4(q, pool, table, seqlens, o, lse, scale, None, want_lse)
    dev, bf16 = _device_of(q, "q"), torch.bfloat16
    if q.dim() != 4 or not _is(q, q.shape, bf16, dev):
        _need(q, "q", (None,) * 4, (bf16,))
    B, Sq, Hq, d = shape = q.shape
    n_pages, Hkv, page, max_pages = _kv4(pool, table, seqlens, B, None, d, dev)
    if o is None:
        o = torch.empty_like(q)
    elif not _is(o, shape, bf16, dev):
        _need(o, "o", shape, (bf16,), q.device)
    if lse is None:
        if want_lse:
            lse = q.new_empty((B, Hq, Sq), dtype=torch.float32)
    elif not _is(lse, (B, Hq, Sq), torch.float32, dev):
        _need(lse, "lse", (B, Hq, Sq), (torch.float32,), q.device)
    n = _decode_kv4_workspace(B, Sq, Hq, Hkv, d, page, max_pages)
    work = pool.new_empty(n) if n else None
    rc = lib().attn_decode_kv4(q.data_ptr(), pool.data_ptr(), table.data_ptr(), seqlens.data_ptr(), o.data_ptr(),
                               None if lse is None else lse.data_ptr(), None if work is None else work.data_ptr(), n,
                               B, Sq, Hq, Hkv, d, n_pages, page, max_pages,
                               1.0 / math.sqrt(d) if scale is None else float(scale), _stream_here(dev))
    if rc:
        _check(rc)
    return o, lse


def copy_pages(pool, src, dst, stream=None):
    """Copy pages src[i] of a pool to pages dst[i].  pool: a contiguous CUDA tensor of
    equal pages along its first dimension; src, dst: host int arrays.  A source may
    repeat; no page may be a destination twice, or source and destination.  Returns pool."""
    if stream is not None:
        with _on(stream):
            return copy_pages(pool, src, dst)
    dev = _device_of(pool, "pool")
    if not pool.numel() or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous tensor of at least one page")
    n_pages = len(pool)
    src, dst = np.asarray(src), np.asarray(dst)
    if src.ndim != 1 or src.shape != dst.shape:
        raise ValueError(f"src and dst must be vectors of one length, got {src.shape} and {dst.shape}")
    n = len(src)
    for name, x in (("src", src), ("dst", dst)):
        if n and x.dtype != np.int32:
            if not np.issubdtype(x.dtype, np.integer):
                raise ValueError(f"{name} must hold integers, got {x.dtype}")
            if x.min() < 0 or x.max() >= n_pages:
                raise ValueError(f"{name} names a page outside the pool of {n_pages} pages")
    rc = lib().attn_copy_pages(pool.data_ptr(), pool.numel() // n_pages * pool.element_size(), n_pages,
                               src.astype(np.int32, copy=False).tobytes(), dst.astype(np.int32, copy=False).tobytes(),
                               n, _stream_here(dev))
    if rc:
        _check(rc)
    return pool


def attn_bwd(q, k, v, o, lse, dout, scale=None, mask_kind=MASK_NONE, block_map=None, stream=None):
    """Gradients of attn_fwd (bf16): q, o, dout [B,Nq,Hq,d]; k, v [B,Nkv,Hkv,d];
    lse [B,Hq,Nq] fp32 from the forward; the mask as for attn_fwd.
    Returns (dq, dk, dv) like q, k, v."""
    import torch
    _need(q, "q", (None,) * 4, (torch.bfloat16,))
    B, Nq, Hq, d = q.shape
    _need(k, "k", (B, None, None, d), (torch.bfloat16,), q.device)
    Nkv, Hkv = k.shape[1], k.shape[2]
    _need(v, "v", k.shape, (torch.bfloat16,), q.device)
    _need(o, "o", q.shape, (torch.bfloat16,), q.device)
    _need(dout, "dout", q.shape, (torch.bfloat16,), q.device)
    _need(lse, "lse", (B, Hq, Nq), (torch.float32,), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    bm = _bm(block_map, Nq, Nkv)
    _check(lib().attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Nq, Nkv, d, float(scale),
                          mask_kind, _np_ptr(bm), _stream_ptr(stream)))
    return dq, dk, dv


def frame_block_map(n_frames: int, frame_len: int) -> np.ndarray:
    nb = (n_frames * frame_len + 15) // 16
    out = np.zeros((nb, nb), np.uint8)
    _check(lib().attn_frame_block_map(n_frames, frame_len, _np_ptr(out)))
    return out


def classify(mask_kind, block_map, Nq, Nkv, tq, tk) -> np.ndarray:
    out = np.zeros(((Nq + tq - 1) // tq, (Nkv + tk - 1) // tk), np.uint8)
    bm = _bm(block_map, Nq, Nkv)
    _check(lib().attn_classify(mask_kind, _np_ptr(bm), Nq, Nkv, tq, tk, _np_ptr(out)))
    return out


def plan(mask_kind, block_map, Nq, Nkv):
    """The tile schedule attn_fwd runs: (qtiles [n,4], kvtiles [m,3]) int32."""
    bm = _bm(block_map, Nq, Nkv)
    nq, nk = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().attn_plan(mask_kind, _np_ptr(bm), Nq, Nkv, None, 0, None, 0,
                           ctypes.byref(nq), ctypes.byref(nk)))
    qt = np.zeros((nq.value, 4), np.int32)
    kt = np.zeros((nk.value, 3), np.int32)
    _check(lib().attn_plan(mask_kind, _np_ptr(bm), Nq, Nkv, _np_ptr(qt), nq.value, _np_ptr(kt),
                           nk.value, ctypes.byref(nq), ctypes.byref(nk)))
    return qt, kt


def sync_status(stream=None) -> None:
    """Synchronise the stream and raise if a kernel latched a device error."""
    _check(lib().attn_sync_status(_stream_ptr(stream)))


def debug_fault(kind: int) -> None:
    """Test hook: kind 1 makes the next bf16 attn_fwd on this thread run one
    bounded wait out, so that its sync_status raises ATTN_ERR_DEVICE_TIMEOUT."""
    _check(lib().attn_debug_fault(kind))


def shutdown() -> None:
    lib().attn_shutdown()


def version() -> str:
    return lib().attn_version().decode()
