"""The prompt operators on torch tensors (``include/tre.h``, operators of the prompt path).

Each function checks its tensors, allocates what it returns with torch (on the current
stream, so it may be captured in a CUDA graph), and enqueues the native kernel on torch's
current stream of the tensors' device.  What a C caller could get wrong too raises
``tre.TreError``; a tensor of another type, device or shape raises ``ValueError``.  The
operators have no derivatives: an input that requires a gradient is refused while gradients
are recorded, one with a forward-mode gradient always.

The attention and the product bound their waits on the device.  One that runs out of time
(about two seconds: another program holds the GPU, or a fault of the kernel) leaves the
call's outputs unspecified; no later call raises for it.  ``tre.tre_ops_status()`` waits for
the current device, returns ``tre.TRE_ERR_DEP_TIMEOUT`` if that has happened since it was last
asked, and 0 otherwise: ask before results are relied on.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad

from . import tre
from .synth import mxfp4_pitch

_TYPES = {torch.bfloat16: tre.TRE_BF16, torch.float32: tre.TRE_F32}


# torch.cuda.current_stream(d).cuda_stream without the Stream object (3 us of a 10 us call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_SMS = {}  # device index -> SM count


def _tensor(t, name: str, ndim: int, dtypes, device=None) -> None:
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.ndim != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, not {t.ndim}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has type {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.stride(-1) != 1 and t.shape[-1] != 1 and t.numel():
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient: the operator has no backward pass")
    # (the level first: asking a tensor costs 0.4 us, and a program without forward mode has none)
    if getattr(forward_ad, "_current_level", 0) >= 0 and \
            forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError(f"{name} has a forward-mode gradient: the operator has no derivative")


def _span(t) -> Tuple[int, int]:
    """The bytes [first, last) that the tensor's elements lie in."""
    if t.numel() == 0:
        return 0, 0
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _apart(out, name: str, /, **inputs) -> None:
    a, b = _span(out)
    for key, t in inputs.items():
        if t is not None:
            c, d = _span(t)
            if c < b and a < d:
                raise ValueError(f"{name} may not overlap {key}")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _call(fn, device, *args) -> None:
    """fn(*args, current stream) with `device` current."""
    stream = _raw_stream(device.index)
    if device.index == torch.cuda.current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != tre.TRE_OK:
        raise tre.TreError(status, fn.__name__)


def _sms(device) -> int:
    n = _SMS.get(device.index)
    if n is None:
        n = _SMS[device.index] = torch.cuda.get_device_properties(device).multi_processor_count
    return n


def _offsets(t, name: str, device) -> None:
    _tensor(t, name, 1, (torch.int32,), device)
    if t.numel() < 2:
        raise ValueError(f"{name} must have at least 2 entries")


def prompt_attention(q, k, v, q_offsets=None, kv_offsets=None, scale: Optional[float] = None,
                     out=None):
    """Causal attention of packed prompts; returns ``out`` [T, Hq, D] bf16.

    q [T, Hq, D], k and v [Hkv, S, D] bf16 in any strides of whole 16-byte units whose last
    dimension is contiguous: an engine's cache ``k_cache[:, :pos + T]`` as it is, packed rows
    [S, Hkv, D] as ``k.transpose(0, 1)``.  D is 64 or 128 and Hq a multiple of Hkv.
    q_offsets, kv_offsets: int32 [n + 1] on the device, the rows of each of n sequences (read
    when the kernel runs); both None: one sequence.  The last query row of a sequence sees
    its last key row; a row that sees no key is zero; rows of no sequence are left as they
    are in ``out`` (unwritten in an ``out`` that the call allocates).
    scale: 1 / sqrt(D) when None."""
    _tensor(q, "q", 3, (torch.bfloat16,))
    _tensor(k, "k", 3, (torch.bfloat16,), q.device)
    _tensor(v, "v", 3, (torch.bfloat16,), q.device)
    T, Hq, D = q.shape
    Hkv, S, _ = k.shape
    if k.shape != v.shape or k.shape[2] != D:
        raise ValueError(f"shapes do not fit: q {tuple(q.shape)}, k {tuple(k.shape)}, "
                         f"v {tuple(v.shape)}")
    if (q_offsets is None) != (kv_offsets is None):
        raise ValueError("q_offsets and kv_offsets go together")
    n = 0
    if q_offsets is not None:
        _offsets(q_offsets, "q_offsets", q.device)
        _offsets(kv_offsets, "kv_offsets", q.device)
        if q_offsets.numel() != kv_offsets.numel():
            raise ValueError("q_offsets and kv_offsets differ in length")
        n = q_offsets.numel() - 1
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _tensor(out, "out", 3, (torch.bfloat16,), q.device)
        if out.shape != q.shape:
            raise ValueError(f"out has shape {tuple(out.shape)}")
        _apart(out, "out", q=q, k=k, v=v, q_offsets=q_offsets, kv_offsets=kv_offsets)
    a = tre.tre_attention(Hq, Hkv, D, n, T, S, q.stride(0), q.stride(1), k.stride(1), k.stride(0),
                          v.stride(1), v.stride(0), out.stride(0), out.stride(1),
                          1.0 / math.sqrt(D) if scale is None else scale)
    need = tre.tre_prompt_attention_workspace(a, _sms(q.device))
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    _call(tre.lib.tre_prompt_attention, q.device, a, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          _ptr(q_offsets), _ptr(kv_offsets), out.data_ptr(), _ptr(ws), need)
    return out


def mxfp4_quantize(w, out=None):
    """Weights [..., K] (bf16 or fp32, K a multiple of 32) to the engine's MXFP4 rows, uint8
    [..., mxfp4_pitch(K)]: per 32 weights the scale 2^(floor(log2(max)) - 2), codes to the
    nearest (ties to even), larger magnitudes saturated; a group with a NaN or an infinity
    stands for NaN."""
    if not isinstance(w, torch.Tensor) or w.ndim < 1:
        raise ValueError("w must be a tensor of at least one row")
    flat = w.reshape(-1, w.shape[-1]) if w.numel() else w.new_empty((0, w.shape[-1]))
    _tensor(flat, "w", 2, tuple(_TYPES))
    R, K = flat.shape
    if K <= 0 or K % 32:
        raise ValueError(f"rows must have a positive multiple of 32 weights, not {K}")
    shape = (*w.shape[:-1], mxfp4_pitch(K))
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=w.device)
    else:
        _tensor(out, "out", len(shape), (torch.uint8,), w.device)
        if tuple(out.shape) != shape or not out.is_contiguous():
            raise ValueError(f"out must be contiguous and of shape {shape}")
        _apart(out, "out", w=flat)
    _call(tre.lib.tre_mxfp4_quantize, w.device, flat.data_ptr(), _TYPES[w.dtype], R, K,
          flat.stride(0), out.data_ptr())
    return out


def _rows(w, name: str, ndim: Optional[int], K: int) -> None:
    if ndim is None:  # any number of rows' dimensions
        ndim = max(w.ndim, 1) if isinstance(w, torch.Tensor) else 1
    _tensor(w, name, ndim, (torch.uint8,))
    if K <= 0 or K % 32:
        raise ValueError(f"k must be a positive multiple of 32, not {K}")
    if w.shape[-1] != mxfp4_pitch(K):
        raise ValueError(f"{name}'s rows of {K} weights have {mxfp4_pitch(K)} bytes, "
                         f"not {w.shape[-1]}")
    if not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def mxfp4_dequantize(w, k: int, out_dtype=torch.bfloat16, out=None):
    """The numbers that MXFP4 rows [..., mxfp4_pitch(k)] stand for, [..., k] in bf16 or fp32
    (exact in both)."""
    _rows(w, "w", None, k)
    if out_dtype not in _TYPES:
        raise ValueError(f"out_dtype {out_dtype} is not bf16 or fp32")
    shape = (*w.shape[:-1], k)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=w.device)
    else:
        _tensor(out, "out", len(shape), (out_dtype,), w.device)
        if tuple(out.shape) != shape or not out.is_contiguous():
            raise ValueError(f"out must be contiguous and of shape {shape}")
        _apart(out, "out", w=w)
    _call(tre.lib.tre_mxfp4_dequantize, w.device, w.data_ptr(), w.numel() // w.shape[-1], k,
          _TYPES[out_dtype], out.data_ptr())
    return out


def mxfp4_matmul(x, w, offsets=None, out_dtype=torch.float32, out=None):
    """y[t] = W_e x[t] for the rows t in [offsets[e], offsets[e + 1]); returns [T, N].

    x [T, K] bf16 (row stride of whole 16-byte units), w [E, N, mxfp4_pitch(K)] uint8 (an
    expert slot of ``upload_moe_model`` as it is) or [N, mxfp4_pitch(K)], offsets int32
    [E + 1] on the device (read when the kernel runs) or None with one expert: every row.
    Rows of no expert are left as they are in ``out`` (unwritten in an ``out`` that the call
    allocates)."""
    _tensor(x, "x", 2, (torch.bfloat16,))
    T, K = x.shape
    if isinstance(w, torch.Tensor) and w.ndim == 2:
        w = w.unsqueeze(0)
    _rows(w, "w", 3, K)
    if w.device != x.device:
        raise ValueError(f"w is on {w.device}, not on {x.device}")
    E, N, _ = w.shape
    if E < 1 or N < 1:
        raise ValueError(f"w has shape {tuple(w.shape)}")
    if out_dtype not in _TYPES:
        raise ValueError(f"out_dtype {out_dtype} is not bf16 or fp32")
    if offsets is None and E != 1:
        raise ValueError("several experts need offsets")
    if offsets is not None:
        _offsets(offsets, "offsets", x.device)
        if offsets.numel() != E + 1:
            raise ValueError(f"offsets must have {E + 1} entries")
    if out is None:
        out = x.new_empty((T, N), dtype=out_dtype)
    else:
        _tensor(out, "out", 2, (out_dtype,), x.device)
        if tuple(out.shape) != (T, N):
            raise ValueError(f"out has shape {tuple(out.shape)}")
        _apart(out, "out", x=x, w=w, offsets=offsets)
    _call(tre.lib.tre_mxfp4_matmul, x.device, x.data_ptr(), x.stride(0), w.data_ptr(),
          _ptr(offsets), E, T, N, K, _TYPES[out_dtype], out.data_ptr(), out.stride(0))
    return out


def add_rmsnorm(x, delta, gain, eps: float, x_out=None, out=None):
    """(x + delta, bf16((x + delta) * gain / sqrt(mean((x + delta)^2) + eps))).

    x [T, d] fp32, delta [T, d] bf16 or fp32 or None, gain [d] bf16, d a multiple of 8.
    x_out may be x: the residual stream updated in place."""
    _tensor(x, "x", 2, (torch.float32,))
    T, d = x.shape
    if delta is not None:
        _tensor(delta, "delta", 2, tuple(_TYPES), x.device)
        if delta.shape != x.shape:
            raise ValueError(f"delta has shape {tuple(delta.shape)}")
    _tensor(gain, "gain", 1, (torch.bfloat16,), x.device)
    if gain.shape[0] != d:
        raise ValueError(f"gain has {gain.shape[0]} entries, not {d}")
    own_x, own = x_out is None, out is None
    if own_x:
        x_out = torch.empty_like(x, memory_format=torch.contiguous_format)
    elif x_out is not x:
        _tensor(x_out, "x_out", 2, (torch.float32,), x.device)
        if x_out.shape != x.shape:
            raise ValueError(f"x_out has shape {tuple(x_out.shape)}")
        if x_out.data_ptr() != x.data_ptr() or x_out.stride() != x.stride():
            _apart(x_out, "x_out", x=x)
    if own:
        out = torch.empty_like(x, dtype=torch.bfloat16, memory_format=torch.contiguous_format)
    else:
        _tensor(out, "out", 2, (torch.bfloat16,), x.device)
        if out.shape != x.shape:
            raise ValueError(f"out has shape {tuple(out.shape)}")
        _apart(out, "out", x=x, delta=delta, gain=gain)
    if not own_x:
        _apart(x_out, "x_out", delta=delta, gain=gain, out=None if own else out)
    _call(tre.lib.tre_add_rmsnorm, x.device, x.data_ptr(), x.stride(0), _ptr(delta),
          0 if delta is None else _TYPES[delta.dtype], 0 if delta is None else delta.stride(0),
          gain.data_ptr(), eps, T, d, x_out.data_ptr(), x_out.stride(0), out.data_ptr(),
          out.stride(0))
    return x_out, out
