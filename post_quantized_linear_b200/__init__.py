"""B200 (sm_100a) DualScale / SegLinear quantized linear layer.

Python binding of the C ABI in ``include/segquant.h``: PyTorch supplies device
memory and the current CUDA stream; every step of the layer runs in the
library's CUDA kernels.  Function names follow the C entry points.

SegQuant ("SegQuant: A Semantics-Aware and Generalizable Quantization
Framework for Diffusion Models"): DualScale quantizes the non-negative and
negative parts of each activation with separate static scales and fuses the
two int8 products in one kernel's epilogue (Spanish technical summary 2.B;
Korean technical summary section 2); SegLinear gives each input segment its
own scales (Spanish technical summary 2.A).
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import functools
from typing import Optional, Sequence, Tuple

import torch

from . import _lib
from ._lib import SegQuantError

__all__ = ["QuantizedWeight", "SegQuantError", "calibrate", "quantize_weights", "linear",
           "quantize_activations", "linear_from_codes", "quantize_activations_combined",
           "linear_from_combined", "quantize_activations_single", "linear_from_single",
           "splitk_workspace_size", "splitk_workspace", "linear_from_codes_splitk",
           "linear_accumulators", "stream_status", "qweight_sizes", "calibrate_hadamard",
           "quantize_activations_hadamard", "rotate_weights_hadamard",
           "linear_from_codes_hadamard", "calibrate_act", "quantize_activations_combined_act",
           "group_norm_act", "group_norm_act_backward", "quantize_activations_norm",
           "Adapters", "adapter_add", "adapter_backward"]


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return _lib.SQ_F32
    if t == torch.bfloat16:
        return _lib.SQ_BF16
    raise TypeError(f"unsupported dtype {t}: float32 or bfloat16")


# the current stream's raw handle without building a Stream object (a few
# microseconds per call at small M); the public call where it is missing
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream: Optional[torch.cuda.Stream]):
    """The given stream, else the current stream of the current device (the
    device the library launches on)."""
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _raw_stream is not None:
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_2d(x: torch.Tensor, name: str):
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


@dataclasses.dataclass
class QuantizedWeight:
    """Device codes/scales of a quantized [N, K] weight plus its segment bounds."""
    bits: int
    N: int
    K: int
    kseg: Tuple[int, ...]
    nseg: Tuple[int, ...]
    codes: torch.Tensor    # int8 [N, K] or uint8 [N, K/2]
    scales: torch.Tensor   # float32 [J, N] or float16 [K/128, N]

    @property
    def group(self) -> int:
        return 0 if self.bits == 8 else 128

    def c_struct(self):
        """The C view (sq_qweight) of this weight, rebuilt only when a field
        it is made of has changed."""
        key = (self.bits, self.N, self.K, tuple(self.kseg), tuple(self.nseg),
               self.codes.data_ptr(), self.scales.data_ptr())
        cached = self.__dict__.get("_c_struct")
        if cached is not None and cached[0] == key:
            return cached[1], cached[2]
        ks, ka = _lib.segments(self.kseg)
        ns, na = _lib.segments(self.nseg)
        qw = _lib.SqQWeight(self.bits, self.group, self.N, self.K, ks, ns,
                            ctypes.c_void_p(self.codes.data_ptr()),
                            ctypes.c_void_p(self.scales.data_ptr()))
        self.__dict__["_c_struct"] = (key, qw, (ka, na))
        return qw, (ka, na)


def qweight_sizes(bits: int, N: int, K: int, J: int) -> Tuple[int, int]:
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _lib.check("sq_qweight_sizes", _lib.load().sq_qweight_sizes(
        bits, N, K, J, 0 if bits == 8 else 128, ctypes.byref(cb), ctypes.byref(sb)))
    return cb.value, sb.value


def calibrate(x: torch.Tensor, kseg: Sequence[int], s_pos: Optional[torch.Tensor] = None,
              s_neg: Optional[torch.Tensor] = None, stream=None):
    """Static DualScale scales of the calibration rows ``x`` [rows, K]: (s+, s-) fp32 [J]."""
    _check_2d(x, "x")
    J = len(kseg) - 1
    if s_pos is None:
        s_pos = torch.empty(J, dtype=torch.float32, device=x.device)
    if s_neg is None:
        s_neg = torch.empty(J, dtype=torch.float32, device=x.device)
    seg, keep = _lib.segments(kseg)
    _lib.check("sq_calibrate", _lib.load().sq_calibrate(
        _ptr(x), _dtype_code(x.dtype), x.shape[0], x.shape[1], x.stride(0), ctypes.byref(seg),
        _ptr(s_pos), _ptr(s_neg), _stream(stream)))
    return s_pos, s_neg


def quantize_weights(w: torch.Tensor, kseg: Sequence[int], nseg: Optional[Sequence[int]] = None,
                     bits: int = 8, out: Optional[QuantizedWeight] = None,
                     stream=None) -> QuantizedWeight:
    """Quantize an [N, K] weight: int8 per (channel, K segment) or int4 group 128."""
    _check_2d(w, "w")
    N, K = w.shape
    kseg = tuple(int(b) for b in kseg)
    nseg = tuple(int(b) for b in (nseg if nseg is not None else (0, N)))
    if out is None:
        cb, sb = qweight_sizes(bits, N, K, len(kseg) - 1)
        if bits == 8:
            codes = torch.empty((N, K), dtype=torch.int8, device=w.device)
            scales = torch.empty((len(kseg) - 1, N), dtype=torch.float32, device=w.device)
        else:
            codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
            scales = torch.empty((K // 128, N), dtype=torch.float16, device=w.device)
        assert codes.numel() * codes.element_size() == cb
        assert scales.numel() * scales.element_size() == sb
        out = QuantizedWeight(bits, N, K, kseg, nseg, codes, scales)
    qw, keep = out.c_struct()
    _lib.check("sq_quantize_weights", _lib.load().sq_quantize_weights(
        _ptr(w), _dtype_code(w.dtype), N, K, w.stride(0), ctypes.byref(qw), _stream(stream)))
    return out


def linear(x: torch.Tensor, qw: QuantizedWeight, s_pos: torch.Tensor, s_neg: torch.Tensor,
           bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
           out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The fused forward pass y = DualScale-quantized x times the quantized weight (+ bias)."""
    _check_2d(x, "x")
    M, K = x.shape
    if out is None:
        out = torch.empty((M, qw.N), dtype=out_dtype, device=x.device)
    _check_2d(out, "out")
    c, keep = qw.c_struct()
    _lib.check("sq_linear_forward", _lib.load().sq_linear_forward(
        _ptr(x), _dtype_code(x.dtype), M, K, x.stride(0), ctypes.byref(c), _ptr(s_pos),
        _ptr(s_neg), _ptr(bias), _ptr(out), _dtype_code(out.dtype), out.stride(0), _stream(stream)))
    return out


def linear_from_codes(q_pos: torch.Tensor, q_neg: torch.Tensor, qw: QuantizedWeight,
                      s_pos: torch.Tensor, s_neg: torch.Tensor, bias: Optional[torch.Tensor] = None,
                      out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Forward from pre-quantized DualScale codes (same result as ``linear``)."""
    _check_2d(q_pos, "q_pos")
    _check_2d(q_neg, "q_neg")
    M, K = q_pos.shape
    if q_neg.shape != q_pos.shape or q_neg.stride(0) != q_pos.stride(0):
        raise ValueError("q_pos and q_neg must have the same shape and row stride")
    if out is None:
        out = torch.empty((M, qw.N), dtype=out_dtype, device=q_pos.device)
    _check_2d(out, "out")
    c, keep = qw.c_struct()
    _lib.check("sq_linear_forward_codes", _lib.load().sq_linear_forward_codes(
        _ptr(q_pos), _ptr(q_neg), q_pos.stride(0), M, K, ctypes.byref(c), _ptr(s_pos), _ptr(s_neg),
        _ptr(bias), _ptr(out), _dtype_code(out.dtype), out.stride(0), _stream(stream)))
    return out


def quantize_activations(x: torch.Tensor, kseg: Sequence[int], s_pos: torch.Tensor,
                         s_neg: torch.Tensor, out=None, stream=None):
    """DualScale codes (q+, q-), int8 [M, K] each (row stride a multiple of 16)."""
    _check_2d(x, "x")
    M, K = x.shape
    if out is None:
        ldq = (K + 15) // 16 * 16
        qp = torch.empty((M, ldq), dtype=torch.int8, device=x.device)[:, :K]
        qn = torch.empty((M, ldq), dtype=torch.int8, device=x.device)[:, :K]
    else:
        qp, qn = out
        if qp.stride(0) != qn.stride(0):
            raise ValueError("q_pos and q_neg must share a row stride")
    seg, keep = _lib.segments(kseg)
    _lib.check("sq_quantize_activations", _lib.load().sq_quantize_activations(
        _ptr(x), _dtype_code(x.dtype), M, K, x.stride(0), ctypes.byref(seg), _ptr(s_pos),
        _ptr(s_neg), _ptr(qp), _ptr(qn), qp.stride(0), _stream(stream)))
    return qp, qn


def quantize_activations_combined(x: torch.Tensor, kseg: Sequence[int], s_pos: torch.Tensor,
                                  s_neg: torch.Tensor, out: Optional[torch.Tensor] = None,
                                  stream=None) -> torch.Tensor:
    """DualScale codes in one byte per activation: c = q+ + q-, int8 [M, K]
    (row stride a multiple of 16); q+ = max(c, 0), q- = min(c, 0)."""
    _check_2d(x, "x")
    M, K = x.shape
    if out is None:
        ldc = (K + 15) // 16 * 16
        out = torch.empty((M, ldc), dtype=torch.int8, device=x.device)[:, :K]
    seg, keep = _lib.segments(kseg)
    _lib.check("sq_quantize_activations_combined", _lib.load().sq_quantize_activations_combined(
        _ptr(x), _dtype_code(x.dtype), M, K, x.stride(0), ctypes.byref(seg), _ptr(s_pos),
        _ptr(s_neg), _ptr(out), out.stride(0), _stream(stream)))
    return out


def _act_code(act: str) -> int:
    if act == "silu":
        return _lib.SQ_ACT_SILU
    if act == "gelu":
        return _lib.SQ_ACT_GELU
    raise ValueError(f"unknown activation {act!r}: 'silu' or 'gelu'")


def calibrate_act(z: torch.Tensor, act: str, kseg: Sequence[int],
                  s_pos: Optional[torch.Tensor] = None, s_neg: Optional[torch.Tensor] = None,
                  stream=None):
    """Static DualScale scales (s+, s-) fp32 [J] of X = act(z) over the
    calibration rows of the pre-activation ``z`` [rows, K]; act: 'silu' or 'gelu'."""
    _check_2d(z, "z")
    J = len(kseg) - 1
    if s_pos is None:
        s_pos = torch.empty(J, dtype=torch.float32, device=z.device)
    if s_neg is None:
        s_neg = torch.empty(J, dtype=torch.float32, device=z.device)
    seg, keep = _lib.segments(kseg)
    _lib.check("sq_calibrate_act", _lib.load().sq_calibrate_act(
        _ptr(z), _dtype_code(z.dtype), _act_code(act), z.shape[0], z.shape[1], z.stride(0),
        ctypes.byref(seg), _ptr(s_pos), _ptr(s_neg), _stream(stream)))
    return s_pos, s_neg


def quantize_activations_combined_act(z: torch.Tensor, act: str, kseg: Sequence[int],
                                      s_pos: torch.Tensor, s_neg: torch.Tensor,
                                      out: Optional[torch.Tensor] = None,
                                      stream=None) -> torch.Tensor:
    """Combined DualScale codes of X = act(z) (X rounded once to bf16, never
    stored), int8 [M, K] with row stride a multiple of 16; act: 'silu' or 'gelu'."""
    _check_2d(z, "z")
    M, K = z.shape
    if out is None:
        ldc = (K + 15) // 16 * 16
        out = torch.empty((M, ldc), dtype=torch.int8, device=z.device)[:, :K]
    seg, keep = _lib.segments(kseg)
    _lib.check("sq_quantize_activations_combined_act",
               _lib.load().sq_quantize_activations_combined_act(
                   _ptr(z), _dtype_code(z.dtype), _act_code(act), M, K, z.stride(0),
                   ctypes.byref(seg), _ptr(s_pos), _ptr(s_neg), _ptr(out), out.stride(0),
                   _stream(stream)))
    return out


def linear_from_combined(c: torch.Tensor, qw: QuantizedWeight, s_pos: torch.Tensor,
                         s_neg: torch.Tensor, bias: Optional[torch.Tensor] = None,
                         out_dtype: torch.dtype = torch.bfloat16,
                         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Forward from combined DualScale codes (same result as ``linear``); int8 weights."""
    _check_2d(c, "c")
    M, K = c.shape
    if out is None:
        out = torch.empty((M, qw.N), dtype=out_dtype, device=c.device)
    _check_2d(out, "out")
    cw, keep = qw.c_struct()
    _lib.check("sq_linear_forward_combined", _lib.load().sq_linear_forward_combined(
        _ptr(c), c.stride(0), M, K, ctypes.byref(cw), _ptr(s_pos), _ptr(s_neg), _ptr(bias),
        _ptr(out), _dtype_code(out.dtype), out.stride(0), _stream(stream)))
    return out


def quantize_activations_single(x: torch.Tensor, kseg: Sequence[int], s_pos: torch.Tensor,
                                s_neg: torch.Tensor, out: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """Single-scale baseline codes, int8 [M, K]: one symmetric scale per K
    segment, s = max(s_pos, s_neg) (= max|x| / 127 of the calibration rows)."""
    _check_2d(x, "x")
    M, K = x.shape
    if out is None:
        ldc = (K + 15) // 16 * 16
        out = torch.empty((M, ldc), dtype=torch.int8, device=x.device)[:, :K]
    seg, keep = _lib.segments(kseg)
    _lib.check("sq_quantize_activations_single", _lib.load().sq_quantize_activations_single(
        _ptr(x), _dtype_code(x.dtype), M, K, x.stride(0), ctypes.byref(seg), _ptr(s_pos),
        _ptr(s_neg), _ptr(out), out.stride(0), _stream(stream)))
    return out


def linear_from_single(c: torch.Tensor, qw: QuantizedWeight, s_pos: torch.Tensor,
                       s_neg: torch.Tensor, bias: Optional[torch.Tensor] = None,
                       out_dtype: torch.dtype = torch.bfloat16,
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Single-scale baseline forward from ``quantize_activations_single`` codes (int8 weights)."""
    _check_2d(c, "c")
    M, K = c.shape
    if out is None:
        out = torch.empty((M, qw.N), dtype=out_dtype, device=c.device)
    _check_2d(out, "out")
    cw, keep = qw.c_struct()
    _lib.check("sq_linear_forward_single", _lib.load().sq_linear_forward_single(
        _ptr(c), c.stride(0), M, K, ctypes.byref(cw), _ptr(s_pos), _ptr(s_neg), _ptr(bias),
        _ptr(out), _dtype_code(out.dtype), out.stride(0), _stream(stream)))
    return out


def splitk_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace ``linear_from_codes_splitk`` needs on the current device."""
    n = ctypes.c_size_t()
    _lib.check("sq_splitk_workspace_size",
               _lib.load().sq_splitk_workspace_size(M, N, K, ctypes.byref(n)))
    return n.value


def splitk_workspace(M: int, N: int, K: int, device=None) -> torch.Tensor:
    """A zeroed workspace for ``linear_from_codes_splitk`` (uint8, 256-byte aligned)."""
    return torch.zeros(splitk_workspace_size(M, N, K), dtype=torch.uint8, device=device)


def linear_from_codes_splitk(q_pos: torch.Tensor, q_neg: torch.Tensor, qw: QuantizedWeight,
                             s_pos: torch.Tensor, s_neg: torch.Tensor, workspace: torch.Tensor,
                             bias: Optional[torch.Tensor] = None,
                             out_dtype: torch.dtype = torch.bfloat16,
                             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Small-M (M <= 128) forward from DualScale codes, K split across the GPU;
    bit-identical to ``linear_from_codes``.  ``workspace`` from ``splitk_workspace``
    (its counters return to zero after every completed call)."""
    _check_2d(q_pos, "q_pos")
    _check_2d(q_neg, "q_neg")
    M, K = q_pos.shape
    if q_neg.shape != q_pos.shape or q_neg.stride(0) != q_pos.stride(0):
        raise ValueError("q_pos and q_neg must have the same shape and row stride")
    if out is None:
        out = torch.empty((M, qw.N), dtype=out_dtype, device=q_pos.device)
    _check_2d(out, "out")
    c, keep = qw.c_struct()
    _lib.check("sq_linear_forward_codes_splitk", _lib.load().sq_linear_forward_codes_splitk(
        _ptr(q_pos), _ptr(q_neg), q_pos.stride(0), M, K, ctypes.byref(c), _ptr(s_pos), _ptr(s_neg),
        _ptr(bias), _ptr(out), _dtype_code(out.dtype), out.stride(0), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def num_units(qw: QuantizedWeight) -> int:
    return len(qw.kseg) - 1 if qw.bits == 8 else qw.K // 128


def linear_accumulators(x: torch.Tensor, qw: QuantizedWeight, s_pos: torch.Tensor,
                        s_neg: torch.Tensor, stream=None) -> torch.Tensor:
    """Raw int32 accumulators [U, 2, M, N] of the fused kernel (test surface)."""
    _check_2d(x, "x")
    M, K = x.shape
    acc = torch.empty((num_units(qw), 2, M, qw.N), dtype=torch.int32, device=x.device)
    c, keep = qw.c_struct()
    _lib.check("sq_linear_accumulators", _lib.load().sq_linear_accumulators(
        _ptr(x), _dtype_code(x.dtype), M, K, x.stride(0), ctypes.byref(c), _ptr(s_pos),
        _ptr(s_neg), _ptr(acc), _stream(stream)))
    return acc


def stream_status(stream=None) -> int:
    """Synchronize the stream and return (and clear) the device status word."""
    return int(_lib.load().sq_stream_status(_stream(stream)))


def set_wait_budget(cycles: int) -> None:
    """Test hook of the development library (inside ``_lib.dev_library()``):
    device-side pipeline wait budget in SM clock cycles (0 = default, ~1 s)."""
    _lib.check("sq_set_wait_budget", _lib.load().sq_set_wait_budget(int(cycles)))


def debug_starve_pipeline(enable: bool) -> None:
    """Test hook of the development library: GEMM launches issue no TMA
    copies, so their waits expire."""
    _lib.check("sq_debug_starve_pipeline", _lib.load().sq_debug_starve_pipeline(1 if enable else 0))


# ------------------------------------------------- block-Hadamard activations
# HQ-DM ("HQ-DM: Single Hadamard Transformation-Based Quantization-Aware
# Training for Low-Bit Diffusion Models", Spanish technical summary 2.1):
# activations times a block-diagonal Hadamard matrix (blocks of 16 along K)
# before quantization; int4 weights quantized untransformed; the forward is the
# integer product of the XH codes with the int4 codes rotated into the same
# basis, the block normalization 1/4 carried by the activation scales.

def calibrate_hadamard(x: torch.Tensor, kseg: Sequence[int], s_pos: Optional[torch.Tensor] = None,
                       s_neg: Optional[torch.Tensor] = None, stream=None):
    """DualScale scales (s+, s-) fp32 [J] of the transformed calibration rows XH."""
    _check_2d(x, "x")
    J = len(kseg) - 1
    if s_pos is None:
        s_pos = torch.empty(J, dtype=torch.float32, device=x.device)
    if s_neg is None:
        s_neg = torch.empty(J, dtype=torch.float32, device=x.device)
    seg, keep = _lib.segments(kseg)
    _lib.check("sq_calibrate_hadamard", _lib.load().sq_calibrate_hadamard(
        _ptr(x), _dtype_code(x.dtype), x.shape[0], x.shape[1], x.stride(0), ctypes.byref(seg),
        _ptr(s_pos), _ptr(s_neg), _stream(stream)))
    return s_pos, s_neg


def quantize_activations_hadamard(x: torch.Tensor, kseg: Sequence[int], s_pos: torch.Tensor,
                                  s_neg: torch.Tensor, out=None, stream=None):
    """DualScale codes (q+, q-) of XH, int8 [M, K] each (row stride a multiple of 16)."""
    _check_2d(x, "x")
    M, K = x.shape
    if out is None:
        ldq = (K + 15) // 16 * 16
        qp = torch.empty((M, ldq), dtype=torch.int8, device=x.device)[:, :K]
        qn = torch.empty((M, ldq), dtype=torch.int8, device=x.device)[:, :K]
    else:
        qp, qn = out
        if qp.stride(0) != qn.stride(0):
            raise ValueError("q_pos and q_neg must share a row stride")
    seg, keep = _lib.segments(kseg)
    _lib.check("sq_quantize_activations_hadamard", _lib.load().sq_quantize_activations_hadamard(
        _ptr(x), _dtype_code(x.dtype), M, K, x.stride(0), ctypes.byref(seg), _ptr(s_pos),
        _ptr(s_neg), _ptr(qp), _ptr(qn), qp.stride(0), _stream(stream)))
    return qp, qn


def rotate_weights_hadamard(qw: QuantizedWeight, out: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """The int4 codes of ``qw`` rotated into the transform's basis, int8 [N, K]."""
    if qw.bits != 4:
        raise ValueError("the Hadamard forward takes int4 weights")
    if out is None:
        out = torch.empty((qw.N, qw.K), dtype=torch.int8, device=qw.codes.device)
    _check_2d(out, "out")
    c, keep = qw.c_struct()
    _lib.check("sq_rotate_weights_hadamard", _lib.load().sq_rotate_weights_hadamard(
        ctypes.byref(c), _ptr(out), out.stride(0), _stream(stream)))
    return out


def linear_from_codes_hadamard(q_pos: torch.Tensor, q_neg: torch.Tensor, qw: QuantizedWeight,
                               w_rot: torch.Tensor, s_pos: torch.Tensor, s_neg: torch.Tensor,
                               bias: Optional[torch.Tensor] = None,
                               out_dtype: torch.dtype = torch.bfloat16,
                               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Forward from the XH codes and the rotated int4 weight codes."""
    _check_2d(q_pos, "q_pos")
    _check_2d(q_neg, "q_neg")
    _check_2d(w_rot, "w_rot")
    M, K = q_pos.shape
    if q_neg.shape != q_pos.shape or q_neg.stride(0) != q_pos.stride(0):
        raise ValueError("q_pos and q_neg must have the same shape and row stride")
    if out is None:
        out = torch.empty((M, qw.N), dtype=out_dtype, device=q_pos.device)
    _check_2d(out, "out")
    c, keep = qw.c_struct()
    _lib.check("sq_linear_forward_codes_hadamard", _lib.load().sq_linear_forward_codes_hadamard(
        _ptr(q_pos), _ptr(q_neg), q_pos.stride(0), M, K, ctypes.byref(c), _ptr(w_rot),
        w_rot.stride(0), _ptr(s_pos), _ptr(s_neg), _ptr(bias), _ptr(out), _dtype_code(out.dtype),
        out.stride(0), _stream(stream)))
    return out


# --------------------------------------------- group norm with an activation
# The norm in front of the quantized layers of a U-Net or an image decoder,
# channels last: maps are [B, S, C] with S = H*W (for an NCHW tensor in the
# channels_last memory format, ``t.permute(0, 2, 3, 1).flatten(1, 2)``).
#
# These calls and the adapters' allocate their results in the order of ``stream``
# where one is given: another stream that reads them has to wait for it, and
# calls ``record_stream`` on what it may still read after the last reference is gone.

_NORM_ACTS = {"none": 0, "silu": _lib.SQ_ACT_SILU, "gelu": _lib.SQ_ACT_GELU}
# the current device's index without the lazy-initialization check; the public call where it is missing
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _norm_act_code(act: str) -> int:
    code = _NORM_ACTS.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}: 'none', 'silu' or 'gelu'")
    return code


def _stream_ptr(stream: Optional[torch.cuda.Stream], dev: int):
    """The raw handle of the given stream, else of the current one of device ``dev``."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(dev)
    return torch.cuda.current_stream().cuda_stream


def _map(x: torch.Tensor, name: str, shape=None):
    """(device, position stride, image stride) of a checked channels-last map [B, S, C]; a
    single position or image has no stride that matters."""
    st = x.stride()
    sh = x.shape
    if len(st) != 3 or (st[2] != 1 and sh[2] != 1):
        raise ValueError(f"{name} must be a 3-D [B, S, C] tensor with unit channel stride")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if shape is not None and sh != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(sh)}")
    return x.get_device(), st[1] if sh[1] > 1 else max(sh[2], 1), st[0] if sh[0] > 1 else 0


def _same_device(dev: int, *others: int):
    """Launches go to the current device: every tensor has to be there."""
    cur = _current_device()
    if dev != cur or any(d != cur for d in others):
        raise ValueError("tensors must be on the current CUDA device")


def _check_f32(t: Optional[torch.Tensor], shape, name: str, dev: int):
    """An optional contiguous fp32 tensor of the given shape on device ``dev``: its pointer or None."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(shape)} "
                         "on the current device")
    return t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _norm_workspace_size(device: int, B: int, S: int, C: int, groups: int, xt: int, backward: int) -> int:
    n = ctypes.c_size_t()
    _lib.check("sq_group_norm_workspace_size", _lib.load().sq_group_norm_workspace_size(
        B, S, C, groups, xt, backward, ctypes.byref(n)))
    return n.value


_segments_of = functools.lru_cache(maxsize=256)(_lib.segments)   # of a tuple of ints, never changed


_NO_STREAM = contextlib.nullcontext()


def _in_order(stream):
    """Context for what a call allocates: memory in ``stream``'s order (None: the current
    stream's), since a block that was freed in another one may still be in use there."""
    return _NO_STREAM if stream is None else torch.cuda.stream(stream)


def group_norm_act(x: torch.Tensor, groups: int, gamma: Optional[torch.Tensor] = None,
                   beta: Optional[torch.Tensor] = None, eps: float = 1e-5, act: str = "none",
                   out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                   return_stats: bool = False, stream=None):
    """y = act(group_norm(x) * gamma + beta) of a channels-last map ``x`` [B, S, C];
    act: 'none', 'silu' or 'gelu'.  ``out`` may be ``x`` itself.  With
    ``return_stats`` also the fp32 [B, groups, 2] means and reciprocal deviations
    that ``group_norm_act_backward`` takes."""
    dev, ldx, xbs = _map(x, "x")
    shape = x.shape
    B, S, C = shape
    if out is None:
        ldy, ybs, dy = C, S * C, dev
    else:
        dy, ldy, ybs = _map(out, "out", shape)
    _same_device(dev, dy)
    xt = _dtype_code(x.dtype)
    wn = _norm_workspace_size(dev, B, S, C, groups, xt, 0)
    with _in_order(stream):
        if out is None:
            if (out_dtype is None or out_dtype is x.dtype) and x.is_contiguous():
                out = torch.empty_like(x)
            else:
                out = torch.empty(shape, dtype=out_dtype or x.dtype, device=x.device)
        stats = x.new_empty((B, groups, 2), dtype=torch.float32) if return_stats else None
        ws = x.new_empty(wn, dtype=torch.uint8) if wn else None
    st = _lib.load().sq_group_norm_act(
        x.data_ptr(), xt, B, S, C, ldx, xbs, groups, _check_f32(gamma, (C,), "gamma", dev),
        _check_f32(beta, (C,), "beta", dev), eps, _norm_act_code(act), out.data_ptr(),
        _dtype_code(out.dtype), ldy, ybs, None if stats is None else stats.data_ptr(),
        None if ws is None else ws.data_ptr(), wn, _stream_ptr(stream, dev))
    if st:
        raise SegQuantError("sq_group_norm_act", st)
    return (out, stats) if return_stats else out


def quantize_activations_norm(x: torch.Tensor, groups: int, gamma: Optional[torch.Tensor],
                              beta: Optional[torch.Tensor], kseg: Sequence[int], s_pos: torch.Tensor,
                              s_neg: torch.Tensor, eps: float = 1e-5, act: str = "none", out=None,
                              return_y: bool = False, stream=None):
    """DualScale codes (q+, q-) of y = act(group_norm(x)) rounded to bf16, int8
    [B*S, C] each (row stride a multiple of 16), in one pass over ``x`` [B, S, C]; they
    feed ``linear_from_codes``.  With ``return_y`` (q+, q-, y), y bf16 [B*S, C] (the
    input of adapters beside the layer)."""
    dev, ldx, xbs = _map(x, "x")
    B, S, C = x.shape
    J = len(kseg) - 1
    _same_device(dev)
    ldq = (C + 15) // 16 * 16
    if out is not None:
        qp, qn = out
        for t, name in ((qp, "q_pos"), (qn, "q_neg")):
            _same_device(_check_rows(t, B * S, C, name)[0])
            if t.dtype != torch.int8:
                raise ValueError(f"{name} must be int8")
        if qp.stride(0) != qn.stride(0):
            raise ValueError("q_pos and q_neg must share a row stride")
        if B * S > 1:
            ldq = qp.stride(0)
    seg, keep = _segments_of(tuple(map(int, kseg)))
    xt = _dtype_code(x.dtype)
    wn = _norm_workspace_size(dev, B, S, C, groups, xt, 0)
    with _in_order(stream):
        if out is None:
            qp, qn = x.new_empty((2, B * S, ldq), dtype=torch.int8).unbind()
            if ldq != C:
                qp, qn = qp[:, :C], qn[:, :C]
        y = x.new_empty((B * S, C), dtype=torch.bfloat16) if return_y else None
        ws = x.new_empty(wn, dtype=torch.uint8) if wn else None
    st = _lib.load().sq_quantize_activations_norm(
        x.data_ptr(), xt, B, S, C, ldx, xbs, groups, _check_f32(gamma, (C,), "gamma", dev),
        _check_f32(beta, (C,), "beta", dev), eps, _norm_act_code(act), ctypes.byref(seg),
        _check_f32(s_pos, (J,), "s_pos", dev), _check_f32(s_neg, (J,), "s_neg", dev), qp.data_ptr(),
        qn.data_ptr(), ldq, None if y is None else y.data_ptr(), C,
        None if ws is None else ws.data_ptr(), wn, _stream_ptr(stream, dev))
    if st:
        raise SegQuantError("sq_quantize_activations_norm", st)
    return (qp, qn, y) if return_y else (qp, qn)


def group_norm_act_backward(dy: torch.Tensor, x: torch.Tensor, stats: torch.Tensor,
                            gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                            act: str = "none", dx: Optional[torch.Tensor] = None, stream=None):
    """Gradients (dx, dgamma, dbeta) of ``group_norm_act``: dx of x's type, dgamma and
    dbeta fp32 [C] (also where gamma or beta is None: those of ones and zeros).
    ``stats`` as returned by the forward call; ``dx`` may be ``x`` or ``dy``."""
    dev, ldx, xbs = _map(x, "x")
    shape = x.shape
    d2, lddy, dybs = _map(dy, "dy", shape)
    B, S, C = shape
    if stats.dim() != 3:
        raise ValueError("stats must be the [B, groups, 2] tensor of the forward call")
    groups = stats.shape[1]
    if dx is None:
        d3, lddx, dxbs = dev, C, S * C
    else:
        d3, lddx, dxbs = _map(dx, "dx", shape)
    if dy.dtype != x.dtype or (dx is not None and dx.dtype != x.dtype):
        raise TypeError("dy and dx must have x's dtype")
    _same_device(dev, d2, d3)
    xt = _dtype_code(x.dtype)
    wn = _norm_workspace_size(dev, B, S, C, groups, xt, 1)
    with _in_order(stream):
        if dx is None:
            dx = torch.empty_like(x) if x.is_contiguous() else torch.empty(shape, dtype=x.dtype, device=x.device)
        grads = x.new_empty((2, C), dtype=torch.float32)
        ws = x.new_empty(wn, dtype=torch.uint8) if wn else None
    g = grads.data_ptr()
    st = _lib.load().sq_group_norm_act_backward(
        dy.data_ptr(), lddy, dybs, x.data_ptr(), xt, B, S, C, ldx, xbs, groups,
        _check_f32(stats, (B, groups, 2), "stats", dev), _check_f32(gamma, (C,), "gamma", dev),
        _check_f32(beta, (C,), "beta", dev), _norm_act_code(act), dx.data_ptr(), lddx, dxbs, g, g + 4 * C,
        None if ws is None else ws.data_ptr(), wn, _stream_ptr(stream, dev))
    if st:
        raise SegQuantError("sq_group_norm_act_backward", st)
    dgamma, dbeta = grads.unbind()
    return dx, dgamma, dbeta


# ------------------------------------------------------- low-rank adapters
@dataclasses.dataclass(frozen=True)
class Adapters:
    """L low-rank adapters of a [N, K] projection: a bf16 [L, R, K], b bf16 [L, N, R],
    scale fp32 [L] (None: 1).  Adapters of smaller rank are padded with zeros."""
    a: torch.Tensor
    b: torch.Tensor
    scale: Optional[torch.Tensor] = None

    def __post_init__(self):
        a, b = self.a, self.b
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise ValueError("a must be [L, R, K] and b [L, N, R]")
        for t, name in ((a, "a"), (b, "b")):
            if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
                raise ValueError(f"{name} must be a contiguous bfloat16 CUDA tensor")
        s = self.scale
        if s is not None and (s.dtype != torch.float32 or s.shape != (a.shape[0],) or not s.is_cuda
                              or not s.is_contiguous()):
            raise ValueError("scale must be a contiguous float32 CUDA tensor of shape [L]")
        if a.device != b.device or (s is not None and s.device != a.device):
            raise ValueError("a, b and scale must be on the same device")

    def c_struct(self):
        """The C view (sq_adapters), rebuilt only when a tensor it is made of has moved."""
        s = self.scale
        key = (self.a.data_ptr(), self.b.data_ptr(), 0 if s is None else s.data_ptr())
        cached = self.__dict__.get("_c_struct")
        if cached is None or cached[0] != key:
            L, R, K = self.a.shape
            cached = (key, _lib.SqAdapters(L, R, K, self.b.shape[1], key[0], key[1], key[2] or None))
            self.__dict__["_c_struct"] = cached
        return cached[1]


def _check_rows(t: torch.Tensor, rows: int, cols: int, name: str):
    """(device, row stride) of a checked [rows, cols] matrix."""
    st = t.stride()
    if len(st) != 2 or st[1] != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], not {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device(), st[0] if rows > 1 else cols


def _check_requests(bounds: torch.Tensor, index: torch.Tensor, adapters: Adapters) -> Tuple[int, int]:
    """(requests, device) of checked request tensors."""
    n = index.numel()
    if (bounds.dtype is not torch.int32 or index.dtype is not torch.int32 or index.dim() != 1
            or bounds.shape != (n + 1,) or not bounds.is_contiguous() or not index.is_contiguous()):
        raise ValueError("bounds must be int32 [requests + 1] and index int32 [requests]")
    dev = adapters.a.get_device()
    _same_device(dev, bounds.get_device(), index.get_device())
    return n, dev


def adapter_add(y: torch.Tensor, x: torch.Tensor, adapters: Adapters, bounds: torch.Tensor,
                index: torch.Tensor, return_hidden: bool = False, stream=None,
                out: Optional[torch.Tensor] = None):
    """Adds the requests' low-rank terms to the shared projection's output ``y`` [M, N]
    in place: rows bounds[q] .. bounds[q+1] of ``x`` [M, K] use adapter index[q]
    (below 0: none), y += scale * (x a^T) b^T.  Rows of no request are left as they
    are.  ``bounds`` int32 [Q + 1] and ``index`` int32 [Q] stay on the device.  For a
    fused q | k | v projection with adapters of its own per part, call it on column
    slices of ``y``.  With ``return_hidden`` returns (y, hidden), hidden = x a^T in fp32
    [M, R] for ``adapter_backward``; otherwise y.

    A bf16 ``y`` holds a rounded value, and its sum is rounded again.  To round once, let
    ``linear_from_codes`` write float32 and give a bfloat16 ``out`` [M, N]: it receives y + the
    term (y's values in rows without an adapter), ``y`` stays as it is, ``out`` is returned."""
    n, dev = _check_requests(bounds, index, adapters)
    c = adapters.c_struct()
    M = x.shape[0]
    dx, ldx = _check_rows(x, M, c.K, "x")
    dy, ldy = _check_rows(y, M, c.N, "y")
    if dx != dev or dy != dev:
        raise ValueError("x and y must be on the current CUDA device")
    if out is not None:
        do, ldo = _check_rows(out, M, c.N, "out")
        if do != dev:
            raise ValueError("out must be on the current CUDA device")
        if y.dtype is not torch.float32 or out.dtype is not torch.bfloat16:
            raise TypeError("with out, y must be float32 and out bfloat16")
    with _in_order(stream):
        hidden = x.new_empty((M, c.R), dtype=torch.float32) if return_hidden else None
    if out is not None:
        name, st = "sq_adapter_add_to", _lib.load().sq_adapter_add_to(
            x.data_ptr(), _dtype_code(x.dtype), M, ldx, c, bounds.data_ptr(), index.data_ptr(), n, y.data_ptr(), ldy,
            out.data_ptr(), ldo, None if hidden is None else hidden.data_ptr(), _stream_ptr(stream, dev))
        y = out
    else:
        name, st = "sq_adapter_add", _lib.load().sq_adapter_add(
            x.data_ptr(), _dtype_code(x.dtype), M, ldx, c, bounds.data_ptr(), index.data_ptr(), n, y.data_ptr(),
            _dtype_code(y.dtype), ldy, None if hidden is None else hidden.data_ptr(), _stream_ptr(stream, dev))
    if st:
        raise SegQuantError(name, st)
    return (y, hidden) if return_hidden else y


def adapter_backward(dy: torch.Tensor, x: torch.Tensor, hidden: torch.Tensor, adapters: Adapters,
                     bounds: torch.Tensor, index: torch.Tensor, stream=None):
    """Gradients (dx, da, db) of the term ``adapter_add`` adds: dx [M, K] of x's type
    (zeros in rows without an adapter), da fp32 [L, R, K], db fp32 [L, N, R], each the sum
    over all requests of its adapter.  ``hidden`` as returned by ``adapter_add``."""
    n, dev = _check_requests(bounds, index, adapters)
    c = adapters.c_struct()
    M, R, K, N, L = x.shape[0], c.R, c.K, c.N, c.L
    d1, ldx = _check_rows(x, M, K, "x")
    d2, lddy = _check_rows(dy, M, N, "dy")
    if d1 != dev or d2 != dev:
        raise ValueError("x and dy must be on the current CUDA device")
    wn = _adapter_workspace_size(M, R)
    with _in_order(stream):
        dx = x.new_empty((M, K))
        da = x.new_empty((L, R, K), dtype=torch.float32)
        db = x.new_empty((L, N, R), dtype=torch.float32)
        ws = x.new_empty(wn, dtype=torch.uint8)
    st = _lib.load().sq_adapter_backward(
        dy.data_ptr(), _dtype_code(dy.dtype), M, lddy, x.data_ptr(), _dtype_code(x.dtype), ldx,
        _check_f32(hidden, (M, R), "hidden", dev), c, bounds.data_ptr(), index.data_ptr(), n,
        dx.data_ptr(), K, da.data_ptr(), db.data_ptr(), ws.data_ptr(), wn, _stream_ptr(stream, dev))
    if st:
        raise SegQuantError("sq_adapter_backward", st)
    return dx, da, db


@functools.lru_cache(maxsize=4096)
def _adapter_workspace_size(M: int, R: int) -> int:
    n = ctypes.c_size_t()
    _lib.check("sq_adapter_backward_workspace_size",
               _lib.load().sq_adapter_backward_workspace_size(M, R, ctypes.byref(n)))
    return n.value
