"""Torch-facing wrappers of the C ABI, same names as the C entry points.

PyTorch supplies device memory and the current stream; every step of the
path runs in the library's CUDA kernels.  Functions that produce tensors
allocate them with ``torch.empty`` (outputs and the workspace the library asks
for) unless the caller passes them in, which the bench does to keep
allocation out of the timed region.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import ACT_TYPES, CAdamWConfig, CDropoutConfig, CNF4Weight, CODE_TYPES, DQ_TYPES, QLORA_BF16, QLORA_F32, \
    check, lib

BLOCKSIZE = 64
DQ_BLOCK = 256


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


# the current stream's handle without building a Stream object (3 us of a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream: torch.cuda.Stream | None = None) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


@dataclass
class NF4Weight:
    """A quantized frozen weight W [rows = N, cols = K] and its constants.

    codes [ceil(N*K/2)] uint8 (element 2i in the high nibble of byte i);
    without double quantization ``absmax`` [nb] fp32; with it ``absmax_q8``
    [nb] uint8, ``absmax_scale`` [ceil(nb/256)] fp32 and ``absmax_offset``
    [1] fp32; nb = ceil(N*K / blocksize).  ``code_type`` "nf4" or "fp4",
    ``dq_type`` "int8" or "e4m3" (the 8-bit code book of the constants).
    """

    rows: int
    cols: int
    double_quant: bool
    codes: torch.Tensor
    absmax: torch.Tensor | None = None
    absmax_q8: torch.Tensor | None = None
    absmax_scale: torch.Tensor | None = None
    absmax_offset: torch.Tensor | None = None
    blocksize: int = BLOCKSIZE
    code_type: str = "nf4"
    dq_type: str = "int8"

    @property
    def nblocks(self) -> int:
        return (self.rows * self.cols + self.blocksize - 1) // self.blocksize

    def c_struct(self) -> CNF4Weight:
        return CNF4Weight(self.rows, self.cols, self.blocksize, int(self.double_quant),
                          _ptr(self.codes), _ptr(self.absmax), _ptr(self.absmax_q8),
                          _ptr(self.absmax_scale), _ptr(self.absmax_offset),
                          CODE_TYPES[self.code_type], DQ_TYPES[self.dq_type])

    def storage_bytes(self) -> int:
        t = [self.codes, self.absmax, self.absmax_q8, self.absmax_scale, self.absmax_offset]
        return sum(x.numel() * x.element_size() for x in t if x is not None)

    @staticmethod
    def empty(rows: int, cols: int, double_quant: bool = True, device="cuda", blocksize: int = BLOCKSIZE,
              code_type: str = "nf4", dq_type: str = "int8") -> "NF4Weight":
        n = rows * cols
        nb = (n + blocksize - 1) // blocksize
        codes = torch.empty((n + 1) // 2, dtype=torch.uint8, device=device)
        fmt = dict(blocksize=blocksize, code_type=code_type, dq_type=dq_type)
        if double_quant:
            return NF4Weight(rows, cols, True, codes,
                             absmax_q8=torch.empty(nb, dtype=torch.uint8, device=device),
                             absmax_scale=torch.empty((nb + DQ_BLOCK - 1) // DQ_BLOCK, dtype=torch.float32, device=device),
                             absmax_offset=torch.empty(1, dtype=torch.float32, device=device), **fmt)
        return NF4Weight(rows, cols, False, codes, absmax=torch.empty(nb, dtype=torch.float32, device=device), **fmt)


def _workspace(nbytes: int, device, ws: torch.Tensor | None) -> torch.Tensor:
    if ws is not None and ws.numel() >= nbytes:
        return ws
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def qlora_nf4_quantize_workspace(rows: int, cols: int, double_quant: bool = True,
                                 blocksize: int = BLOCKSIZE) -> int:
    return int(lib().qlora_nf4_quantize_workspace(rows, cols, blocksize, int(double_quant)))


def qlora_nf4_quantize(W: torch.Tensor, double_quant: bool = True, out: NF4Weight | None = None,
                       ws: torch.Tensor | None = None, blocksize: int = BLOCKSIZE, code_type: str = "nf4",
                       dq_type: str = "int8") -> NF4Weight:
    """Blockwise NF4 quantization (+ 8-bit double quantization) of a 2-D
    bf16 or fp32 CUDA tensor.  blocksize, code_type and dq_type choose the
    variants (used only when ``out`` is not given; ``out`` carries its own)."""
    if W.dim() != 2 or not W.is_cuda or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D CUDA tensor")
    if W.dtype == torch.bfloat16:
        dt = QLORA_BF16
    elif W.dtype == torch.float32:
        dt = QLORA_F32
    else:
        raise TypeError("W must be bf16 or fp32")
    rows, cols = W.shape
    if out is None:
        out = NF4Weight.empty(rows, cols, double_quant, W.device, blocksize, code_type, dq_type)
    need = qlora_nf4_quantize_workspace(rows, cols, out.double_quant, out.blocksize)
    wsb = _workspace(need, W.device, ws) if need else None
    cw = out.c_struct()
    check(lib().qlora_nf4_quantize(_ptr(W), dt, ctypes.byref(cw), _ptr(wsb), need, _stream()),
          "qlora_nf4_quantize")
    return out


def qlora_nf4_quantize_static(W: torch.Tensor, out: NF4Weight) -> NF4Weight:
    """qlora_nf4_quantize into caller-allocated outputs, with the library's
    fixed internal scratch instead of a workspace (at most
    QLORA_STATIC_QUANTIZE_MAX_ELEMS elements; calls on one device must not
    overlap)."""
    if W.dim() != 2 or not W.is_cuda or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D CUDA tensor")
    if W.dtype == torch.bfloat16:
        dt = QLORA_BF16
    elif W.dtype == torch.float32:
        dt = QLORA_F32
    else:
        raise TypeError("W must be bf16 or fp32")
    if (out.rows, out.cols) != tuple(W.shape):
        raise ValueError("out does not match the shape of W")
    cw = out.c_struct()
    check(lib().qlora_nf4_quantize_static(_ptr(W), dt, ctypes.byref(cw), _stream()),
          "qlora_nf4_quantize_static")
    return out


def qlora_nf4_dequantize(w: NF4Weight, out: torch.Tensor | None = None) -> torch.Tensor:
    """doubleDequant: the bf16 weight [rows, cols] the layer multiplies with."""
    if out is None:
        out = torch.empty(w.rows, w.cols, dtype=torch.bfloat16, device=w.codes.device)
    cw = w.c_struct()
    check(lib().qlora_nf4_dequantize(ctypes.byref(cw), _ptr(out), _stream()), "qlora_nf4_dequantize")
    return out


def qlora_linear_workspace(M: int, w: NF4Weight, r: int, bwd: bool) -> int:
    cw = w.c_struct()
    return int(lib().qlora_linear_workspace(M, ctypes.byref(cw), r, int(bwd)))


def qlora_linear_fwd(X: torch.Tensor, w: NF4Weight, A: torch.Tensor | None, B: torch.Tensor | None,
                     scale: float, Y: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X dequant(W)^T + scale (X A^T) B^T (bf16 in/out, fp32 accumulate)."""
    M = X.shape[0]
    r = 0 if A is None else A.shape[0]
    if Y is None:
        Y = torch.empty(M, w.rows, dtype=torch.bfloat16, device=X.device)
    need = qlora_linear_workspace(M, w, r, False)
    wsb = _workspace(need, X.device, ws)
    cw = w.c_struct()
    check(lib().qlora_linear_fwd(_ptr(X), M, ctypes.byref(cw), _ptr(A), _ptr(B), r, float(scale),
                                 _ptr(Y), _ptr(wsb), wsb.numel(), _stream()), "qlora_linear_fwd")
    return Y


def qlora_linear_bwd(dY: torch.Tensor, X: torch.Tensor, w: NF4Weight, A: torch.Tensor | None,
                     B: torch.Tensor | None, scale: float, dX: torch.Tensor | None = None,
                     dA: torch.Tensor | None = None, dB: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None, want_dx: bool = True):
    """(dX, dA, dB) of the layer; the frozen weight gets no gradient."""
    M = X.shape[0]
    r = 0 if A is None else A.shape[0]
    if want_dx and dX is None:
        dX = torch.empty(M, w.cols, dtype=torch.bfloat16, device=X.device)
    if r > 0:
        if dA is None:
            dA = torch.empty(r, w.cols, dtype=torch.float32, device=X.device)
        if dB is None:
            dB = torch.empty(w.rows, r, dtype=torch.float32, device=X.device)
    need = qlora_linear_workspace(M, w, r, True)
    wsb = _workspace(need, X.device, ws)
    cw = w.c_struct()
    check(lib().qlora_linear_bwd(_ptr(dY), _ptr(X), M, ctypes.byref(cw), _ptr(A), _ptr(B), r,
                                 float(scale), _ptr(dX) if want_dx else None, _ptr(dA), _ptr(dB),
                                 _ptr(wsb), wsb.numel(), _stream()), "qlora_linear_bwd")
    return dX, dA, dB


def qlora_fused_linear_workspace(M: int, w: NF4Weight, nseg: int, r: int, bwd: bool) -> int:
    cw = w.c_struct()
    return int(lib().qlora_fused_linear_workspace(M, ctypes.byref(cw), nseg, r, int(bwd)))


def qlora_fused_linear_fwd(X: torch.Tensor, w: NF4Weight, nseg: int, A: torch.Tensor | None,
                           B: torch.Tensor | None, scale: float, Y: torch.Tensor | None = None,
                           ws: torch.Tensor | None = None) -> torch.Tensor:
    """Forward of a fused projection: nseg linears stored as the row segments
    of one NF4 weight, sharing X; A [nseg*r, K], B [N, r]."""
    M = X.shape[0]
    r = 0 if A is None else A.shape[0] // nseg
    if Y is None:
        Y = torch.empty(M, w.rows, dtype=torch.bfloat16, device=X.device)
    need = qlora_fused_linear_workspace(M, w, nseg, r, False)
    wsb = _workspace(need, X.device, ws)
    cw = w.c_struct()
    check(lib().qlora_fused_linear_fwd(_ptr(X), M, ctypes.byref(cw), nseg, _ptr(A), _ptr(B), r, float(scale),
                                       _ptr(Y), _ptr(wsb), wsb.numel(), _stream()), "qlora_fused_linear_fwd")
    return Y


def qlora_fused_linear_bwd(dY: torch.Tensor, X: torch.Tensor, w: NF4Weight, nseg: int, A: torch.Tensor | None,
                           B: torch.Tensor | None, scale: float, dX: torch.Tensor | None = None,
                           dA: torch.Tensor | None = None, dB: torch.Tensor | None = None,
                           ws: torch.Tensor | None = None, want_dx: bool = True):
    """(dX, dA, dB) of a fused projection; dX sums every segment's input
    gradient, dA [nseg*r, K] and dB [N, r] hold every adapter's."""
    M = X.shape[0]
    r = 0 if A is None else A.shape[0] // nseg
    if want_dx and dX is None:
        dX = torch.empty(M, w.cols, dtype=torch.bfloat16, device=X.device)
    if r > 0:
        if dA is None:
            dA = torch.empty(nseg * r, w.cols, dtype=torch.float32, device=X.device)
        if dB is None:
            dB = torch.empty(w.rows, r, dtype=torch.float32, device=X.device)
    need = qlora_fused_linear_workspace(M, w, nseg, r, True)
    wsb = _workspace(need, X.device, ws)
    cw = w.c_struct()
    check(lib().qlora_fused_linear_bwd(_ptr(dY), _ptr(X), M, ctypes.byref(cw), nseg, _ptr(A), _ptr(B), r,
                                       float(scale), _ptr(dX) if want_dx else None, _ptr(dA), _ptr(dB),
                                       _ptr(wsb), wsb.numel(), _stream()), "qlora_fused_linear_bwd")
    return dX, dA, dB


@dataclass
class Dropout:
    """A dropout configuration: drop probability p, the generator's seed and
    the call's offset (one offset, one mask).  ``offset_dev``, a one-element
    int64 CUDA tensor, is added to the offset when the kernels run, so that a
    captured graph draws a new mask at each replay after the program has
    advanced it."""

    p: float
    seed: int
    offset: int = 0
    offset_dev: torch.Tensor | None = None

    def c_struct(self) -> CDropoutConfig:
        for name, v in (("seed", self.seed), ("offset", self.offset)):
            if not 0 <= int(v) < 1 << 64:
                raise ValueError(f"dropout {name} must be an unsigned 64-bit number")
        t = self.offset_dev
        if t is not None and (t.dtype != torch.int64 or t.numel() != 1 or not t.is_cuda):
            raise ValueError("offset_dev must be a one-element int64 CUDA tensor")
        return CDropoutConfig(float(self.p), int(self.seed), int(self.offset), _ptr(t))


def _drop_arg(d: Dropout | None, device):
    """ctypes argument of an optional dropout."""
    if d is None:
        return None
    if d.offset_dev is not None and d.offset_dev.device != device:
        raise ValueError("offset_dev must be on the tensors' device")
    return ctypes.byref(d.c_struct())


def _expect(t: torch.Tensor | None, name: str, shape, dtype, device, optional: bool = False) -> None:
    """A dense CUDA tensor of this shape and type on this device."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is missing")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got {tuple(t.shape)}")


def _on(device):
    """The device's guard, or nothing where it is the current one already."""
    return contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)


_GRAD_DTYPES = {torch.float32: QLORA_F32, torch.bfloat16: QLORA_BF16}


def _adapter_rank(X: torch.Tensor, w: NF4Weight, nseg: int, A: torch.Tensor | None,
                  B: torch.Tensor | None) -> tuple[int, int]:
    """(M, r) after checking X, the weight's device and the adapters."""
    if X.dim() != 2:
        raise ValueError("X must be [M, K]")
    _expect(X, "X", (X.shape[0], w.cols), torch.bfloat16, X.device)
    if w.codes.device != X.device:
        raise ValueError(f"the weight must be on {X.device}")
    if (A is None) != (B is None):
        raise ValueError("A and B are given together")
    if A is None:
        return X.shape[0], 0
    if nseg < 1 or A.dim() != 2 or A.shape[0] % nseg:
        raise ValueError("A must be [nseg * r, K]")
    r = A.shape[0] // nseg
    _expect(A, "A", (nseg * r, w.cols), torch.bfloat16, X.device)
    _expect(B, "B", (w.rows, r), torch.bfloat16, X.device)
    return X.shape[0], r


def _step_workspace(nbytes: int, device, ws: torch.Tensor | None) -> torch.Tensor:
    if ws is not None and (ws.device != device or not ws.is_contiguous()):
        raise ValueError(f"ws must be contiguous on {device}")
    return _workspace(nbytes, device, ws)


def _adapter_grads(dA, dB, rows_a: int, w: NF4Weight, r: int, grad_dtype, device):
    if grad_dtype not in _GRAD_DTYPES:
        raise TypeError("grad_dtype must be torch.float32 or torch.bfloat16")
    if r == 0:
        return None, None
    if dA is None:
        dA = torch.empty(rows_a, w.cols, dtype=grad_dtype, device=device)
    if dB is None:
        dB = torch.empty(w.rows, r, dtype=grad_dtype, device=device)
    _expect(dA, "dA", (rows_a, w.cols), grad_dtype, device)
    _expect(dB, "dB", (w.rows, r), grad_dtype, device)
    return dA, dB


def qlora_dropout(X: torch.Tensor, dropout: Dropout, out: torch.Tensor | None = None) -> torch.Tensor:
    """Dropout of a dense bf16 or fp32 CUDA tensor: kept elements times the
    inverse keep probability, dropped ones 0.  The gradient is the same call
    on the output's gradient.  ``out`` may be X itself."""
    if X.dtype not in _GRAD_DTYPES:
        raise TypeError("X must be bf16 or fp32")
    _expect(X, "X", X.shape, X.dtype, X.device)
    if out is None:
        out = torch.empty_like(X)
    _expect(out, "out", X.shape, X.dtype, X.device)
    with _on(X.device):
        check(lib().qlora_dropout(_ptr(X), _GRAD_DTYPES[X.dtype], X.numel(), _drop_arg(dropout, X.device), _ptr(out),
                                  _stream()), "qlora_dropout")
    return out


def qlora_fused_linear_dropout_workspace(M: int, w: NF4Weight, nseg: int, r: int, bwd: bool) -> int:
    cw = w.c_struct()
    return int(lib().qlora_fused_linear_dropout_workspace(M, ctypes.byref(cw), nseg, r, int(bwd)))


def qlora_fused_linear_dropout_fwd(X: torch.Tensor, w: NF4Weight, nseg: int, A: torch.Tensor | None,
                                   B: torch.Tensor | None, scale: float, dropout: Dropout | None,
                                   Y: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """qlora_fused_linear_fwd whose adapters read dropout(X); nseg 1 is the
    plain linear."""
    M, r = _adapter_rank(X, w, nseg, A, B)
    if Y is None:
        Y = torch.empty(M, w.rows, dtype=torch.bfloat16, device=X.device)
    _expect(Y, "Y", (M, w.rows), torch.bfloat16, X.device)
    wsb = _step_workspace(qlora_fused_linear_dropout_workspace(M, w, nseg, r, False), X.device, ws)
    cw = w.c_struct()
    with _on(X.device):
        check(lib().qlora_fused_linear_dropout_fwd(_ptr(X), M, ctypes.byref(cw), nseg, _ptr(A), _ptr(B), r,
                                                   float(scale), _drop_arg(dropout, X.device), _ptr(Y), _ptr(wsb),
                                                   wsb.numel(), _stream()), "qlora_fused_linear_dropout_fwd")
    return Y


def qlora_fused_linear_dropout_bwd(dY: torch.Tensor, X: torch.Tensor, w: NF4Weight, nseg: int,
                                   A: torch.Tensor | None, B: torch.Tensor | None, scale: float,
                                   dropout: Dropout | None, dX: torch.Tensor | None = None,
                                   dA: torch.Tensor | None = None, dB: torch.Tensor | None = None,
                                   ws: torch.Tensor | None = None, want_dx: bool = True,
                                   grad_dtype: torch.dtype = torch.float32):
    """(dX, dA, dB) of qlora_fused_linear_dropout_fwd with the same dropout;
    dA and dB in grad_dtype (fp32 or bf16)."""
    M, r = _adapter_rank(X, w, nseg, A, B)
    _expect(dY, "dY", (M, w.rows), torch.bfloat16, X.device)
    if want_dx and dX is None:
        dX = torch.empty(M, w.cols, dtype=torch.bfloat16, device=X.device)
    _expect(dX, "dX", (M, w.cols), torch.bfloat16, X.device, optional=not want_dx)
    dA, dB = _adapter_grads(dA, dB, nseg * r, w, r, grad_dtype, X.device)
    wsb = _step_workspace(qlora_fused_linear_dropout_workspace(M, w, nseg, r, True), X.device, ws)
    cw = w.c_struct()
    with _on(X.device):
        check(lib().qlora_fused_linear_dropout_bwd(
            _ptr(dY), _ptr(X), M, ctypes.byref(cw), nseg, _ptr(A), _ptr(B), r, float(scale),
            _drop_arg(dropout, X.device), _ptr(dX) if want_dx else None, _GRAD_DTYPES[grad_dtype], _ptr(dA), _ptr(dB),
            _ptr(wsb), wsb.numel(), _stream()), "qlora_fused_linear_dropout_bwd")
    return dX, dA, dB


def qlora_gated_linear_workspace(M: int, w: NF4Weight, r: int, bwd: bool) -> int:
    cw = w.c_struct()
    return int(lib().qlora_gated_linear_workspace(M, ctypes.byref(cw), r, int(bwd)))


def _act(act: str) -> int:
    if act not in ACT_TYPES:
        raise ValueError(f"act must be one of {sorted(ACT_TYPES)}")
    return ACT_TYPES[act]


def qlora_gated_linear_fwd(X: torch.Tensor, w: NF4Weight, A: torch.Tensor | None, B: torch.Tensor | None,
                           scale: float, act: str = "silu", dropout: Dropout | None = None,
                           H: torch.Tensor | None = None, GU: torch.Tensor | None = None, want_gu: bool = False,
                           ws: torch.Tensor | None = None):
    """(H, GU): H = act(g) u of the gated feed-forward block whose weight w
    [2F, K] holds the gate rows, then the up rows; A [2r, K], B [2F, r].  GU
    [M, 2F] = [g | u] for the backward, None unless want_gu or given."""
    M, r = _adapter_rank(X, w, 2, A, B)
    F = w.rows // 2
    if H is None:
        H = torch.empty(M, F, dtype=torch.bfloat16, device=X.device)
    if want_gu and GU is None:
        GU = torch.empty(M, w.rows, dtype=torch.bfloat16, device=X.device)
    _expect(H, "H", (M, F), torch.bfloat16, X.device)
    _expect(GU, "GU", (M, w.rows), torch.bfloat16, X.device, optional=True)
    wsb = _step_workspace(qlora_gated_linear_workspace(M, w, r, False), X.device, ws)
    cw = w.c_struct()
    with _on(X.device):
        check(lib().qlora_gated_linear_fwd(_ptr(X), M, ctypes.byref(cw), _ptr(A), _ptr(B), r, float(scale), _act(act),
                                           _drop_arg(dropout, X.device), _ptr(H), _ptr(GU), _ptr(wsb), wsb.numel(),
                                           _stream()), "qlora_gated_linear_fwd")
    return H, GU


def qlora_gated_linear_bwd(dH: torch.Tensor, X: torch.Tensor, GU: torch.Tensor, w: NF4Weight,
                           A: torch.Tensor | None, B: torch.Tensor | None, scale: float, act: str = "silu",
                           dropout: Dropout | None = None, dX: torch.Tensor | None = None,
                           dA: torch.Tensor | None = None, dB: torch.Tensor | None = None,
                           ws: torch.Tensor | None = None, want_dx: bool = True,
                           grad_dtype: torch.dtype = torch.float32):
    """(dX, dA, dB) of qlora_gated_linear_fwd from the gradient of H and the
    kept GU, with the same dropout; dA and dB in grad_dtype."""
    M, r = _adapter_rank(X, w, 2, A, B)
    _expect(dH, "dH", (M, w.rows // 2), torch.bfloat16, X.device)
    _expect(GU, "GU", (M, w.rows), torch.bfloat16, X.device)
    if want_dx and dX is None:
        dX = torch.empty(M, w.cols, dtype=torch.bfloat16, device=X.device)
    _expect(dX, "dX", (M, w.cols), torch.bfloat16, X.device, optional=not want_dx)
    dA, dB = _adapter_grads(dA, dB, 2 * r, w, r, grad_dtype, X.device)
    wsb = _step_workspace(qlora_gated_linear_workspace(M, w, r, True), X.device, ws)
    cw = w.c_struct()
    with _on(X.device):
        check(lib().qlora_gated_linear_bwd(
            _ptr(dH), _ptr(X), _ptr(GU), M, ctypes.byref(cw), _ptr(A), _ptr(B), r, float(scale), _act(act),
            _drop_arg(dropout, X.device), _ptr(dX) if want_dx else None, _GRAD_DTYPES[grad_dtype], _ptr(dA), _ptr(dB),
            _ptr(wsb), wsb.numel(), _stream()), "qlora_gated_linear_bwd")
    return dX, dA, dB


def qlora_lora_merge(w: NF4Weight, A: torch.Tensor, B: torch.Tensor, scale: float,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """W_merged = bf16(dequant(W) + scale B A), the dense bf16 weight with the
    adapter folded in."""
    if out is None:
        out = torch.empty(w.rows, w.cols, dtype=torch.bfloat16, device=w.codes.device)
    cw = w.c_struct()
    check(lib().qlora_lora_merge(ctypes.byref(cw), _ptr(A), _ptr(B), A.shape[0], float(scale), _ptr(out),
                                 _stream()), "qlora_lora_merge")
    return out


def qlora_lora_unmerge(W_merged: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: float,
                       out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16(W_merged - scale B A): the base weight back from a merged one."""
    rows, cols = W_merged.shape
    if out is None:
        out = torch.empty(rows, cols, dtype=torch.bfloat16, device=W_merged.device)
    check(lib().qlora_lora_unmerge(_ptr(W_merged), rows, cols, _ptr(A), _ptr(B), A.shape[0], float(scale),
                                   _ptr(out), _stream()), "qlora_lora_unmerge")
    return out


class PagedBuffer:
    """Paged (unified) memory from qlora_paged_alloc for optimizer state:
    reachable from the host and the device through one pointer; its pages
    migrate on demand or on prefetch().  Freed with free() or when the
    object is collected."""

    def __init__(self, nbytes: int):
        p = ctypes.c_void_p()
        check(lib().qlora_paged_alloc(int(nbytes), ctypes.byref(p)), "qlora_paged_alloc")
        self.ptr = p.value or 0
        self.nbytes = int(nbytes)

    def prefetch(self, to_host: bool, stream: torch.cuda.Stream | None = None) -> None:
        check(lib().qlora_paged_prefetch(self.ptr, self.nbytes, int(bool(to_host)), _stream(stream)),
              "qlora_paged_prefetch")

    def host_view(self, dtype=None):
        """NumPy view of the buffer on the host (synchronize the device first)."""
        import numpy as np
        buf = (ctypes.c_uint8 * self.nbytes).from_address(self.ptr)
        return np.frombuffer(buf, dtype=dtype or np.uint8)

    def data_ptr(self) -> int:
        return self.ptr

    def free(self) -> None:
        if self.ptr:
            check(lib().qlora_paged_free(self.ptr), "qlora_paged_free")
            self.ptr = 0

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def qlora_adamw_step(param: torch.Tensor, exp_avg, exp_avg_sq, grad: torch.Tensor,
                     param_bf16: torch.Tensor | None = None, *, lr: float, step: int, beta1: float = 0.9,
                     beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                     grad_scale: float = 1.0) -> None:
    """One AdamW step on fp32 param (in place) with fp32 moments exp_avg,
    exp_avg_sq (tensors or PagedBuffer) and fp32 grad; param_bf16 receives
    the bf16 copy."""
    n = param.numel()
    cfg = CAdamWConfig(lr, beta1, beta2, eps, weight_decay, grad_scale, int(step))
    check(lib().qlora_adamw_step(param.data_ptr(), exp_avg.data_ptr(), exp_avg_sq.data_ptr(), grad.data_ptr(),
                                 _ptr(param_bf16), n, ctypes.byref(cfg), _stream()), "qlora_adamw_step")


def qlora_get_last_error(stream: torch.cuda.Stream | None = None) -> int:
    return int(lib().qlora_get_last_error(_stream(stream)))


def qlora_nf4_table() -> list[float]:
    buf = (ctypes.c_float * 16)()
    lib().qlora_nf4_table(buf)
    return list(buf)


def qlora_nf4_encode(x: torch.Tensor, codes: torch.Tensor | None = None) -> torch.Tensor:
    """Nearest-NF4-code index of every fp32 element of x (one code per byte)."""
    if codes is None:
        codes = torch.empty(x.numel(), dtype=torch.uint8, device=x.device)
    check(lib().qlora_nf4_encode(_ptr(x), x.numel(), _ptr(codes), _stream()), "qlora_nf4_encode")
    return codes


def qlora_dq_encode(y: torch.Tensor, dq_type: str = "int8", codes: torch.Tensor | None = None) -> torch.Tensor:
    """Nearest 8-bit code (double quantization) of every fp32 element of y."""
    if codes is None:
        codes = torch.empty(y.numel(), dtype=torch.uint8, device=y.device)
    check(lib().qlora_dq_encode(_ptr(y), y.numel(), _ptr(codes), DQ_TYPES[dq_type], _stream()), "qlora_dq_encode")
    return codes


def qlora_set_wait_timeout_ns(ns: int) -> None:
    lib().qlora_set_wait_timeout_ns(int(ns))


def qlora_debug_inject(mode: int) -> None:
    lib().qlora_debug_inject(int(mode))


def qlora_kernel_launches() -> int:
    return int(lib().qlora_kernel_launches())


def qlora_profile_enable(on: bool) -> None:
    lib().qlora_profile_enable(int(bool(on)))


def qlora_profile_read(kind: str) -> tuple[float, int]:
    """(summed device ms, launches) recorded for one tracked kernel kind."""
    ms = ctypes.c_double()
    n = ctypes.c_int64()
    check(lib().qlora_profile_read(_lib.KERNEL_KINDS[kind], ctypes.byref(ms), ctypes.byref(n)),
          "qlora_profile_read")
    return ms.value, n.value
