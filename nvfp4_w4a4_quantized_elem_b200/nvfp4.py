"""ctypes binding of libnvfp4.so (C ABI in include/nvfp4.h).

Argument marshalling only: every step of the NVFP4 W4A4 path runs in the CUDA
library. PyTorch supplies device memory (output tensors allocated here for
convenience; callers may pass their own) and the current stream. There is no
CPU fallback: if the library is missing or a call fails, an exception is
raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")
# Dynamic quantization of x with rows * k * 2 bytes up to this bound runs
# one kernel (NVFP4_ONE_PASS_MAX_BYTES of nvfp4.h): no amax pass.
ONE_PASS_MAX_BYTES = 65536
# nvfp4_linear quantizes at most this many tokens inside the few-token GEMM
# (NVFP4_LINEAR_IN_KERNEL_MAX_TOKENS of nvfp4.h)
LINEAR_IN_KERNEL_MAX_TOKENS = 8

NVFP4_OK = 0
STATUS_NAMES = {0: "NVFP4_OK", 1: "NVFP4_ERR_INVALID_ARG", 2: "NVFP4_ERR_UNSUPPORTED",
                3: "NVFP4_ERR_MISALIGNED", 4: "NVFP4_ERR_CUDA", 5: "NVFP4_ERR_TIMEOUT"}

# every symbol include/nvfp4.h declares
EXPORTS = ("nvfp4_status_string", "nvfp4_sf_bytes", "nvfp4_quantize_workspace_bytes",
           "nvfp4_quantize", "nvfp4_quantize_noalloc", "nvfp4_calibrate_global",
           "nvfp4_gemm_workspace_bytes", "nvfp4_gemm", "nvfp4_linear_workspace_bytes",
           "nvfp4_linear", "nvfp4_gemm_epilogue", "nvfp4_linear_epilogue",
           "nvfp4_gemm_swiglu_quant",
           "nvfp4_gemm_swiglu_quant_dynamic_workspace_bytes", "nvfp4_gemm_swiglu_quant_dynamic",
           "nvfp4_fuse_group_scales", "nvfp4_silu_mul", "nvfp4_read_fault",
           "nvfp4_linear_attention_workspace_bytes", "nvfp4_linear_attention",
           "nvfp4_linear_attention_step",
           "nvfp4_selftest_wait_timeout", "nvfp4_selftest_gemm_stall",
           "nvfp4_selftest_linear_attention_stall")

_BF16, _FP32 = torch.bfloat16, torch.float32

# activations of the GEMM epilogue (nvfp4_activation)
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

_lib = None
_lock = threading.Lock()


class NVFP4Error(RuntimeError):
    def __init__(self, what: str, status: int):
        super().__init__(f"{what} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libnvfp4.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} not found: build it with "
                "`python -m nvfp4_w4a4_quantized_elem_b200.build` (nvcc, sm_100a)")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I, SZ, U32P = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                               ctypes.c_size_t, ctypes.POINTER(ctypes.c_uint32))
        prompts = [P, I64, P, I64, P, I64, P, P, ctypes.c_float, I64, I, I, I, I, I64, P, P, I64,
                   P, P, P, I64, P, SZ]
        sigs = {
            "nvfp4_status_string": (ctypes.c_char_p, [I]),
            "nvfp4_sf_bytes": (SZ, [I64, I64]),
            "nvfp4_quantize_workspace_bytes": (SZ, [I64, I64]),
            "nvfp4_quantize": (I, [P, I64, I64, I64, P, P, P, P, P, SZ, P]),
            "nvfp4_quantize_noalloc": (I, [P, I64, I64, I64, P, P, P, P, P]),
            "nvfp4_calibrate_global": (I, [P, I64, I64, I64, P, P, P, SZ, P]),
            "nvfp4_gemm_workspace_bytes": (SZ, [I64, I64, I64]),
            "nvfp4_gemm": (I, [P, P, P, P, P, P, P, I, I64, I64, I64, I64, P, SZ, P]),
            "nvfp4_linear_workspace_bytes": (SZ, [I64, I64, I64]),
            "nvfp4_linear": (I, [P, I64, I64, I64, P, P, P, P, I64, P, I, I64, P, SZ, P]),
            "nvfp4_gemm_epilogue": (I, [P, P, P, P, P, P, P, I, P, I64, P, I, I64, I64, I64, I64,
                                        P, SZ, P]),
            "nvfp4_linear_epilogue": (I, [P, I64, I64, I64, P, P, P, P, I64, P, I, P, I64, P, I,
                                          I64, P, SZ, P]),
            "nvfp4_gemm_swiglu_quant": (I, [P, P, P, P, P, P, P, P, P, I64, I64, I64, P]),
            "nvfp4_gemm_swiglu_quant_dynamic_workspace_bytes": (SZ, [I64, I64]),
            "nvfp4_gemm_swiglu_quant_dynamic": (I, [P, P, P, P, P, P, P, P, P, I64, I64, I64,
                                                    P, SZ, P]),
            "nvfp4_fuse_group_scales": (I, [I, P, I64, P, P, P, P, P]),
            "nvfp4_silu_mul": (I, [P, I64, I64, I64, P, I64, P]),
            "nvfp4_linear_attention_workspace_bytes": (SZ, [I64, I64, I, I, I]),
            "nvfp4_linear_attention": (I, [*prompts, P]),
            "nvfp4_selftest_linear_attention_stall": (I, [*prompts, I, I, ctypes.c_uint64, P]),
            "nvfp4_linear_attention_step": (I, [P, I64, P, I64, P, I64, P, P, ctypes.c_float, I64,
                                                I, I, I, I, P, I64, P, P, I64, P]),
            "nvfp4_read_fault": (I, [P, U32P]),
            "nvfp4_selftest_wait_timeout": (I, [ctypes.c_uint64, P]),
            "nvfp4_selftest_gemm_stall": (I, [P, P, P, P, P, P, P, I64, I64, I64, ctypes.c_uint64,
                                              P, SZ, P]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
        return L


def _check(status: int, what: str) -> None:
    if status != NVFP4_OK:
        raise NVFP4Error(what, status)


# A call of a few microseconds on the GPU waits for the host otherwise: plain
# integers go through ctypes as they are, and the current stream is asked for
# by its handle (torch.cuda.current_stream() builds an object, ~3 us).
def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream: torch.cuda.Stream | None) -> int:
    if stream is not None:
        return stream.cuda_stream
    torch.cuda.init()
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


# Buffers that a call makes for itself belong to the stream its kernels run on:
# made (or zero-filled) on the current stream, nothing would order the fill, or
# what a recycled block still serves, before them. `stream` None is the current
# stream. What is handed to the caller is recorded as used on the caller's
# stream, so that its memory is not reused under work queued there. The inputs
# are the caller's: ordered before `stream`, and kept until it has read them.
def _on(stream: torch.cuda.Stream | None):
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _empty(shape, dtype: torch.dtype, device, stream: torch.cuda.Stream | None) -> torch.Tensor:
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _given(t: torch.Tensor, stream: torch.cuda.Stream | None) -> torch.Tensor:
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _empty_nvfp4(rows: int, k: int, device, stream: torch.cuda.Stream | None) -> NVFP4Tensor:
    if stream is None:
        return NVFP4Tensor.empty(rows, k, device)
    with torch.cuda.stream(stream):
        t = NVFP4Tensor.empty(rows, k, device)
    for part in (t.codes, t.sf, t.global_scale):
        _given(part, stream)
    return t


def _require_cuda(t: torch.Tensor, name: str, dtype: torch.dtype | None = None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _scratch(workspace: torch.Tensor | None, dev: int) -> tuple[int | None, int]:
    """Pointer and bytes of a caller's workspace on cuda:``dev``."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _global(g: torch.Tensor | None, name: str, dev: int) -> int | None:
    """Pointer of a global scale on cuda:``dev``."""
    if g is None:
        return None
    if g.get_device() != dev or g.dtype is not _FP32 or g.numel() < 1:
        raise ValueError(f"{name} must be a {_FP32} element on cuda:{dev}")
    return g.data_ptr()


def _operand(t: NVFP4Tensor, name: str, dev: int) -> tuple[int, int, int]:
    """Pointers of codes, scales and global of an operand on cuda:``dev``."""
    codes, sf, g = t.codes, t.sf, t.global_scale
    if dev < 0 or codes.get_device() != dev or sf.get_device() != dev or g.get_device() != dev:
        raise ValueError(f"{name} must be on the CUDA device of the call's other tensors")
    return codes.data_ptr(), sf.data_ptr(), g.data_ptr()


def _output(t: NVFP4Tensor, rows: int, k: int, dev: int) -> tuple[int, int, int]:
    """The same of an output for [rows, k]."""
    if (t.rows, t.k) != (rows, k):
        raise ValueError(f"out must be an NVFP4 tensor for [{rows}, {k}]")
    return _operand(t, "out", dev)


def sf_bytes(rows: int, k: int) -> int:
    return int(lib().nvfp4_sf_bytes(rows, k))


def quantize_workspace_bytes(rows: int, k: int) -> int:
    return int(lib().nvfp4_quantize_workspace_bytes(rows, k))


@dataclass
class NVFP4Tensor:
    """A [rows, k] tensor in NVFP4: packed E2M1 codes, swizzled E4M3 block
    scales and the FP32 global scale (a 1-element device tensor)."""
    codes: torch.Tensor        # uint8 [rows, k // 2]
    sf: torch.Tensor           # uint8 [sf_bytes(rows, k)]
    global_scale: torch.Tensor  # float32 [1]
    rows: int
    k: int

    def __post_init__(self):
        # once, not in every call: 8 bits each, codes [rows, k/2], scales padded to
        # 128 rows and 4 blocks of 16; the calls hand them on as pointers
        codes, sf, g = self.codes, self.sf, self.global_scale
        if (codes.numel() * 2 < self.rows * self.k or codes.element_size() != 1
                or sf.numel() < -(-self.rows // 128) * 128 * (-(-self.k // 64) * 4)
                or sf.element_size() != 1 or not codes.is_contiguous() or not sf.is_contiguous()):
            raise ValueError("an NVFP4 tensor needs contiguous 8-bit codes and scales for "
                             f"[{self.rows}, {self.k}]")
        if g.dtype is not _FP32 or g.numel() < 1:
            raise ValueError(f"an NVFP4 tensor's global scale must be a {_FP32} element")

    @staticmethod
    def empty(rows: int, k: int, device="cuda") -> "NVFP4Tensor":
        t = object.__new__(NVFP4Tensor)  # right as made: without __post_init__
        t.codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=device)
        t.sf = torch.empty(sf_bytes(rows, k), dtype=torch.uint8, device=device)
        t.global_scale = torch.empty(1, dtype=torch.float32, device=device)
        t.rows, t.k = rows, k
        return t


def quantize(x: torch.Tensor, global_scale: torch.Tensor | None = None,
             out: NVFP4Tensor | None = None, workspace: torch.Tensor | None = None,
             stream: torch.cuda.Stream | None = None) -> NVFP4Tensor:
    """nvfp4_quantize: bf16 [rows, k] (rows may be strided) -> NVFP4Tensor.
    ``global_scale`` None => dynamic global (amax pass + quantizer; one
    kernel when x is at most ONE_PASS_MAX_BYTES)."""
    _require_cuda(x, "x", torch.bfloat16)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride along k")
    rows, k = x.shape
    if out is None:
        out = _empty_nvfp4(rows, k, x.device, stream)
    if global_scale is None and workspace is None:
        workspace = _empty(quantize_workspace_bytes(rows, k), torch.uint8, x.device, stream)
    dev = x.get_device()
    st = lib().nvfp4_quantize(_ptr(x), rows, k, x.stride(0),
                              _global(global_scale, "global_scale", dev),
                              *_output(out, rows, k, dev), *_scratch(workspace, dev),
                              _stream(stream))
    _check(st, "nvfp4_quantize")
    return out


def quantize_noalloc(x: torch.Tensor, out: NVFP4Tensor, global_scale: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None) -> NVFP4Tensor:
    """nvfp4_quantize_noalloc: as quantize(), for callers that cannot
    allocate device memory. No workspace: the amax pass uses a fixed device
    array inside the library (shared by every call on the device; calls that
    overlap on the GPU race). The caller supplies the output buffers."""
    _require_cuda(x, "x", torch.bfloat16)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride along k")
    rows, k = x.shape
    dev = x.get_device()
    st = lib().nvfp4_quantize_noalloc(_ptr(x), rows, k, x.stride(0),
                                      _global(global_scale, "global_scale", dev),
                                      *_output(out, rows, k, dev), _stream(stream))
    _check(st, "nvfp4_quantize_noalloc")
    return out


class Calibrator:
    """Static global scale from a stream of calibration batches
    (nvfp4_calibrate_global): observe() each batch, then use .global_scale
    as quantize(..., global_scale=...)."""

    def __init__(self, device="cuda"):
        self.running_amax = torch.zeros(1, dtype=torch.float32, device=device)
        self.global_scale = torch.ones(1, dtype=torch.float32, device=device)
        self._ws = self._ws_stream = None

    def observe(self, x: torch.Tensor, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
        _require_cuda(x, "x", torch.bfloat16)
        if x.dim() != 2 or x.stride(1) != 1:
            raise ValueError("x must be 2-D with unit stride along k")
        rows, k = x.shape
        need = quantize_workspace_bytes(rows, k)
        if self._ws is None or self._ws.numel() < need or self._ws_stream != _stream(stream):
            self._ws = _empty(need, torch.uint8, x.device, stream)
            self._ws_stream = _stream(stream)
        st = lib().nvfp4_calibrate_global(_ptr(x), rows, k, x.stride(0), _ptr(self.running_amax),
                                          _ptr(self.global_scale), _ptr(self._ws), self._ws.numel(),
                                          _stream(stream))
        _check(st, "nvfp4_calibrate_global")
        return self.global_scale


_Y_TYPES = {_BF16: 0, _FP32: 1}


def _product(out: torch.Tensor | None, dtype: torch.dtype, m: int, n: int, dev: int, like: torch.Tensor,
             stream: torch.cuda.Stream | None):
    """The [m, n] output of a product on cuda:``dev``, made or checked: (out,
    (pointer, type, row pitch))."""
    if out is None:
        if dtype not in _Y_TYPES:
            raise ValueError(f"out must be bf16/fp32, not {dtype}")
        out = _given(_empty((m, n), dtype, like.device, stream), stream)
        return out, (out.data_ptr(), _Y_TYPES[dtype], n)
    if out.dtype not in _Y_TYPES or out.shape != (m, n) or out.stride(1) != 1:
        raise ValueError(f"out must be bf16/fp32 [{m}, {n}] with unit column stride")
    if out.get_device() != dev:
        raise ValueError(f"out must be on cuda:{dev}")
    return out, (out.data_ptr(), _Y_TYPES[out.dtype], out.stride(0))


def _epilogue(bias: torch.Tensor | None, activation: str, residual: torch.Tensor | None,
              m: int, n: int, device: torch.device):
    """Checked epilogue arguments: (bias pointer, activation code, residual
    pointer, residual row pitch)."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    for t, name in ((bias, "bias"), (residual, "residual")):
        if t is not None:
            _require_cuda(t, name, torch.bfloat16)
            if t.device != device:
                raise ValueError(f"{name} must be on {device}")
    if bias is not None and (tuple(bias.shape) != (n,) or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous vector of {n}")
    ldr = 0
    if residual is not None:
        if tuple(residual.shape) != (m, n) or (n > 1 and residual.stride(1) != 1):
            raise ValueError(f"residual must be [{m}, {n}] with unit column stride")
        # a single row's pitch is free; a C caller may give any valid one
        ldr = residual.stride(0) if m > 1 else -(-n // 8) * 8
    return _ptr(bias), ACTIVATIONS[activation], _ptr(residual), ldr


def gemm_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(lib().nvfp4_gemm_workspace_bytes(m, n, k))


def gemm(a: NVFP4Tensor, b: NVFP4Tensor, out: torch.Tensor | None = None,
         out_dtype: torch.dtype = torch.bfloat16, workspace: torch.Tensor | None = None,
         stream: torch.cuda.Stream | None = None, bias: torch.Tensor | None = None,
         activation: str = "none", residual: torch.Tensor | None = None) -> torch.Tensor:
    """nvfp4_gemm: Y[m, n] = dequant(A) @ dequant(B).T (A = activations
    [m, k], B = weights [n, k]); bf16 or fp32 output. ``workspace`` (at least
    gemm_workspace_bytes) lets few-token GEMMs share the work across all SMs
    (stream-K). With ``bias`` (bf16 [n]), ``activation`` (a key of ACTIVATIONS)
    or ``residual`` (bf16 [m, n], may be ``out``): nvfp4_gemm_epilogue,
    Y = act(product + bias) + residual in FP32, rounded once."""
    if a.k != b.k:
        raise ValueError("k mismatch")
    m, n, k = a.rows, b.rows, a.k
    dev = a.codes.get_device()
    operands = (*_operand(a, "a", dev), *_operand(b, "b", dev))
    out, y = _product(out, out_dtype, m, n, dev, a.codes, stream)
    ws, ws_bytes = _scratch(workspace, dev)
    if bias is not None or residual is not None or activation != "none":
        st = lib().nvfp4_gemm_epilogue(
            *operands, *_epilogue(bias, activation, residual, m, n, a.codes.device), *y, m, n, k,
            ws, ws_bytes, _stream(stream))
        _check(st, "nvfp4_gemm_epilogue")
        return out
    st = lib().nvfp4_gemm(*operands, *y, m, n, k, ws, ws_bytes, _stream(stream))
    _check(st, "nvfp4_gemm")
    return out


def interleave_gate_up(w_gate_up: torch.Tensor) -> torch.Tensor:
    """Row order nvfp4_gemm_swiglu_quant expects: [2*ffn, k] with gate rows
    [0, ffn) and up rows [ffn, 2ffn) -> blocks of 128 (gate b, up b, ...).
    Offline weight preparation (a row permutation)."""
    two_ffn = w_gate_up.shape[0]
    ffn = two_ffn // 2
    if two_ffn % 256:
        raise ValueError("ffn must be a multiple of 128")
    idx = torch.arange(two_ffn, device=w_gate_up.device).view(2, ffn // 128, 128)
    return w_gate_up[idx.transpose(0, 1).reshape(-1)]


def gemm_swiglu_quant(a: NVFP4Tensor, b_interleaved: NVFP4Tensor, h_global: torch.Tensor,
                      out: NVFP4Tensor | None = None,
                      stream: torch.cuda.Stream | None = None) -> NVFP4Tensor:
    """nvfp4_gemm_swiglu_quant: NVFP4 h = quantize(silu(gate) * up, h_global)
    straight from the gate_up GEMM (weights row-interleaved, see
    interleave_gate_up)."""
    if a.k != b_interleaved.k:
        raise ValueError("k mismatch")
    m, ffn, k = a.rows, b_interleaved.rows // 2, a.k
    dev = a.codes.get_device()
    h_ptr = _global(h_global, "h_global", dev)
    if out is None:
        out = _empty_nvfp4(m, ffn, a.codes.device, stream)
    with _on(stream):
        out.global_scale.copy_(h_global.reshape(1))
    st = lib().nvfp4_gemm_swiglu_quant(*_operand(a, "a", dev),
                                       *_operand(b_interleaved, "b_interleaved", dev), h_ptr,
                                       *_output(out, m, ffn, dev)[:2], m, ffn, k, _stream(stream))
    _check(st, "nvfp4_gemm_swiglu_quant")
    return out


def swiglu_quant_dynamic_workspace(m: int, ffn: int, device="cuda") -> torch.Tensor:
    """Workspace of gemm_swiglu_quant_dynamic (bf16 h + per-CTA maxima)."""
    nb = int(lib().nvfp4_gemm_swiglu_quant_dynamic_workspace_bytes(m, ffn))
    return torch.empty(nb, dtype=torch.uint8, device=device)


def gemm_swiglu_quant_dynamic(a: NVFP4Tensor, b_interleaved: NVFP4Tensor,
                              out: NVFP4Tensor | None = None,
                              workspace: torch.Tensor | None = None,
                              stream: torch.cuda.Stream | None = None) -> NVFP4Tensor:
    """nvfp4_gemm_swiglu_quant_dynamic: NVFP4 h = quantize(silu(gate) * up)
    with h's own dynamic global (weights row-interleaved, see
    interleave_gate_up). ``workspace`` from swiglu_quant_dynamic_workspace()
    (allocated here when None); its first m*ffn*2 bytes hold h in bf16."""
    if a.k != b_interleaved.k:
        raise ValueError("k mismatch")
    m, ffn, k = a.rows, b_interleaved.rows // 2, a.k
    if out is None:
        out = _empty_nvfp4(m, ffn, a.codes.device, stream)
    if workspace is None:
        with _on(stream):
            workspace = swiglu_quant_dynamic_workspace(m, ffn, a.codes.device)
    dev = a.codes.get_device()
    st = lib().nvfp4_gemm_swiglu_quant_dynamic(
        *_operand(a, "a", dev), *_operand(b_interleaved, "b_interleaved", dev),
        *_output(out, m, ffn, dev), m, ffn, k, *_scratch(workspace, dev), _stream(stream))
    _check(st, "nvfp4_gemm_swiglu_quant_dynamic")
    return out


def fuse_group_scales(modules: list[NVFP4Tensor], sf_out: torch.Tensor | None = None,
                      global_out: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None):
    """nvfp4_fuse_group_scales: fold per-module globals into one (g* = min)
    and write the swizzled scales of the row-concatenated group.
    Returns (sf_fused, global_fused)."""
    n = len(modules)
    k = modules[0].k
    total = sum(m.rows for m in modules)
    dev = modules[0].codes.device
    index = modules[0].codes.get_device()
    if any(m.k != k for m in modules):
        raise ValueError("the modules of a group share k")
    sf_in = [_operand(m, "every module", index)[1] for m in modules]
    if sf_out is None:
        sf_out = _given(_empty(sf_bytes(total, k), torch.uint8, dev, stream), stream)
    elif (sf_out.get_device() != index or not sf_out.is_contiguous() or sf_out.element_size() != 1
          or sf_out.numel() < sf_bytes(total, k)):
        raise ValueError(f"sf_out must be {sf_bytes(total, k)} contiguous bytes on {dev}")
    if global_out is None:
        global_out = _given(_empty(1, torch.float32, dev, stream), stream)
    global_ptr = _global(global_out, "global_out", index)
    with _on(stream):
        globals_in = torch.cat([m.global_scale for m in modules])
    rows = (ctypes.c_int64 * n)(*[m.rows for m in modules])
    ptrs = (ctypes.c_void_p * n)(*sf_in)
    st = lib().nvfp4_fuse_group_scales(n, ctypes.cast(rows, ctypes.c_void_p), k,
                                       ctypes.cast(ptrs, ctypes.c_void_p), _ptr(globals_in),
                                       _ptr(sf_out), global_ptr, _stream(stream))
    _check(st, "nvfp4_fuse_group_scales")
    return sf_out, global_out


def fuse_group(modules: list[NVFP4Tensor], stream=None) -> NVFP4Tensor:
    """The repaired fused tensor: concatenated codes, folded scales, g*."""
    sf, g = fuse_group_scales(modules, stream=stream)
    with _on(stream):
        codes = torch.cat([m.codes for m in modules], dim=0)
    _given(codes, stream)
    return NVFP4Tensor(codes, sf, g, codes.shape[0], modules[0].k)


def silu_mul(y: torch.Tensor, out: torch.Tensor | None = None,
             stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """nvfp4_silu_mul: h = silu(y[:, :n]) * y[:, n:] in bf16."""
    _require_cuda(y, "y", torch.bfloat16)
    if y.dim() != 2 or y.shape[1] % 2 or y.stride(1) != 1:
        raise ValueError("y must be [m, 2n] with unit column stride")
    m, n = y.shape[0], y.shape[1] // 2
    if out is None:
        out = _given(_empty((m, n), torch.bfloat16, y.device, stream), stream)
    elif (out.shape != (m, n) or out.dtype is not _BF16 or out.device != y.device
          or out.stride(1) != 1):
        raise ValueError(f"out must be bf16 [{m}, {n}] with unit column stride on {y.device}")
    st = lib().nvfp4_silu_mul(_ptr(y), m, n, y.stride(0), _ptr(out), out.stride(0),
                              _stream(stream))
    _check(st, "nvfp4_silu_mul")
    return out


def _heads(q, k, v, decay, beta, state, out, stream):
    """Checked arguments shared by linear_attention and its step: (h_k, h_v,
    d_k, d_v, row pitches of q, k, v and out, out). One condition per tensor, not
    a loop over them: a call on one token waits for the host."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("q must be a CUDA tensor")
    if dev != torch.cuda.current_device():
        raise ValueError(f"q is on cuda:{dev}, the current device is {torch.cuda.current_device()}")
    qs, vs = q.shape, v.shape
    if (len(qs) != 3 or len(vs) != 3 or k.shape != qs or vs[0] != qs[0]
            or not (q.dtype is k.dtype is v.dtype is _BF16)
            or k.get_device() != dev or v.get_device() != dev):
        raise ValueError(f"q and k must be [rows, h_k, d_k], v [rows, h_v, d_v], all {_BF16} on "
                         f"cuda:{dev}")
    rows, hk, dk = qs
    _, hv, dv = vs
    if out is None:
        out = _given(_empty(vs, _BF16, q.device, stream), stream)
    elif out.shape != vs or out.dtype is not _BF16 or out.get_device() != dev:
        raise ValueError(f"out must be {_BF16} {list(vs)} on cuda:{dev}")
    gates = (rows, hv)
    if (decay.shape != gates or decay.dtype is not _FP32 or decay.get_device() != dev
            or not decay.is_contiguous()):
        raise ValueError(f"decay must be contiguous {_FP32} {list(gates)} on cuda:{dev}")
    if beta is not None and (beta.shape != gates or beta.dtype is not _FP32
                             or beta.get_device() != dev or not beta.is_contiguous()):
        raise ValueError(f"beta must be contiguous {_FP32} {list(gates)} on cuda:{dev}")
    if state is not None and (state.shape[1:] != (hv, dk, dv) or state.dtype is not _FP32
                              or state.get_device() != dev or not state.is_contiguous()):
        raise ValueError(f"state must be contiguous {_FP32} [slots] + {[hv, dk, dv]} on cuda:{dev}")
    lq, hq, eq = q.stride()
    lk, hk_, ek = k.stride()
    lv, hv_, ev = v.stride()
    lo, ho, eo = out.stride()
    if ((dk > 1 and (eq != 1 or ek != 1)) or (hk > 1 and (hq != dk or hk_ != dk))
            or (dv > 1 and (ev != 1 or eo != 1)) or (hv > 1 and (hv_ != dv or ho != dv))):
        raise ValueError("the heads of a row of q, k, v and out must be contiguous")
    if rows > 1:
        return hk, hv, dk, dv, (lq, lk, lv, lo), out
    ldk, ldv = -(-hk * dk // 8) * 8, -(-hv * dv // 8) * 8  # a single row's pitch is free
    return hk, hv, dk, dv, (ldk, ldk, ldv, ldv), out


def _int32(t: torch.Tensor | None, name: str, n: int, device) -> None:
    if t is not None:
        if (t.dtype is not torch.int32 or t.shape != (n,) or not t.is_contiguous()
                or t.device != device):
            raise ValueError(f"{name} must be a contiguous {torch.int32} vector of {n} on {device}")


def linear_attention_workspace_bytes(total: int, n_seq: int, h_k: int, h_v: int, d_k: int) -> int:
    return int(lib().nvfp4_linear_attention_workspace_bytes(total, n_seq, h_k, h_v, d_k))


def linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor,
                     beta: torch.Tensor | None = None, *, cu_seqlens: torch.Tensor | None = None,
                     state: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                     resume: torch.Tensor | None = None, scale: float | None = None,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """nvfp4_linear_attention: gated linear attention over packed prompts; with
    ``beta`` the gated delta rule. q, k bf16 [total, h_k, d_k], v bf16 [total,
    h_v, d_v] (views of a fused projection are fine), decay (log) and beta FP32
    [total, h_v]; ``cu_seqlens`` int32 [n_seq + 1] (None: one sequence); final
    states go to ``state`` FP32 [slots, h_v, d_k, d_v] at ``slots`` (int32
    [n_seq], None: in order), and come from there where ``resume`` (int32
    [n_seq]) is nonzero. ``scale`` defaults to d_k ** -0.5. The workspace is
    allocated here when None."""
    return _prompts("nvfp4_linear_attention", (), q, k, v, decay, beta, cu_seqlens, state, slots,
                    resume, scale, out, workspace, stream)


def _prompts(call, more, q, k, v, decay, beta, cu_seqlens, state, slots, resume, scale, out,
             workspace, stream):
    """linear_attention, or its self-test: ``more`` are its further arguments."""
    hk, hv, dk, dv, (ldq, ldk, ldv, ldo), out = _heads(q, k, v, decay, beta, state, out, stream)
    total = q.shape[0]
    n_seq = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    _int32(cu_seqlens, "cu_seqlens", n_seq + 1, q.device)
    _int32(slots, "slots", n_seq, q.device)
    _int32(resume, "resume", n_seq, q.device)
    if workspace is None:
        need = linear_attention_workspace_bytes(total, n_seq, hk, hv, dk)
        workspace = _empty(need, torch.uint8, q.device, stream)
    st = getattr(lib(), call)(
        _ptr(q), ldq, _ptr(k), ldk, _ptr(v), ldv, _ptr(decay), _ptr(beta),
        dk ** -0.5 if scale is None else scale, total, hk, hv, dk, dv, n_seq, _ptr(cu_seqlens),
        _ptr(state), 0 if state is None else state.shape[0], _ptr(slots), _ptr(resume), _ptr(out),
        ldo, *_scratch(workspace, q.get_device()), *more, _stream(stream))
    _check(st, call)
    return out


def linear_attention_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor,
                          beta: torch.Tensor | None = None, *, state: torch.Tensor,
                          slots: torch.Tensor | None = None, scale: float | None = None,
                          out: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """nvfp4_linear_attention_step: one token per row, states updated in place.
    Shapes as linear_attention with rows = batch; ``slots`` int32 [batch] (None:
    row i uses slot i), a slot outside the pool marks a padding row."""
    hk, hv, dk, dv, (ldq, ldk, ldv, ldo), out = _heads(q, k, v, decay, beta, state, out, stream)
    batch = q.shape[0]
    _int32(slots, "slots", batch, q.device)
    st = lib().nvfp4_linear_attention_step(
        _ptr(q), ldq, _ptr(k), ldk, _ptr(v), ldv, _ptr(decay), _ptr(beta),
        dk ** -0.5 if scale is None else scale, batch, hk, hv, dk, dv, _ptr(state),
        state.shape[0], _ptr(slots), _ptr(out), ldo, _stream(stream))
    _check(st, "nvfp4_linear_attention_step")
    return out


def read_fault(stream: torch.cuda.Stream | None = None) -> int:
    """Synchronise, return and clear the kernels' timeout fault word."""
    v = ctypes.c_uint32(0)
    st = lib().nvfp4_read_fault(_stream(stream), ctypes.byref(v))
    if st not in (NVFP4_OK, 5):
        raise NVFP4Error("nvfp4_read_fault", st)
    return int(v.value)


def selftest_wait_timeout(limit_ns: int = 1_000_000,
                          stream: torch.cuda.Stream | None = None) -> None:
    """nvfp4_selftest_wait_timeout: make one bounded wait give up on the GPU
    (read_fault() then returns 256)."""
    _check(lib().nvfp4_selftest_wait_timeout(limit_ns, _stream(stream)),
           "nvfp4_selftest_wait_timeout")


def selftest_gemm_stall(a: NVFP4Tensor, b: NVFP4Tensor, limit_ns: int = 1_000_000,
                        workspace: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None) -> None:
    """nvfp4_selftest_gemm_stall: run the GEMM kernel for these operands
    with its first ring stage never filled and every wait limited to
    ``limit_ns``; the kernel gives up and returns (read_fault() then returns
    the role bits that timed out)."""
    m, n, k = a.rows, b.rows, a.k
    y = _empty((m, n), torch.bfloat16, a.codes.device, stream)
    dev = a.codes.get_device()
    _check(lib().nvfp4_selftest_gemm_stall(*_operand(a, "a", dev), *_operand(b, "b", dev),
                                           _ptr(y), m, n, k, limit_ns, *_scratch(workspace, dev),
                                           _stream(stream)),
           "nvfp4_selftest_gemm_stall")


def selftest_linear_attention_stall(
        q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor,
        beta: torch.Tensor | None = None, *, kernel: int, cta: int = 0, limit_ns: int = 1_000_000,
        cu_seqlens: torch.Tensor | None = None, state: torch.Tensor | None = None,
        slots: torch.Tensor | None = None, resume: torch.Tensor | None = None,
        scale: float | None = None, out: torch.Tensor | None = None,
        workspace: torch.Tensor | None = None,
        stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """nvfp4_selftest_linear_attention_stall: linear_attention with CTA ``cta`` of
    its first (``kernel`` 0) or second (1) kernel never issuing its first product
    or load, and every wait limited to ``limit_ns``: it gives up and returns, its
    head's state stays as it was (read_fault() then returns 512, or 1024 and / or
    2048)."""
    return _prompts("nvfp4_selftest_linear_attention_stall", (kernel, cta, limit_ns), q, k, v,
                    decay, beta, cu_seqlens, state, slots, resume, scale, out, workspace, stream)


def linear_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(lib().nvfp4_linear_workspace_bytes(m, n, k))


def linear_workspace(m: int, n: int, k: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for linear() at these sizes (keep it: calls
    leave the bytes that must start at zero zeroed again)."""
    return torch.zeros(linear_workspace_bytes(m, n, k), dtype=torch.uint8, device=device)


def linear(x: torch.Tensor, w: NVFP4Tensor, out: torch.Tensor | None = None,
           out_dtype: torch.dtype = torch.bfloat16, global_scale: torch.Tensor | None = None,
           workspace: torch.Tensor | None = None,
           stream: torch.cuda.Stream | None = None, bias: torch.Tensor | None = None,
           activation: str = "none", residual: torch.Tensor | None = None) -> torch.Tensor:
    """nvfp4_linear, the W4A4 linear layer in one call: quantize x (dynamic
    global, or the static ``global_scale``) and multiply with the NVFP4
    weights ``w`` [n, k]; the GEMM's launch overlaps the quantization.
    ``workspace`` from linear_workspace() (allocated here when None).
    With ``bias`` (bf16 [n]), ``activation`` (a key of ACTIVATIONS) or
    ``residual`` (bf16 [m, n], may be ``out``): nvfp4_linear_epilogue,
    Y = act(product + bias) + residual in FP32, rounded once."""
    _require_cuda(x, "x", torch.bfloat16)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride along k")
    m, k = x.shape
    if k != w.k:
        raise ValueError("k mismatch")
    n = w.rows
    dev = x.get_device()
    out, y = _product(out, out_dtype, m, n, dev, x, stream)
    if workspace is None:
        with _on(stream):
            workspace = linear_workspace(m, n, k, x.device)
    args = (_ptr(x), m, k, x.stride(0), _global(global_scale, "global_scale", dev),
            *_operand(w, "w", dev), n)
    ws, ws_bytes = _scratch(workspace, dev)
    if bias is not None or residual is not None or activation != "none":
        st = lib().nvfp4_linear_epilogue(
            *args, *_epilogue(bias, activation, residual, m, n, x.device), *y, ws, ws_bytes,
            _stream(stream))
        _check(st, "nvfp4_linear_epilogue")
        return out
    st = lib().nvfp4_linear(*args, *y, ws, ws_bytes, _stream(stream))
    _check(st, "nvfp4_linear")
    return out
