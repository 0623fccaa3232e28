"""Thin ctypes binding over libvqmi.so (include/vq.h): argument marshalling only.

Every step of the computation runs in the library's HIP kernels; PyTorch only
provides device memory and the current stream.  There is no fallback: if the
library is missing this module raises on import.
"""

from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libvqmi.so")

VQ_OK, VQ_ERR_NULL, VQ_ERR_GEOMETRY, VQ_ERR_SHAPE, VQ_ERR_ALIGN, VQ_ERR_WORKSPACE, VQ_ERR_HIP = range(7)
STATUS_NAMES = ["VQ_OK", "VQ_ERR_NULL", "VQ_ERR_GEOMETRY", "VQ_ERR_SHAPE", "VQ_ERR_ALIGN",
                "VQ_ERR_WORKSPACE", "VQ_ERR_HIP"]


class VQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES[status] if 0 <= status < 7 else status}: {message}")
        self.status = status
        self.message = message


VQ_DTYPE_F32, VQ_DTYPE_F16, VQ_DTYPE_BF16, VQ_DTYPE_E4M3 = 0, 1, 2, 3
VQ_EPILOGUE_NONE, VQ_EPILOGUE_SWIGLU, VQ_EPILOGUE_COMBINE = 0, 1, 2
EPILOGUES = {None: VQ_EPILOGUE_NONE, "none": VQ_EPILOGUE_NONE, "swiglu": VQ_EPILOGUE_SWIGLU,
             "combine": VQ_EPILOGUE_COMBINE}


class CIo(ctypes.Structure):
    """Mirror of `vq_io`."""
    _fields_ = [
        ("x_dtype", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32),
        ("epilogue", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("route_weights", ctypes.c_void_p),
    ]


class CRouter(ctypes.Structure):
    """Mirror of `vq_router`."""
    _fields_ = [
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("logits_dtype", ctypes.c_int32),
        ("groups", ctypes.c_int32),
        ("top_groups", ctypes.c_int32),
        ("group_score", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("reserved", ctypes.c_int32),
        ("bias", ctypes.c_void_p),
    ]


class CFP8Tensor(ctypes.Structure):
    """Mirror of `vq_fp8_tensor`."""
    _fields_ = [
        ("values", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("rows", ctypes.c_int32),
        ("cols", ctypes.c_int32),
        ("value_bytes", ctypes.c_int64),
        ("scale_elems", ctypes.c_int64),
    ]


class CNormSpec(ctypes.Structure):
    """Mirror of `vq_norm_spec`."""
    _fields_ = [
        ("cols", ctypes.c_int32),
        ("block_dtype", ctypes.c_int32),
        ("residual_dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("h_dtype", ctypes.c_int32),
        ("gate", ctypes.c_int32),
        ("gate_act", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("alpha", ctypes.c_float),
        ("beta", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
        ("post_weight", ctypes.c_void_p),
        ("pre_weight", ctypes.c_void_p),
        ("gate_values", ctypes.c_void_p),
    ]


class CTensor(ctypes.Structure):
    """Mirror of `vq_tensor`."""
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("codebook", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("rows", ctypes.c_int32),
        ("cols", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("log2_k", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("codebook_per_expert", ctypes.c_int32),
        ("codebook_elems", ctypes.c_int64),
        ("code_words", ctypes.c_int64),
        ("scale_elems", ctypes.c_int64),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m vq_dequant_matmul_gemv_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    i32 = ctypes.c_int32
    T = ctypes.POINTER(CTensor)
    IO = ctypes.POINTER(CIo)
    sig = {
        "vq_gemv_ex": (i32, [T, IO, P, i32, P, P]),
        "vq_gemm_ex": (i32, [T, IO, P, i32, P, P]),
        "vq_moe_gemv_ex": (i32, [T, IO, P, i32, P, i32, i32, P, P]),
        "vq_moe_gemm_ex": (i32, [T, IO, P, i32, P, i32, i32, P, P, ctypes.c_size_t, P]),
        "vq_words_per_row": (i32, [i32, i32, i32]),
        "vq_dequant": (i32, [T, i32, P, P]),
        "vq_gemv": (i32, [T, P, i32, P, P]),
        "vq_gemm": (i32, [T, P, i32, P, P]),
        "vq_moe_gemv": (i32, [T, P, i32, P, i32, i32, P, P]),
        "vq_moe_workspace_bytes": (ctypes.c_size_t, [i32, i32, i32]),
        "vq_moe_gemm": (i32, [T, P, i32, P, i32, i32, P, P, ctypes.c_size_t, P]),
        "vq_moe_gemm_no_alloc": (i32, [T, P, i32, P, i32, i32, P, P]),
        "vq_encode_workspace_bytes": (ctypes.c_size_t, [i32, i32, i32, i32, i32]),
        "vq_encode": (i32, [P, i32, i32, i32, i32, i32, P, i32, P, i32, P, P, P, P, P, ctypes.c_size_t, P]),
        "vq_moe_route": (i32, [P, P, i32, P, P, P]),
        "vq_fp8_quant": (i32, [P, i32, i32, i32, P, P, P]),
        "vq_fp8_workspace_bytes": (ctypes.c_size_t, [i32, i32, i32]),
        "vq_fp8_gemm": (i32, [P, P, P, P, i32, P, P, ctypes.c_size_t, P]),
        "vq_fp8_gemm_fast": (i32, [P, P, P, P, i32, P, P, ctypes.c_size_t, P]),
        "vq_norm": (i32, [P, P, P, i32, P, P, P, P]),
        "vq_last_error": (ctypes.c_char_p, []),
        "vq_status_name": (ctypes.c_char_p, [i32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


LIB = _load()

EXPORTED = ("vq_words_per_row", "vq_dequant", "vq_gemv", "vq_gemm", "vq_moe_gemv", "vq_gemv_ex",
            "vq_gemm_ex", "vq_moe_gemv_ex", "vq_moe_gemm_ex",
            "vq_moe_workspace_bytes", "vq_moe_gemm", "vq_moe_gemm_no_alloc", "vq_encode_workspace_bytes",
            "vq_encode", "vq_moe_route", "vq_fp8_quant", "vq_fp8_workspace_bytes", "vq_fp8_gemm",
            "vq_fp8_gemm_fast", "vq_norm",
            "vq_last_error", "vq_status_name")


def check(status: int) -> None:
    if status != VQ_OK:
        raise VQError(status, LIB.vq_last_error().decode())


def words_per_row(cols: int, d: int, log2_k: int) -> int:
    return LIB.vq_words_per_row(cols, d, log2_k)


def workspace_bytes(T: int, top_k: int, num_experts: int) -> int:
    return LIB.vq_moe_workspace_bytes(T, top_k, num_experts)


# --------------------------------------------------------------------------
# torch-facing wrappers
# --------------------------------------------------------------------------

_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _dev_check(*ts, device=None):
    """Every tensor on the GPU (on `device` when given), contiguous."""
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must live on the GPU")
        if device is not None and t.device != device:
            raise ValueError(f"tensor on {t.device}, expected {device} (the weights' device)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _check_out(y, dtype, shape, name="y"):
    torch = _torch()
    if y.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {y.dtype}")
    if tuple(y.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(y.shape)}")
    del torch


@dataclass
class VQTensor:
    """Device-resident VQ tensor (see `vq_tensor` in include/vq.h).

    codes    int32/uint32 [E][rows][Wr] (or [rows][Wr]) packed code words
    codebook fp16 [K][d] or [E][K][d]
    scales   fp16 [E][rows][cols/group] (or [rows][cols/group])
    """
    codes: object
    codebook: object
    scales: object
    rows: int
    cols: int
    d: int
    log2_k: int
    group: int
    num_experts: int = 1
    codebook_per_expert: bool = False

    @property
    def device(self):
        return self.codes.device

    def cstruct(self) -> CTensor:
        """The C descriptor; buffer lengths travel with it so the library
        refuses codes, scales or a codebook of the wrong size."""
        torch = _torch()
        _dev_check(self.codes, self.codebook, self.scales, device=self.codes.device)
        if self.codebook.dtype != torch.float16 or self.scales.dtype != torch.float16:
            raise ValueError("codebook and scales must be fp16")
        if self.codes.element_size() * self.codes.numel() % 4:
            raise ValueError("codes must hold whole uint32 words")
        return CTensor(self.codes.data_ptr(), self.codebook.data_ptr(), self.scales.data_ptr(),
                       self.rows, self.cols, self.d, self.log2_k, self.group, self.num_experts,
                       int(self.codebook_per_expert), self.codebook.numel(),
                       self.codes.numel() * self.codes.element_size() // 4, self.scales.numel())

    @classmethod
    def from_host(cls, arrays: dict, spec, device="cuda", codebook_per_expert=False):
        """Copy numpy arrays (codes/codebook/scales as produced by synth.tensor)
        to the device."""
        import numpy as np
        torch = _torch()
        codes = torch.from_numpy(np.ascontiguousarray(arrays["codes"]).view(np.int32)).to(device)
        cb = torch.from_numpy(np.ascontiguousarray(arrays["codebook"])).to(device)
        sc = torch.from_numpy(np.ascontiguousarray(arrays["scales"])).to(device)
        return cls(codes, cb, sc, spec.rows, spec.cols, spec.d, spec.log2_k, spec.group,
                   spec.experts, codebook_per_expert)


def dequant(w: VQTensor, expert: int = 0, out=None, stream=None):
    torch = _torch()
    if out is None:
        out = torch.empty((w.rows, w.cols), dtype=torch.float16, device=w.codes.device)
    _check_out(out, torch.float16, (w.rows, w.cols), "out")
    _dev_check(out, device=w.device)
    cs = w.cstruct()
    check(LIB.vq_dequant(ctypes.byref(cs), expert, _ptr(out), _stream(stream)))
    return out


_DTYPE_CODES = {}


def _dtype_code(dt):
    if not _DTYPE_CODES:
        torch = _torch()
        _DTYPE_CODES.update({torch.float32: VQ_DTYPE_F32, torch.float16: VQ_DTYPE_F16,
                             torch.bfloat16: VQ_DTYPE_BF16})
    if dt not in _DTYPE_CODES:
        raise ValueError(f"unsupported dtype {dt}")
    return _DTYPE_CODES[dt]


def _io(x, y_dtype, epilogue, route_weights):
    """The vq_io of a call, or None for the plain call (fp16 x, fp32 y)."""
    torch = _torch()
    if epilogue not in EPILOGUES:
        raise ValueError(f"epilogue must be one of {sorted(k for k in EPILOGUES if k)}")
    epi = EPILOGUES[epilogue]
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("x must be fp16 or bf16")
    if x.dtype == torch.float16 and y_dtype == torch.float32 and epi == VQ_EPILOGUE_NONE:
        return None
    rw = 0
    if epi == VQ_EPILOGUE_COMBINE:
        if route_weights is None or route_weights.dtype != torch.float32:
            raise ValueError("the combine needs fp32 route_weights [T][top_k]")
        rw = route_weights.data_ptr()
    return CIo(_dtype_code(x.dtype), _dtype_code(y_dtype), epi, 0, rw)


def _dense(fn, fn_ex, w: VQTensor, x, y, stream, y_dtype=None, epilogue=None):
    torch = _torch()
    if x.dtype not in (torch.float16, torch.bfloat16) or x.dim() != 2 or x.shape[1] != w.cols:
        raise ValueError("x must be fp16 or bf16 [T][cols]")
    T = x.shape[0]
    y_dtype = y.dtype if (y is not None and y_dtype is None) else (y_dtype or torch.float32)
    ycols = w.rows // 2 if epilogue == "swiglu" else w.rows
    if epilogue == "combine":
        raise ValueError("the combine applies to routed calls only")
    # a stack of experts (vq_gemm only): y[t][e] = W_e x[t]
    yshape = (T, ycols) if w.num_experts == 1 else (T, w.num_experts, ycols)
    if y is None:
        y = torch.empty(yshape, dtype=y_dtype, device=x.device)
    _check_out(y, y_dtype, yshape)
    _dev_check(x, y, device=w.device)
    cs = w.cstruct()
    io = _io(x, y_dtype, epilogue, None)
    if io is None:
        check(fn(ctypes.byref(cs), _ptr(x), T, _ptr(y), _stream(stream)))
    else:
        check(fn_ex(ctypes.byref(cs), ctypes.byref(io), _ptr(x), T, _ptr(y), _stream(stream)))
    return y


def gemv(w: VQTensor, x, y=None, stream=None, y_dtype=None, epilogue=None):
    """y = x W^T through vq_gemv (vq_gemv_ex for bf16 x, a non-fp32 y or an
    epilogue: "swiglu" on interleaved gate/up rows gives silu(gate) * up).
    On a stack of E experts, y is [T][E][rows]: every expert times the same x."""
    return _dense(LIB.vq_gemv, LIB.vq_gemv_ex, w, x, y, stream, y_dtype, epilogue)


def gemm(w: VQTensor, x, y=None, stream=None, y_dtype=None, epilogue=None):
    """y = x W^T through vq_gemm (MFMA); options as for gemv.  On a stack of
    E experts, y is [T][E][rows]: every expert times the same x."""
    return _dense(LIB.vq_gemm, LIB.vq_gemm_ex, w, x, y, stream, y_dtype, epilogue)


def _moe_prep(w, x, ids, x_per_slot, y, y_dtype=None, epilogue=None):
    torch = _torch()
    T, top_k = ids.shape
    if ids.dtype != torch.int32:
        raise ValueError("expert ids must be int32 [T][top_k]")
    want = (T, top_k, w.cols) if x_per_slot else (T, w.cols)
    if x.dtype not in (torch.float16, torch.bfloat16) or tuple(x.shape) != want:
        raise ValueError(f"x must be fp16 or bf16 {want}")
    y_dtype = y.dtype if (y is not None and y_dtype is None) else (y_dtype or torch.float32)
    if epilogue == "combine":
        yshape = (T, w.rows)
    else:
        yshape = (T, top_k, w.rows // 2 if epilogue == "swiglu" else w.rows)
    if y is None:
        y = torch.empty(yshape, dtype=y_dtype, device=x.device)
    _check_out(y, y_dtype, yshape)
    _dev_check(x, ids, y, device=w.device)
    return T, top_k, y, y_dtype


def moe_gemv(w: VQTensor, x, ids, x_per_slot=False, y=None, stream=None, y_dtype=None, epilogue=None,
             route_weights=None):
    """Routed experts, decode-shaped (vq_moe_gemv / vq_moe_gemv_ex).  epilogue
    "combine" with fp32 route_weights [T][top_k] gives y [T][rows] = the
    router-weighted sum over each token's slots."""
    T, top_k, y, y_dtype = _moe_prep(w, x, ids, x_per_slot, y, y_dtype, epilogue)
    if route_weights is not None:
        _dev_check(route_weights, device=w.device)
    cs = w.cstruct()
    io = _io(x, y_dtype, epilogue, route_weights)
    if io is None:
        check(LIB.vq_moe_gemv(ctypes.byref(cs), _ptr(x), int(bool(x_per_slot)), _ptr(ids), T, top_k,
                              _ptr(y), _stream(stream)))
    else:
        check(LIB.vq_moe_gemv_ex(ctypes.byref(cs), ctypes.byref(io), _ptr(x), int(bool(x_per_slot)), _ptr(ids),
                                 T, top_k, _ptr(y), _stream(stream)))
    return y


def moe_gemm(w: VQTensor, x, ids, x_per_slot=False, y=None, workspace=None, stream=None, y_dtype=None,
             epilogue=None, route_weights=None):
    """Routed experts, prefill-shaped (vq_moe_gemm / vq_moe_gemm_ex); options
    as for moe_gemv."""
    torch = _torch()
    T, top_k, y, y_dtype = _moe_prep(w, x, ids, x_per_slot, y, y_dtype, epilogue)
    if route_weights is not None:
        _dev_check(route_weights, device=w.device)
    need = workspace_bytes(T, top_k, w.num_experts)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    _dev_check(workspace, device=w.device)
    cs = w.cstruct()
    io = _io(x, y_dtype, epilogue, route_weights)
    if io is None:
        check(LIB.vq_moe_gemm(ctypes.byref(cs), _ptr(x), int(bool(x_per_slot)), _ptr(ids), T, top_k,
                              _ptr(y), _ptr(workspace), workspace.numel(), _stream(stream)))
    else:
        check(LIB.vq_moe_gemm_ex(ctypes.byref(cs), ctypes.byref(io), _ptr(x), int(bool(x_per_slot)), _ptr(ids),
                                 T, top_k, _ptr(y), _ptr(workspace), workspace.numel(), _stream(stream)))
    return y


def moe_gemm_no_alloc(w: VQTensor, x, ids, x_per_slot=False, y=None, stream=None):
    """vq_moe_gemm_no_alloc: vq_moe_gemm with the library's static scratch
    instead of a workspace (allocates nothing when y is given)."""
    T, top_k, y, _ = _moe_prep(w, x, ids, x_per_slot, y)
    cs = w.cstruct()
    check(LIB.vq_moe_gemm_no_alloc(ctypes.byref(cs), _ptr(x), int(bool(x_per_slot)), _ptr(ids), T, top_k,
                                   _ptr(y), _stream(stream)))
    return y


def encode(w, d: int, log2_k: int, group: int, sample_idx, uniforms, iters: int, workspace=None, stream=None):
    """vq_encode: fit a VQ tensor to fp32 weights w [rows][cols] on the GPU.
    sample_idx: int32 [n_sample] subvector indices for k-means++; uniforms:
    fp64 [K] draws.  Returns (VQTensor, relerr as a 0-d fp64 device tensor)."""
    torch = _torch()
    if w.dtype != torch.float32 or w.dim() != 2:
        raise ValueError("w must be fp32 [rows][cols]")
    if sample_idx.dtype != torch.int32 or uniforms.dtype != torch.float64:
        raise ValueError("sample_idx must be int32 and uniforms fp64")
    rows, cols = w.shape
    K = 1 << log2_k
    if uniforms.numel() != K:
        raise ValueError(f"uniforms must hold K = {K} values")
    dev = w.device
    _dev_check(w, sample_idx, uniforms, device=dev)
    wr = words_per_row(cols, d, log2_k)
    if wr < 0:
        raise ValueError("unsupported geometry")
    codes = torch.empty((rows, wr), dtype=torch.int32, device=dev)
    codebook = torch.empty((K, d), dtype=torch.float16, device=dev)
    scales = torch.empty((rows, cols // group), dtype=torch.float16, device=dev)
    relerr = torch.empty((), dtype=torch.float64, device=dev)
    need = LIB.vq_encode_workspace_bytes(rows, cols, d, log2_k, sample_idx.numel())
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _dev_check(workspace, device=dev)
    check(LIB.vq_encode(_ptr(w), rows, cols, d, log2_k, group, _ptr(sample_idx), sample_idx.numel(), _ptr(uniforms),
                        iters, _ptr(codes), _ptr(codebook), _ptr(scales), _ptr(relerr), _ptr(workspace),
                        workspace.numel(), _stream(stream)))
    return VQTensor(codes, codebook, scales, rows, cols, d, log2_k, group), relerr


# --------------------------------------------------------------------------
# routing to experts
# --------------------------------------------------------------------------

VQ_SCORE_SOFTMAX, VQ_SCORE_SIGMOID = 0, 1
VQ_GROUP_MAX, VQ_GROUP_TOP2 = 0, 1
SCORES = {"softmax": VQ_SCORE_SOFTMAX, "sigmoid": VQ_SCORE_SIGMOID}
GROUP_SCORES = {"max": VQ_GROUP_MAX, "top2": VQ_GROUP_TOP2}


# Descriptors as bytes, in the layouts of CRouter, CFP8Tensor, CIo and CNormSpec
# (packing takes a third of a ctypes structure's time).
_pack_router = struct.Struct("<8ifiQ").pack
_pack_fp8 = struct.Struct("<QQiiqq").pack
_pack_io = struct.Struct("<4iQ").pack
_pack_norm = struct.Struct("<8i4f3Q").pack


def _placed(t, index):
    """The tensor is contiguous on GPU `index`."""
    if t.get_device() != index:
        raise ValueError(f"tensor on {t.device}, expected cuda:{index} (the GPU of the other tensors)")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")


def _gpu(t):
    """Index of the GPU the tensor is on; it is contiguous there."""
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return index


def _address(t):
    return None if t is None else t.data_ptr()


def _rows(T, cols, dtype, device):
    """An uninitialised [T][cols] (empty_strided takes a quarter less time than
    empty, which parses its sizes)."""
    return _TORCH.empty_strided((T, cols), (cols, 1), dtype=dtype, device=device)


def _elsewhere(device, stream):
    """The context a call has to enter first: the given stream's, or that of
    tensors on another GPU than the current one.  None where the current
    device and stream are the ones to use."""
    torch = _TORCH
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream on {stream.device}, tensors on {device}")
        return torch.cuda.stream(stream)
    return torch.cuda.device(device) if torch._C._cuda_getDevice() != device.index else None


def _raw_stream(index) -> int:
    """Handle of the GPU's current stream."""
    return _TORCH._C._cuda_getCurrentRawStream(index)


@dataclass
class Router:
    """How a router's logits become expert ids and weights (see `vq_router` in
    include/vq.h): score "softmax" or "sigmoid", bias fp32 [num_experts] or
    None, group_score "max" or "top2"."""
    num_experts: int
    top_k: int
    score: str = "softmax"
    bias: object = None
    groups: int = 1
    top_groups: int = 1
    group_score: str = "max"
    renormalize: bool = True
    scale: float = 1.0


def moe_route(router: Router, logits, ids=None, weights=None, stream=None):
    """Expert ids int32 [T][top_k] and route weights fp32 [T][top_k] for
    moe_gemv / moe_gemm, from logits [T][num_experts] (fp32, fp16 or bf16)."""
    torch = _torch()
    r = router
    if r.score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    if r.group_score not in GROUP_SCORES:
        raise ValueError(f"group_score must be one of {sorted(GROUP_SCORES)}")
    shape = logits.shape
    if len(shape) != 2 or shape[1] != r.num_experts:
        raise ValueError(f"logits must be [T][{r.num_experts}]")
    T, k = shape[0], r.top_k
    gpu = _gpu(logits)
    dev = logits.device
    bias = 0
    if r.bias is not None:
        if r.bias.dtype != torch.float32 or r.bias.shape != (r.num_experts,):
            raise ValueError(f"bias must be fp32 [{r.num_experts}]")
        _placed(r.bias, gpu)
        bias = r.bias.data_ptr()
    if ids is not None:
        _check_out(ids, torch.int32, (T, k), "ids")
        _placed(ids, gpu)
    if weights is not None:
        _check_out(weights, torch.float32, (T, k), "weights")
        _placed(weights, gpu)
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return moe_route(router, logits, ids, weights)
    slots = k if 0 <= k <= 64 else 0  # the library refuses any other k: nothing is allocated for it
    if ids is None:
        ids = _rows(T, slots, torch.int32, dev)
    if weights is None:
        weights = _rows(T, slots, torch.float32, dev)
    cr = _pack_router(r.num_experts, k, SCORES[r.score], _dtype_code(logits.dtype), r.groups, r.top_groups,
                      GROUP_SCORES[r.group_score], bool(r.renormalize), r.scale, 0, bias)
    check(LIB.vq_moe_route(cr, logits.data_ptr(), T, ids.data_ptr(), weights.data_ptr(),
                           _raw_stream(gpu)))
    return ids, weights


# --------------------------------------------------------------------------
# e4m3 tensors with a scale for each block of 128
# --------------------------------------------------------------------------

def _blocks(n: int) -> int:
    return -(-n // 128)


@dataclass
class FP8Tensor:
    """Device-resident e4m3 weight (see `vq_fp8_tensor` in include/vq.h).

    values  float8_e4m3fn (or uint8 codes) [rows][cols]
    scales  fp32 [ceil(rows/128)][ceil(cols/128)]
    """
    values: object
    scales: object

    @property
    def device(self):
        return self.values.device

    def checked(self):
        """(rows, cols, index of the GPU both tensors are on), after the checks
        of their types, shapes and places."""
        torch = _torch()
        v, s = self.values, self.scales
        if v.dtype not in (torch.float8_e4m3fn, torch.uint8) or v.dim() != 2:
            raise ValueError("w.values must be float8_e4m3fn (or uint8 codes) [rows][cols]")
        rows, cols = v.shape
        if s.dtype != torch.float32 or s.shape != (_blocks(rows), _blocks(cols)):
            raise ValueError(f"w.scales must be fp32 {(_blocks(rows), _blocks(cols))} (one value for each 128 x 128 "
                             f"block), got {s.dtype} {tuple(s.shape)}")
        gpu = _gpu(v)
        _placed(s, gpu)
        return rows, cols, gpu

    def cstruct(self) -> CFP8Tensor:
        rows, cols, _ = self.checked()
        return CFP8Tensor(self.values.data_ptr(), self.scales.data_ptr(), rows, cols, rows * cols, self.scales.numel())


def fp8_quant(x, q=None, scales=None, stream=None):
    """e4m3 values [T][cols] and fp32 scales [T][ceil(cols/128)] of fp16 or
    bf16 activations x [T][cols] (vq_fp8_quant)."""
    torch = _torch()
    if x.dtype not in (torch.float16, torch.bfloat16) or x.dim() != 2:
        raise ValueError("x must be fp16 or bf16 [T][cols]")
    T, cols = x.shape
    gpu = _gpu(x)
    dev = x.device
    sshape = (T, _blocks(cols))
    if q is not None:
        _check_out(q, torch.float8_e4m3fn, (T, cols), "q")
        _placed(q, gpu)
    if scales is not None:
        _check_out(scales, torch.float32, sshape, "scales")
        _placed(scales, gpu)
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return fp8_quant(x, q, scales)
    if q is None:
        q = _rows(T, cols, torch.float8_e4m3fn, dev)
    if scales is None:
        scales = _rows(*sshape, torch.float32, dev)
    check(LIB.vq_fp8_quant(x.data_ptr(), _dtype_code(x.dtype), T, cols, q.data_ptr(), scales.data_ptr(),
                           _raw_stream(gpu)))
    return q, scales


def fp8_gemm(w: FP8Tensor, x, x_scales, y=None, workspace=None, stream=None, y_dtype=None, epilogue=None,
             fast=False):
    """y = x W^T of e4m3 activations (values [T][cols], scales
    [T][ceil(cols/128)]) through vq_fp8_gemm, decode and prefill alike;
    epilogue "swiglu" on interleaved gate/up rows gives silu(gate) * up.
    fast, for a 16-bit y: vq_fp8_gemm_fast, whose products of large batches are
    cut 13 bits below the largest of eight (see include/vq.h)."""
    torch = _torch()
    rows, cols, gpu = w.checked()
    v, ws = w.values, w.scales
    if x.dtype not in (torch.float8_e4m3fn, torch.uint8) or x.dim() != 2 or x.shape[1] != cols:
        raise ValueError(f"x must be float8_e4m3fn (or uint8 codes) [T][{cols}]")
    T = x.shape[0]
    if x_scales.dtype != torch.float32 or x_scales.shape != (T, _blocks(cols)):
        raise ValueError(f"x_scales must be fp32 {(T, _blocks(cols))}")
    if epilogue not in EPILOGUES or epilogue == "combine":
        raise ValueError("epilogue must be None or 'swiglu'")
    y_dtype = y.dtype if (y is not None and y_dtype is None) else (y_dtype or torch.float32)
    yshape = (T, rows // 2 if epilogue == "swiglu" else rows)
    dev = v.device
    _placed(x, gpu)
    _placed(x_scales, gpu)
    if y is not None:
        _check_out(y, y_dtype, yshape)
        _placed(y, gpu)
    if workspace is not None:
        _placed(workspace, gpu)
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return fp8_gemm(w, x, x_scales, y, workspace, None, y_dtype, epilogue, fast)
    if y is None:
        y = _rows(*yshape, y_dtype, dev)
    if workspace is None:
        need = LIB.vq_fp8_workspace_bytes(rows, cols, T)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wptr, wbytes = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                        workspace.numel() * workspace.element_size())
    call = LIB.vq_fp8_gemm_fast if fast else LIB.vq_fp8_gemm
    check(call(_pack_fp8(v.data_ptr(), ws.data_ptr(), rows, cols, rows * cols, ws.numel()),
               _pack_io(VQ_DTYPE_E4M3, _dtype_code(y_dtype), EPILOGUES[epilogue], 0, 0), x.data_ptr(),
               x_scales.data_ptr(), T, y.data_ptr(), wptr, wbytes, _raw_stream(gpu)))
    return y


# --------------------------------------------------------------------------
# norms before and after a block
# --------------------------------------------------------------------------

VQ_GATE_NONE, VQ_GATE_CHANNEL, VQ_GATE_TOKEN, VQ_GATE_FULL = range(4)
VQ_ACT_NONE, VQ_ACT_SIGMOID, VQ_ACT_TANH = range(3)
GATE_ACTS = {None: VQ_ACT_NONE, "none": VQ_ACT_NONE, "sigmoid": VQ_ACT_SIGMOID, "tanh": VQ_ACT_TANH}


def norm(block=None, residual=None, *, post_weight=None, pre_weight=None, gate=None, gate_act=None, alpha=1.0,
         beta=1.0, weight_offset=0.0, eps=1e-6, h_dtype=None, residual_out=None, h=None, h_scales=None,
         store_residual=True, stream=None):
    """The norms around a block with its gate and the residual sum (vq_norm):
    u = norm(block) * post_weight (block itself without one), v = beta *
    residual + alpha * act(gate) * u, h = norm(v) * pre_weight.  Returns (v,
    h, h_scales).

    block, residual  [T][cols], fp32, fp16 or bf16, either may be None
    gate             [cols], [T][1] or [T][cols]; gate_act None, "sigmoid" or "tanh"
    weights, gate    of one dtype
    h_dtype          dtype of h (float8_e4m3fn: with h_scales [T][ceil(cols/128)]);
                     None: no h unless pre_weight or h is given (then their dtype)
    residual_out     may be `residual`; v has residual's dtype (block's without one)
    """
    torch = _torch()
    first = block if block is not None else residual
    if first is None:
        raise ValueError("norm needs a block or a residual")
    if first.dim() != 2:
        raise ValueError("block and residual must be [T][cols]")
    shape = T, cols = first.shape
    dev = first.device
    v_dtype = first.dtype if residual is None else residual.dtype
    if h_dtype is None:
        h_dtype = h.dtype if h is not None else pre_weight.dtype if pre_weight is not None else None
    e4m3 = h_dtype == torch.float8_e4m3fn
    if h_dtype is None and not store_residual:
        raise ValueError("norm has nothing to compute: neither v nor h is wanted")
    gpu = _gpu(first)
    if block is not None and residual is not None:
        _placed(residual, gpu)
        if residual.shape != shape:
            raise ValueError("block and residual must have the same shape [T][cols]")
    post = pre = gates = kind = 0
    w_dtype = None
    if post_weight is not None:
        _placed(post_weight, gpu)
        if post_weight.shape != (cols,):
            raise ValueError(f"post_weight must be [{cols}]")
        w_dtype, post = post_weight.dtype, post_weight.data_ptr()
    if pre_weight is not None:
        _placed(pre_weight, gpu)
        if pre_weight.shape != (cols,):
            raise ValueError(f"pre_weight must be [{cols}]")
        if w_dtype is not None and pre_weight.dtype != w_dtype:
            raise ValueError("post_weight, pre_weight and gate must have one dtype")
        w_dtype, pre = pre_weight.dtype, pre_weight.data_ptr()
    if gate is not None:
        _placed(gate, gpu)
        if w_dtype is not None and gate.dtype != w_dtype:
            raise ValueError("post_weight, pre_weight and gate must have one dtype")
        kind = (VQ_GATE_FULL if gate.shape == shape else VQ_GATE_CHANNEL if gate.shape == (cols,) else
                VQ_GATE_TOKEN if gate.shape == (T, 1) else 0)
        if kind == 0:
            raise ValueError(f"gate must be [{cols}], [{T}][1] or [{T}][{cols}]")
        w_dtype, gates = gate.dtype, gate.data_ptr()
    if gate_act not in GATE_ACTS:
        raise ValueError(f"gate_act must be None or one of {sorted(k for k in GATE_ACTS if k)}")
    if residual_out is not None:
        _check_out(residual_out, v_dtype, shape, "residual_out")
        _placed(residual_out, gpu)
    if h is not None:
        _check_out(h, h_dtype, shape, "h")
        _placed(h, gpu)
    if h_scales is not None:
        _check_out(h_scales, torch.float32, (T, _blocks(cols)), "h_scales")
        _placed(h_scales, gpu)
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return norm(block, residual, post_weight=post_weight, pre_weight=pre_weight, gate=gate,
                        gate_act=gate_act, alpha=alpha, beta=beta, weight_offset=weight_offset, eps=eps,
                        h_dtype=h_dtype, residual_out=residual_out, h=h, h_scales=h_scales,
                        store_residual=store_residual)
    if residual_out is None and store_residual:
        residual_out = _rows(T, cols, v_dtype, dev)
    if h is None and h_dtype is not None:
        h = _rows(T, cols, h_dtype, dev)
    if h_scales is None and e4m3:
        h_scales = _rows(T, _blocks(cols), torch.float32, dev)
    spec = _pack_norm(cols, _dtype_code(first.dtype), _dtype_code(v_dtype), _dtype_code(w_dtype or torch.float32),
                      VQ_DTYPE_E4M3 if e4m3 else _dtype_code(h_dtype or torch.float32), kind,
                      GATE_ACTS[gate_act] if kind else VQ_ACT_NONE, 0, alpha, beta, eps, weight_offset, post, pre, gates)
    check(LIB.vq_norm(spec, _address(block), _address(residual), T, _address(residual_out), _address(h),
                      _address(h_scales), _raw_stream(gpu)))
    return residual_out, h, h_scales
