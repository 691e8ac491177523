"""Python binding of ``libnvfp4ffn.so``, the MI355X (gfx950) dense SwiGLU FFN
with NVFP4 weights, the same FFN in 8-bit integers, the norms before and after
it, and the 8-bit paged KV cache and its attention next to it.

Argument marshalling only: every step of the FFN runs in the library's HIP
kernels; PyTorch supplies device memory and the current stream.  The names
and argument order follow the C ABI in ``include/nvfp4ffn.h``.  There is no
CPU fallback: if the library is not built, importing works but every call
raises :class:`Nvfp4LibraryMissing`.

Tensors: activations are ``torch.bfloat16`` ``[rows, cols]`` contiguous on
the GPU; a weight is any object with ``codes`` (uint8 ``[n, k/2]``),
``scales`` (uint8 ``[n, k/16]``, E4M3 bits) and ``tensor_scale`` (or
``ts``) -- see :class:`NVFP4Weight`; a W8A8 weight has ``codes`` (uint8
``[n, k]``, E4M3 bits) and ``scales`` (float32 ``[ceil(n/128),
ceil(k/128)]``) -- see :class:`FP8Weight`; an int8 weight has ``codes`` (int8
``[n, k]``) and ``scales`` (float32 ``[n]``) -- see :class:`Int8Weight` -- and
meets bf16 rows or :class:`Int8Rows`.  The ``kv8_*`` calls take a
:class:`KV8Cache`, a page table and lengths (int32, on the GPU) and bf16
``[rows, heads, dim]`` arrays that may be parts of a larger one; what they
return, unless the caller gave it, belongs to the stream they run on.
"""

from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import NamedTuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4ffn.so")

NVFP4_OK = 0
NVFP4_EINVAL = -1
NVFP4_ESHAPE = -2
NVFP4_ENOMEM = -3
NVFP4_EHIP = -4

__all__ = [
    "NVFP4Weight", "Nvfp4Error", "Nvfp4LibraryMissing",
    "nvfp4_gemm_w4a16", "nvfp4_gemm_w4a4", "nvfp4_quantize_rows", "silu_mul",
    "dense_ffn_forward_noalloc",
    "nvfp4_gate_up_silu_w4a16", "dense_ffn_forward", "dense_ffn_forward_w4a4",
    "nvfp4_gate_up_views", "dense_ffn_forward_fused", "LoraPair", "nvfp4_lora_delta",
    "dense_ffn_forward_lora", "FP8Weight", "fp8_quantize_rows", "fp8_gemm_w8a8",
    "dense_ffn_forward_w8a8", "Q2Weight", "q2_gemm_w2a16", "dense_ffn_forward_q2",
    "Int8Weight", "Int8Rows", "int8_quantize_rows", "int8_gemm_w8a8", "dense_ffn_forward_int8",
    "int8_workspace", "rms_norm", "rms_norm_residual",
    "KV8Cache", "kv8_cache", "kv8_append", "kv8_attention", "kv8_workspace", "kv8_evict",
    "kv8_evict_workspace",
    "nvfp4_last_error", "nvfp4_release", "nvfp4_abi_version", "load_library",
    "nvfp4_probe_mfma_bf16",
    "nvfp4_probe_read",
    "nvfp4_probe_encode",
]


class Nvfp4Error(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"nvfp4ffn error {code}: {message}")
        self.code = code


class Nvfp4LibraryMissing(RuntimeError):
    pass


class _CWeight(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("tensor_scale", ctypes.c_float),
        ("n", ctypes.c_int32),
        ("k", ctypes.c_int32),
    ]


class _CLoraPair(ctypes.Structure):
    _fields_ = [
        ("a", ctypes.c_void_p),
        ("b", ctypes.c_void_p),
        ("rank", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class _CLora(ctypes.Structure):
    _fields_ = [("gate", _CLoraPair), ("up", _CLoraPair), ("down", _CLoraPair)]


@dataclass
class LoraPair:
    """One LoRA pair on the GPU: dW = scale * b . a, a bf16 [rank, k], b bf16 [n, rank]."""
    a: torch.Tensor
    b: torch.Tensor
    scale: float = 1.0


@dataclass
class NVFP4Weight:
    """One NVFP4 matrix W[n][k] on the GPU."""
    codes: torch.Tensor    # uint8 [n, k/2], even k in the low nibble
    scales: torch.Tensor   # uint8 [n, k/16], E4M3FN bit patterns
    tensor_scale: float = 1.0


@dataclass
class FP8Weight:
    """One block-scaled FP8 matrix W[n][k] on the GPU."""
    codes: torch.Tensor   # uint8 [n, k], E4M3FN bit patterns
    scales: torch.Tensor  # float32 [ceil(n/128), ceil(k/128)]


class _CFp8Weight(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("n", ctypes.c_int32),
        ("k", ctypes.c_int32),
    ]


@dataclass
class Q2Weight:
    """One packed-Q2 matrix W[n][k] on the GPU."""
    codes: torch.Tensor   # uint8 [n, k/4], element 4j+i in bits 2i..2i+1 of byte j
    scales: torch.Tensor  # fp16 (or its uint16/int16 bits) [n, k/group]
    group: int = 128


class _CQ2Weight(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("group", ctypes.c_int32),
        ("n", ctypes.c_int32),
        ("k", ctypes.c_int32),
    ]


@dataclass
class Int8Weight:
    """One int8 matrix W[n][k] on the GPU with a scale for each output channel
    (int8_quantize_rows of a bf16 weight gives its fields)."""
    codes: torch.Tensor   # int8 [n, k]
    scales: torch.Tensor  # float32 [n]


class Int8Rows(NamedTuple):
    """Activation rows in int8 on the GPU with a scale for each row."""
    codes: torch.Tensor      # int8 [m, k]
    row_scale: torch.Tensor  # float32 [m]


class _CInt8Weight(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("n", ctypes.c_int32),
        ("k", ctypes.c_int32),
    ]


@dataclass
class KV8Cache:
    """A pool of pages of an 8-bit KV cache on the GPU.  A page's codes of one
    head are in the kernels' operand order (include/nvfp4ffn.h), not in
    [page, dim] order; the shape gives their sizes."""
    k_codes: torch.Tensor   # uint8 [pages, heads, page, dim], E4M3FN bit patterns
    v_codes: torch.Tensor   # as k_codes
    k_scales: torch.Tensor  # uint8 [pages, heads], E8M0: value = e4m3(code) * 2^(scale - 127)
    v_scales: torch.Tensor  # as k_scales
    weights: torch.Tensor | None = None  # float32 [pages, page], attention weight received


class _CKv8Cache(ctypes.Structure):
    _fields_ = [
        ("k_codes", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
        ("pages", ctypes.c_int32),
        ("heads", ctypes.c_int32),
        ("dim", ctypes.c_int32),
        ("page", ctypes.c_int32),
    ]


class _CKv8Batch(ctypes.Structure):
    _fields_ = [
        ("table", ctypes.c_void_p),
        ("lens", ctypes.c_void_p),
        ("starts", ctypes.c_void_p),
        ("seqs", ctypes.c_int32),
        ("cols", ctypes.c_int32),
        ("rows", ctypes.c_int32),
        ("max_rows", ctypes.c_int32),
        ("max_len", ctypes.c_int32),
    ]


class _CKv8Rows(ctypes.Structure):
    _fields_ = [
        ("ptr", ctypes.c_void_p),
        ("row_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
    ]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the C-ABI library and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise Nvfp4LibraryMissing(
            f"{path} is not built; run `python -m nvfp4_weight_dense_amd.build`")
    L = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    wp = ctypes.POINTER(_CWeight)
    f32 = ctypes.c_float
    w8 = vp  # a packed descriptor, or a reference to its ctypes structure
    kc = kb = kr = vp  # a packed descriptor, or a reference to its ctypes structure
    sig = {
        "nvfp4_gemm_w4a16": [vp, i32, wp, vp, vp],
        "nvfp4_gemm_w4a4": [vp, i32, wp, vp, vp],
        "nvfp4_quantize_rows": [vp, i32, i32, vp, vp, vp, vp],
        "silu_mul": [vp, vp, vp, i64, vp],
        "nvfp4_gate_up_silu_w4a16": [vp, i32, wp, wp, vp, vp],
        "dense_ffn_forward": [vp, i32, i32, i32, wp, wp, wp, vp, vp],
        "dense_ffn_forward_w4a4": [vp, i32, i32, i32, wp, wp, wp, vp, vp],
        "dense_ffn_forward_noalloc": [vp, i32, i32, i32, wp, wp, wp, vp, vp],
        "nvfp4_gate_up_views": [wp, wp, wp],
        "dense_ffn_forward_fused": [vp, i32, i32, i32, wp, wp, vp, vp],
        "nvfp4_lora_delta": [vp, i32, i32, ctypes.POINTER(_CLoraPair), i32, vp, vp],
        "dense_ffn_forward_lora": [vp, i32, i32, i32, wp, wp, wp, ctypes.POINTER(_CLora), vp, vp],
        "q2_gemm_w2a16": [vp, i32, ctypes.POINTER(_CQ2Weight), vp, vp],
        "dense_ffn_forward_q2": [vp, i32, i32, i32, ctypes.POINTER(_CQ2Weight),
                                 ctypes.POINTER(_CQ2Weight), ctypes.POINTER(_CQ2Weight), vp, vp],
        "fp8_quantize_rows": [vp, i32, i32, vp, vp, vp],
        "fp8_gemm_w8a8": [vp, i32, ctypes.POINTER(_CFp8Weight), vp, vp],
        "dense_ffn_forward_w8a8": [vp, i32, i32, i32, ctypes.POINTER(_CFp8Weight),
                                   ctypes.POINTER(_CFp8Weight), ctypes.POINTER(_CFp8Weight), vp, vp],
        "int8_quantize_rows": [vp, i32, i32, vp, vp, vp],
        "int8_gemm_w8a8": [vp, vp, i32, w8, vp, vp, i64, vp],
        "dense_ffn_forward_int8": [vp, vp, i32, i32, i32, w8, w8, w8, vp, vp, i64, vp],
        "rms_norm": [vp, i32, i32, vp, f32, f32, vp, vp, vp, vp],
        "rms_norm_residual": [vp, vp, i32, i32, i32, vp, vp, i32, f32, i32, vp, f32, f32, vp, vp, vp, vp, vp],
        "kv8_append": [kr, kr, kc, kb, vp],
        "kv8_attention": [kr, i32, ctypes.c_float, i32, kc, kb, vp, vp, i32, vp, i64, vp],
        "kv8_evict": [kc, kb, vp, i32, i32, i32, i32, vp, vp, vp],
        "kv8_evict_noalloc": [kc, kb, vp, i32, i32, i32, i32, vp, vp, vp, i64, vp],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    L.nvfp4_probe_mfma_bf16.argtypes = [i32, i32, vp, vp]
    L.nvfp4_probe_mfma_bf16.restype = ctypes.c_int
    L.nvfp4_probe_read.argtypes = [vp, i64, ctypes.c_uint32, vp, vp]
    L.nvfp4_probe_read.restype = ctypes.c_int
    L.nvfp4_probe_encode.argtypes = [vp, i64, ctypes.c_float, vp, vp, vp, vp]
    L.nvfp4_probe_encode.restype = ctypes.c_int
    L.int8_gemm_workspace.argtypes = [i32, w8]
    L.int8_gemm_workspace.restype = i64
    L.dense_ffn_int8_workspace.argtypes = [i32, i32, i32]
    L.dense_ffn_int8_workspace.restype = i64
    L.kv8_attention_workspace.argtypes = [i32, kc, kb]
    L.kv8_attention_workspace.restype = i64
    L.kv8_evict_workspace.argtypes = [kc, kb]
    L.kv8_evict_workspace.restype = i64
    L.nvfp4_last_error.argtypes = []
    L.nvfp4_last_error.restype = ctypes.c_char_p
    L.nvfp4_release.argtypes = []
    L.nvfp4_release.restype = None
    L.nvfp4_abi_version.argtypes = []
    L.nvfp4_abi_version.restype = ctypes.c_int32
    _lib = L
    return L


# ---- marshalling helpers -------------------------------------------------------

_U8, _I8, _I32, _F32, _BF16 = torch.uint8, torch.int8, torch.int32, torch.float32, torch.bfloat16


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(rc: int):
    if rc != NVFP4_OK:
        raise Nvfp4Error(rc, nvfp4_last_error())


def _act(t: torch.Tensor, name: str, k: int | None = None) -> torch.Tensor:
    """A bf16 [rows, cols] activation; with k, cols must equal k."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.dim() != 2 \
            or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous 2-D bfloat16 tensor")
    if k is not None and t.shape[1] != k:
        raise ValueError(f"{name}: has {t.shape[1]} columns, the weight has k={k}")
    return t


def _out(t: torch.Tensor | None, m: int, n: int, like: torch.Tensor, name: str) -> torch.Tensor:
    """A caller's bf16 [m, n] output (checked), or a new one on like's device."""
    if t is None:
        return torch.empty((m, n), dtype=torch.bfloat16, device=like.device)
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.dim() != 2 \
            or tuple(t.shape) != (m, n) or not t.is_contiguous():
        got = tuple(t.shape) if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: expected a contiguous bfloat16 [{m}, {n}] tensor, got {got}")
    return t


def _gpu(first: torch.Tensor, *rest):
    """Every tensor on the GPU, on first's device (checked after the shapes)."""
    if not first.is_cuda:
        raise ValueError("expected GPU tensors")
    for t in rest:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors on {t.device} and {first.device}: expected one device")


def _cweight(w) -> _CWeight:
    codes, scales = w.codes, w.scales
    ts = getattr(w, "tensor_scale", None)
    if ts is None:
        ts = w.ts
    for t, nm in ((codes, "codes"), (scales, "scales")):
        if t.dtype != torch.uint8 or t.dim() != 2 or not t.is_contiguous():
            raise ValueError(f"weight {nm}: expected a contiguous 2-D uint8 tensor")
    n, half_k = codes.shape
    if tuple(scales.shape) != (n, (2 * half_k) // 16):
        raise ValueError(f"weight scales: expected [n={n}, k/16={(2 * half_k) // 16}], "
                         f"got {tuple(scales.shape)}")
    return _CWeight(codes.data_ptr(), scales.data_ptr(), float(ts), int(n), int(half_k * 2))


def _wt(w):
    """The weight's tensors (for the device check)."""
    return (w.codes, w.scales)


# ---- C ABI, same names --------------------------------------------------------

def nvfp4_abi_version() -> int:
    return int(load_library().nvfp4_abi_version())


def nvfp4_last_error() -> str:
    return load_library().nvfp4_last_error().decode()


def nvfp4_release() -> None:
    load_library().nvfp4_release()


def nvfp4_probe_mfma_bf16(workgroups: int, iters: int, sink: torch.Tensor, stream=None) -> None:
    """Enqueue the register-only bf16 MFMA loop (a measurement aid):
    workgroups * 4 * iters * 4 * 32768 flops; sink is a float32 GPU tensor of
    at least 256 elements."""
    L = load_library()
    if sink.dtype != torch.float32 or sink.numel() < 256 or not sink.is_cuda:
        raise ValueError("sink: expected a float32 GPU tensor of at least 256 elements")
    _check(L.nvfp4_probe_mfma_bf16(int(workgroups), int(iters), _ptr(sink), _stream(stream)))


def nvfp4_probe_read(src: torch.Tensor, nbytes: int, never: int, sink: torch.Tensor, stream=None) -> None:
    """Enqueue one streaming read of the first nbytes bytes of src (a
    measurement aid; a contiguous GPU tensor, nbytes a multiple of 16 within
    it); sink is a float32 GPU tensor of at least 256 elements, written only
    if the xor fold of the bytes equals `never`."""
    L = load_library()
    if not src.is_cuda or not src.is_contiguous() or nbytes > src.numel() * src.element_size():
        raise ValueError("src: expected a contiguous GPU tensor holding nbytes bytes")
    if sink.dtype != torch.float32 or sink.numel() < 256 or not sink.is_cuda:
        raise ValueError("sink: expected a float32 GPU tensor of at least 256 elements")
    _check(L.nvfp4_probe_read(_ptr(src), int(nbytes), int(never) & 0xFFFFFFFF, _ptr(sink), _stream(stream)))


def nvfp4_probe_encode(x: torch.Tensor, d: float, stream=None):
    """The activation quantizers' division and rounding steps on arbitrary
    values (a test aid): x a contiguous float32 GPU tensor with a multiple of
    8 elements, d a positive finite divisor.  Returns (q, e2m1, e4m3): q =
    x / d as the quantizers divide (fp32), and the E2M1 code and E4M3FN byte
    of each x (uint8), as the quantizers encode."""
    L = load_library()
    if not x.is_cuda or x.dtype != torch.float32 or not x.is_contiguous() or x.numel() % 8 != 0 \
            or x.numel() == 0:
        raise ValueError("x: expected a contiguous float32 GPU tensor, a positive multiple of 8 elements")
    q = torch.empty_like(x)
    e2m1 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    e4m3 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(L.nvfp4_probe_encode(_ptr(x), x.numel(), float(d), _ptr(q), _ptr(e2m1), _ptr(e4m3),
                                _stream(stream)))
    return q, e2m1, e4m3


def nvfp4_gemm_w4a16(x: torch.Tensor, w, y: torch.Tensor | None = None, stream=None):
    """y = bf16(x . W^T); x [m, k] bf16 -> y [m, n] bf16."""
    L = load_library()
    cw = _cweight(w)
    x = _act(x, "x", cw.k)
    y = _out(y, x.shape[0], cw.n, x, "y")
    _gpu(x, y, *_wt(w))
    _check(L.nvfp4_gemm_w4a16(_ptr(x), x.shape[0], ctypes.byref(cw), _ptr(y), _stream(stream)))
    return y


def nvfp4_gemm_w4a4(x: torch.Tensor, w, y: torch.Tensor | None = None, stream=None):
    """W4A4 projection: x quantized per row to NVFP4, then x_q . W^T."""
    L = load_library()
    cw = _cweight(w)
    x = _act(x, "x", cw.k)
    y = _out(y, x.shape[0], cw.n, x, "y")
    _gpu(x, y, *_wt(w))
    _check(L.nvfp4_gemm_w4a4(_ptr(x), x.shape[0], ctypes.byref(cw), _ptr(y), _stream(stream)))
    return y


def nvfp4_quantize_rows(x: torch.Tensor, stream=None):
    """Per-row NVFP4 quantizer -> (codes [m, k/2], scales [m, k/16], row_scale [m])."""
    L = load_library()
    x = _act(x, "x")
    _gpu(x)
    m, k = x.shape
    codes = torch.empty((m, k // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((m, k // 16), dtype=torch.uint8, device=x.device)
    rs = torch.empty((m,), dtype=torch.float32, device=x.device)
    _check(L.nvfp4_quantize_rows(_ptr(x), m, k, _ptr(codes), _ptr(scales), _ptr(rs),
                                 _stream(stream)))
    return codes, scales, rs


def silu_mul(gate: torch.Tensor, up: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    """out = bf16(silu(gate) * up); out may be gate."""
    L = load_library()
    for t, nm in ((gate, "gate"), (up, "up")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"silu_mul: {nm} must be a contiguous bf16 tensor")
    if gate.shape != up.shape:
        raise ValueError("silu_mul: gate and up must have one shape")
    if out is None:
        out = torch.empty_like(gate)
    elif not isinstance(out, torch.Tensor) or out.dtype != torch.bfloat16 or \
            out.shape != gate.shape or not out.is_contiguous():
        raise ValueError("silu_mul: out must be a contiguous bf16 tensor of gate's shape")
    _gpu(gate, up, out)
    _check(L.silu_mul(_ptr(gate), _ptr(up), _ptr(out), gate.numel(), _stream(stream)))
    return out


def nvfp4_gate_up_silu_w4a16(x: torch.Tensor, wg, wu, act: torch.Tensor | None = None,
                             stream=None):
    """act = bf16(silu(bf16(x.Wg^T)) * bf16(x.Wu^T))."""
    L = load_library()
    cg, cu = _cweight(wg), _cweight(wu)
    if (cg.n, cg.k) != (cu.n, cu.k):
        raise ValueError(f"wg [{cg.n}, {cg.k}] and wu [{cu.n}, {cu.k}] differ")
    x = _act(x, "x", cg.k)
    act = _out(act, x.shape[0], cg.n, x, "act")
    _gpu(x, act, *_wt(wg), *_wt(wu))
    _check(L.nvfp4_gate_up_silu_w4a16(_ptr(x), x.shape[0], ctypes.byref(cg), ctypes.byref(cu),
                                      _ptr(act), _stream(stream)))
    return act


def _ffn_shapes(x, g, u, d, out):
    """Check x [m, hidden], wg/wu [inter, hidden], wd [hidden, inter] and out
    [m, hidden]; returns (x, out, m, hidden, inter)."""
    inter, hidden = g
    if u != (inter, hidden) or d != (hidden, inter):
        raise ValueError(f"wg {list(g)}, wu {list(u)}, wd {list(d)}: expected wg/wu "
                         f"[inter, hidden] and wd [hidden, inter]")
    x = _act(x, "x", hidden)
    out = _out(out, x.shape[0], hidden, x, "out")
    return x, out, x.shape[0], hidden, inter


def _ffn(fn, x, wg, wu, wd, out, stream):
    cg, cu, cd = _cweight(wg), _cweight(wu), _cweight(wd)
    x, out, m, hidden, inter = _ffn_shapes(x, (cg.n, cg.k), (cu.n, cu.k), (cd.n, cd.k), out)
    _gpu(x, out, *_wt(wg), *_wt(wu), *_wt(wd))
    _check(fn(_ptr(x), m, hidden, inter, ctypes.byref(cg), ctypes.byref(cu), ctypes.byref(cd),
              _ptr(out), _stream(stream)))
    return out


def dense_ffn_forward(x: torch.Tensor, wg, wu, wd, out: torch.Tensor | None = None, stream=None):
    """W4A16 dense SwiGLU FFN: out = (silu(x.Wg^T) * (x.Wu^T)) . Wd^T."""
    return _ffn(load_library().dense_ffn_forward, x, wg, wu, wd, out, stream)


def dense_ffn_forward_w4a4(x: torch.Tensor, wg, wu, wd, out: torch.Tensor | None = None,
                           stream=None):
    """Fixed-format W4A4 FFN (activations quantized per row before each projection)."""
    return _ffn(load_library().dense_ffn_forward_w4a4, x, wg, wu, wd, out, stream)


def dense_ffn_forward_noalloc(x: torch.Tensor, wg, wu, wd, out: torch.Tensor | None = None,
                              stream=None):
    """dense_ffn_forward with the library's fixed device scratch instead of its
    arena: the C call allocates nothing (out, when not given, is allocated
    here by torch).  Shapes whose scratch does not fit raise Nvfp4Error
    (NVFP4_ENOMEM)."""
    return _ffn(load_library().dense_ffn_forward_noalloc, x, wg, wu, wd, out, stream)


def nvfp4_gate_up_views(fused) -> tuple[NVFP4Weight, NVFP4Weight]:
    """(gate, up) views into a fused gate+up weight [2*inter, hidden]: row
    slices of the same codes/scales storage, at the offsets the C-ABI call
    reports (checked here)."""
    L = load_library()
    cf = _cweight(fused)
    cg, cu = _CWeight(), _CWeight()
    _check(L.nvfp4_gate_up_views(ctypes.byref(cf), ctypes.byref(cg), ctypes.byref(cu)))
    inter = cg.n
    ts = float(cf.tensor_scale)
    gate = NVFP4Weight(fused.codes[:inter], fused.scales[:inter], ts)
    up = NVFP4Weight(fused.codes[inter:], fused.scales[inter:], ts)
    for view, c in ((gate, cg), (up, cu)):
        assert view.codes.data_ptr() == c.codes and view.scales.data_ptr() == c.scales
    return gate, up


def dense_ffn_forward_fused(x: torch.Tensor, wgu, wd, out: torch.Tensor | None = None,
                            stream=None):
    """W4A16 dense SwiGLU FFN on a fused gate+up weight [2*inter, hidden]."""
    L = load_library()
    cgu, cd = _cweight(wgu), _cweight(wd)
    if cgu.n % 2:
        raise ValueError(f"wgu: {cgu.n} rows, expected 2*inter")
    inter = cgu.n // 2
    x, out, m, hidden, _ = _ffn_shapes(x, (inter, cgu.k), (inter, cgu.k), (cd.n, cd.k), out)
    _gpu(x, out, *_wt(wgu), *_wt(wd))
    _check(L.dense_ffn_forward_fused(_ptr(x), m, hidden, inter, ctypes.byref(cgu), ctypes.byref(cd),
                                     _ptr(out), _stream(stream)))
    return out


def _clora_pair(p: LoraPair | None, k: int, n: int, name: str) -> _CLoraPair:
    """A LoRA pair for a delta on an [m, n] output from a [m, k] input."""
    if p is None:
        return _CLoraPair(None, None, 0, 0.0)
    for t, nm in ((p.a, "a"), (p.b, "b")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.dim() != 2 \
                or not t.is_contiguous():
            raise ValueError(f"{name} {nm}: expected a contiguous 2-D bfloat16 tensor")
    r = p.a.shape[0]
    if tuple(p.a.shape) != (r, k) or tuple(p.b.shape) != (n, r):
        raise ValueError(f"{name}: a is [rank, k={k}] and b is [n={n}, rank], got a "
                         f"{list(p.a.shape)} and b {list(p.b.shape)}")
    return _CLoraPair(p.a.data_ptr(), p.b.data_ptr(), int(r), float(p.scale))


def _lora_t(p: LoraPair | None):
    return () if p is None else (p.a, p.b)


def nvfp4_lora_delta(x: torch.Tensor, pair: LoraPair, base: torch.Tensor, stream=None):
    """base += pair.scale * (x . a^T) . b^T in place (bf16 base [m, n])."""
    L = load_library()
    x = _act(x, "x")
    base = _act(base, "base")
    m, k = x.shape
    if base.shape[0] != m:
        raise ValueError(f"base: {base.shape[0]} rows, x has {m}")
    if pair is None:
        raise ValueError("lora_delta: pair is None")
    cp = _clora_pair(pair, k, base.shape[1], "lora pair")
    _gpu(x, base, *_lora_t(pair))
    _check(L.nvfp4_lora_delta(_ptr(x), m, k, ctypes.byref(cp), base.shape[1],
                              _ptr(base), _stream(stream)))
    return base


def dense_ffn_forward_lora(x: torch.Tensor, wg, wu, wd, gate: LoraPair | None = None,
                           up: LoraPair | None = None, down: LoraPair | None = None,
                           out: torch.Tensor | None = None, stream=None):
    """W4A16 dense SwiGLU FFN with a LoRA overlay on gate, up and down."""
    L = load_library()
    cg, cu, cd = _cweight(wg), _cweight(wu), _cweight(wd)
    x, out, m, hidden, inter = _ffn_shapes(x, (cg.n, cg.k), (cu.n, cu.k), (cd.n, cd.k), out)
    cl = _CLora(_clora_pair(gate, hidden, inter, "lora gate"), _clora_pair(up, hidden, inter, "lora up"),
                _clora_pair(down, inter, hidden, "lora down"))
    _gpu(x, out, *_wt(wg), *_wt(wu), *_wt(wd), *_lora_t(gate), *_lora_t(up), *_lora_t(down))
    _check(L.dense_ffn_forward_lora(_ptr(x), m, hidden, inter, ctypes.byref(cg), ctypes.byref(cu),
                                    ctypes.byref(cd), ctypes.byref(cl), _ptr(out), _stream(stream)))
    return out


# ---- W8A8 fixed format ----------------------------------------------------------

def _cfp8(w) -> _CFp8Weight:
    if w.codes.dtype != torch.uint8 or w.codes.dim() != 2 or not w.codes.is_contiguous():
        raise ValueError("fp8 weight codes: expected a contiguous 2-D uint8 tensor")
    if w.scales.dtype != torch.float32 or not w.scales.is_contiguous():
        raise ValueError("fp8 weight scales: expected a contiguous float32 tensor")
    n, k = w.codes.shape
    if tuple(w.scales.shape) != ((n + 127) // 128, (k + 127) // 128):
        raise ValueError("fp8 weight scales: expected [ceil(n/128), ceil(k/128)]")
    return _CFp8Weight(w.codes.data_ptr(), w.scales.data_ptr(), int(n), int(k))


def fp8_quantize_rows(x: torch.Tensor, stream=None):
    """Per-row FP8 quantizer -> (codes uint8 [m, k] E4M3, row_scale float32 [m])."""
    L = load_library()
    x = _act(x, "x")
    _gpu(x)
    m, k = x.shape
    codes = torch.empty((m, k), dtype=torch.uint8, device=x.device)
    rs = torch.empty((m,), dtype=torch.float32, device=x.device)
    _check(L.fp8_quantize_rows(_ptr(x), m, k, _ptr(codes), _ptr(rs), _stream(stream)))
    return codes, rs


def fp8_gemm_w8a8(x: torch.Tensor, w, y: torch.Tensor | None = None, stream=None):
    """W8A8 projection: x quantized per row to FP8, then x_q . W^T (block-scaled W)."""
    L = load_library()
    cw = _cfp8(w)
    x = _act(x, "x", cw.k)
    y = _out(y, x.shape[0], cw.n, x, "y")
    _gpu(x, y, *_wt(w))
    _check(L.fp8_gemm_w8a8(_ptr(x), x.shape[0], ctypes.byref(cw), _ptr(y), _stream(stream)))
    return y


def dense_ffn_forward_w8a8(x: torch.Tensor, wg, wu, wd, out: torch.Tensor | None = None,
                           stream=None):
    """Fixed-format W8A8 FFN (FP8 activations per row, block-scaled FP8 weights)."""
    L = load_library()
    cg, cu, cd = _cfp8(wg), _cfp8(wu), _cfp8(wd)
    x, out, m, hidden, inter = _ffn_shapes(x, (cg.n, cg.k), (cu.n, cu.k), (cd.n, cd.k), out)
    _gpu(x, out, *_wt(wg), *_wt(wu), *_wt(wd))
    _check(L.dense_ffn_forward_w8a8(_ptr(x), m, hidden, inter, ctypes.byref(cg), ctypes.byref(cu),
                                    ctypes.byref(cd), _ptr(out), _stream(stream)))
    return out


# ---- packed-Q2 weights ------------------------------------------------------------

def _cq2(w) -> _CQ2Weight:
    if w.codes.dtype != torch.uint8 or w.codes.dim() != 2 or not w.codes.is_contiguous():
        raise ValueError("q2 weight codes: expected a contiguous 2-D uint8 tensor")
    if w.scales.element_size() != 2 or not w.scales.is_contiguous():
        raise ValueError("q2 weight scales: expected a contiguous 16-bit tensor of fp16 bits")
    n, k4 = w.codes.shape
    if int(w.group) <= 0 or tuple(w.scales.shape) != (n, (4 * k4) // int(w.group)):
        raise ValueError("q2 weight scales: expected [n, k/group]")
    return _CQ2Weight(w.codes.data_ptr(), w.scales.data_ptr(), int(w.group), int(n), int(4 * k4))


def q2_gemm_w2a16(x: torch.Tensor, w, y: torch.Tensor | None = None, stream=None):
    """y = bf16(x . W^T) with W = bf16((q - 2) * d) from a packed-Q2 weight."""
    L = load_library()
    cw = _cq2(w)
    x = _act(x, "x", cw.k)
    y = _out(y, x.shape[0], cw.n, x, "y")
    _gpu(x, y, *_wt(w))
    _check(L.q2_gemm_w2a16(_ptr(x), x.shape[0], ctypes.byref(cw), _ptr(y), _stream(stream)))
    return y


def dense_ffn_forward_q2(x: torch.Tensor, wg, wu, wd, out: torch.Tensor | None = None,
                         stream=None):
    """Dense SwiGLU FFN on packed-Q2 weights (bf16 activations)."""
    L = load_library()
    cg, cu, cd = _cq2(wg), _cq2(wu), _cq2(wd)
    x, out, m, hidden, inter = _ffn_shapes(x, (cg.n, cg.k), (cu.n, cu.k), (cd.n, cd.k), out)
    _gpu(x, out, *_wt(wg), *_wt(wu), *_wt(wd))
    _check(L.dense_ffn_forward_q2(_ptr(x), m, hidden, inter, ctypes.byref(cg), ctypes.byref(cu),
                                  ctypes.byref(cd), _ptr(out), _stream(stream)))
    return out


# ---- 8-bit integers ------------------------------------------------------------------

_pack_int8 = struct.Struct("@2P2i").pack


def _cint8(w):
    """(packed int8_weight, n, k)"""
    c, s = w.codes, w.scales
    if c.dtype is not _I8 or c.dim() != 2 or not c.is_contiguous():
        raise ValueError("int8 weight codes: expected a contiguous 2-D int8 tensor")
    n, k = c.shape
    if s.dtype is not _F32 or s.shape != (n,) or not s.is_contiguous():
        raise ValueError(f"int8 weight scales: expected a contiguous float32 [{n}] tensor")
    return _pack_int8(c.data_ptr(), s.data_ptr(), n, k), n, k


def _int8_x(x, k: int):
    """(tensor, its scales' tensor or None) of bf16 rows or Int8Rows with k columns"""
    if not isinstance(x, Int8Rows):
        return _act(x, "x", k), None
    c, s = x
    if c.dtype is not _I8 or c.dim() != 2 or not c.is_contiguous():
        raise ValueError("x codes: expected a contiguous 2-D int8 tensor")
    if c.shape[1] != k:
        raise ValueError(f"x: has {c.shape[1]} columns, the weight has k={k}")
    if s.dtype is not _F32 or s.shape != c.shape[:1] or not s.is_contiguous():
        raise ValueError(f"x row_scale: expected a contiguous float32 [{c.shape[0]}] tensor")
    return c, s


def _on_current(first: torch.Tensor, *rest) -> int:
    """Every tensor on one GPU, which is the current one (checked after the shapes); its index."""
    dev = first.get_device()
    _kv8_on(dev, *rest)
    return dev


def _rows_workspace(t):
    if t is not None and (t.dtype != torch.uint8 or not t.is_contiguous()):
        raise ValueError("workspace: expected a contiguous uint8 tensor (int8_workspace)")
    return (None, 0) if t is None else (t.data_ptr(), t.numel())


def _bf16_out(t, shape, name):
    """A caller's bf16 output (checked); None for one to be made."""
    if t is not None and (not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or t.shape != shape
                          or not t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous bfloat16 {list(shape)} tensor")
    return t


def int8_quantize_rows(x: torch.Tensor, stream=None) -> Int8Rows:
    """Per-row int8 quantizer: Int8Rows(codes int8 [m, k], row_scale float32
    [m]) of bf16 rows (activations, or a weight by its output channels)."""
    L = load_library()
    x = _act(x, "x")
    dev = _on_current(x)
    m, k = x.shape
    codes = _kv8_empty((m, k), _I8, x.device, stream)
    rs = _kv8_empty((m,), _F32, x.device, stream)
    _check(L.int8_quantize_rows(x.data_ptr(), m, k, codes.data_ptr(), rs.data_ptr(), _kv8_stream(stream, dev)))
    return Int8Rows(codes, rs)


def int8_workspace(m: int, *weights) -> torch.Tensor:
    """A workspace for calls of int8_gemm_w8a8 (one weight) or
    dense_ffn_forward_int8 (wg, wu, wd) with these weights and m rows or fewer,
    for one stream (it is cleared on the current one).  Without one, calls
    share the library's scratch arena; a captured call has to bring one."""
    L = load_library()
    c = [_cint8(w) for w in weights]
    m = _i32(m, "m")
    if len(c) == 1:
        n = L.int8_gemm_workspace(m, c[0][0])
    elif len(c) == 3:
        n = L.dense_ffn_int8_workspace(m, c[0][2], c[0][1])
    else:
        raise ValueError(f"{len(c)} weights: expected one, or wg, wu and wd")
    if n < 0:
        _check(int(n))
    return torch.zeros((max(n, 256),), dtype=torch.uint8, device=weights[0].codes.device)


def int8_gemm_w8a8(x, w, y: torch.Tensor | None = None, *, workspace: torch.Tensor | None = None, stream=None):
    """Projection in 8-bit integers: y = bf16(s_row * s_col * (x8 . W8^T)).
    x: bf16 [m, k], quantized by rows in the call, or Int8Rows."""
    L = load_library()
    cw, n, k = _cint8(w)
    xt, xs = _int8_x(x, k)
    m = xt.shape[0]
    y = _bf16_out(y, (m, n), "y")
    ws, nbytes = _rows_workspace(workspace)
    dev = _on_current(xt, xs, y, workspace, w.codes, w.scales)
    if y is None:
        y = _kv8_empty((m, n), _BF16, xt.device, stream)
    _check(L.int8_gemm_w8a8(xt.data_ptr(), None if xs is None else xs.data_ptr(), m, cw, y.data_ptr(), ws, nbytes,
                            _kv8_stream(stream, dev)))
    return y


def dense_ffn_forward_int8(x, wg, wu, wd, out: torch.Tensor | None = None, *,
                           workspace: torch.Tensor | None = None, stream=None):
    """Dense SwiGLU FFN in 8-bit integers (x and act quantized by rows before
    each projection).  x: bf16 [m, hidden] or Int8Rows."""
    L = load_library()
    (cg, inter, hidden), (cu, nu, ku), (cd, nd, kd) = _cint8(wg), _cint8(wu), _cint8(wd)
    if (nu, ku) != (inter, hidden) or (nd, kd) != (hidden, inter):
        raise ValueError(f"wg {[inter, hidden]}, wu {[nu, ku]}, wd {[nd, kd]}: expected wg/wu "
                         f"[inter, hidden] and wd [hidden, inter]")
    xt, xs = _int8_x(x, hidden)
    m = xt.shape[0]
    out = _bf16_out(out, (m, hidden), "out")
    ws, nbytes = _rows_workspace(workspace)
    dev = _on_current(xt, xs, out, workspace, wg.codes, wg.scales, wu.codes, wu.scales, wd.codes, wd.scales)
    if out is None:
        out = _kv8_empty((m, hidden), _BF16, xt.device, stream)
    _check(L.dense_ffn_forward_int8(xt.data_ptr(), None if xs is None else xs.data_ptr(), m, hidden, inter, cg, cu, cd,
                                    out.data_ptr(), ws, nbytes, _kv8_stream(stream, dev)))
    return out


# ---- norms before and after a block -----------------------------------------------------

def _norm_weight(w, k: int, name: str):
    """(whether there is a norm, its weight's tensor or None); w: None (no norm), True (no weight) or bf16 [k]"""
    if w is None or w is False:
        return 0, None
    if w is True:
        return 1, None
    if not isinstance(w, torch.Tensor) or w.dtype is not _BF16 or w.shape != (k,) or not w.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous bfloat16 [{k}] tensor")
    return 1, w


def _at(t):
    return None if t is None else t.data_ptr()


def rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, *, eps: float = 1e-6, weight_offset: float = 0.0,
             int8: bool = False, out: torch.Tensor | None = None, stream=None):
    """x / sqrt(mean(x^2) + eps) * (weight_offset + weight) over the rows of x
    (bf16 [m, k]): bf16 [m, k] (out, which may be x), or with int8 the Int8Rows
    that int8_quantize_rows makes of it."""
    L = load_library()
    x = _act(x, "x")
    m, k = x.shape
    _, w = _norm_weight(weight, k, "weight")
    out = _bf16_out(out, (m, k), "out")
    if int8 and out is not None:
        raise ValueError("out: int8 rows are returned anew")
    dev = _on_current(x, w, out)
    q = None
    if int8:
        q = Int8Rows(_kv8_empty((m, k), _I8, x.device, stream), _kv8_empty((m,), _F32, x.device, stream))
    elif out is None:
        out = _kv8_empty((m, k), _BF16, x.device, stream)
    _check(L.rms_norm(x.data_ptr(), m, k, _at(w), float(weight_offset), float(eps), _at(out),
                      q and q.codes.data_ptr(), q and q.row_scale.data_ptr(), _kv8_stream(stream, dev)))
    return q if int8 else out


def rms_norm_residual(residual: torch.Tensor, y: torch.Tensor, *, post=None, gate: torch.Tensor | None = None,
                      scale: float = 1.0, norm=None, eps: float = 1e-6, weight_offset: float = 0.0,
                      int8: bool = False, h: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """The end of a block, y its output (bf16 [m, k]), and the start of the next:

        h = bf16(residual + scale * gate * post_norm(y)),  n = norm(h)

    post and norm: None (no such norm), True (one without a weight) or the
    norm's weight (bf16 [k]; with weight_offset as in rms_norm).  gate: bf16
    [k], or [gates, k] with gates a divisor of m, each row for m / gates rows.
    h may be residual or y.  Returns (h, n); n is bf16, Int8Rows with int8, or
    None without a norm."""
    L = load_library()
    residual, y = _act(residual, "residual"), _act(y, "y")
    m, k = residual.shape
    if y.shape != residual.shape:
        raise ValueError(f"y: has shape {tuple(y.shape)}, residual {tuple(residual.shape)}")
    post, pw = _norm_weight(post, k, "post")
    nxt, nw = _norm_weight(norm, k, "norm")
    gates = 0
    if gate is not None:
        if not isinstance(gate, torch.Tensor) or gate.dtype is not _BF16 or not gate.is_contiguous() \
                or gate.dim() not in (1, 2) or gate.shape[-1] != k:
            raise ValueError(f"gate: expected a contiguous bfloat16 [{k}] or [gates, {k}] tensor")
        gates = 1 if gate.dim() == 1 else gate.shape[0]
        if m % gates if gates else m:
            raise ValueError(f"gate: {gates} rows do not divide {m}")
        if not gates:  # (no rows, no gates)
            gate = None
    h, out = _bf16_out(h, (m, k), "h"), _bf16_out(out, (m, k), "out")
    if out is not None and (int8 or not nxt):
        raise ValueError("out: only the bf16 result of a norm is written to it")
    if int8 and not nxt:
        raise ValueError("int8: there is no norm to quantize")
    dev = _on_current(residual, y, pw, nw, gate, h, out)
    if h is None:
        h = _kv8_empty((m, k), _BF16, y.device, stream)
    q = None
    if int8:
        q = Int8Rows(_kv8_empty((m, k), _I8, y.device, stream), _kv8_empty((m,), _F32, y.device, stream))
    elif nxt and out is None:
        out = _kv8_empty((m, k), _BF16, y.device, stream)
    _check(L.rms_norm_residual(residual.data_ptr(), y.data_ptr(), m, k, post, _at(pw), _at(gate), gates, float(scale),
                               nxt, _at(nw), float(weight_offset), float(eps), h.data_ptr(), _at(out),
                               q and q.codes.data_ptr(), q and q.row_scale.data_ptr(),
                               _kv8_stream(stream, dev)))
    return h, q if int8 else out


# ---- 8-bit paged KV cache -----------------------------------------------------------

def kv8_cache(pages: int, heads: int, dim: int, page: int = 64, weights: bool = False,
              device="cuda") -> KV8Cache:
    """An empty pool: `pages` pages of `page` tokens (16, 32, 64 or 128) of
    `heads` KV heads of size `dim` (64, 128 or 256); with weights, the
    attention weight each token receives is kept too (kv8_evict needs it)."""
    codes = [torch.zeros((pages, heads, page, dim), dtype=torch.uint8, device=device) for _ in "kv"]
    scales = [torch.full((pages, heads), 127, dtype=torch.uint8, device=device) for _ in "kv"]
    w = torch.zeros((pages, page), dtype=torch.float32, device=device) if weights else None
    return KV8Cache(*codes, *scales, w)


# The descriptors of include/nvfp4ffn.h as packed bytes (kv8_cache, kv8_batch,
# kv8_rows): a decode step is a few microseconds, and ctypes structures take
# one each to fill.  The ctypes classes above have the same layout.
_pack_cache = struct.Struct("@5P4i").pack
_pack_batch = struct.Struct("@3P5i4x").pack
_pack_rows = struct.Struct("@P2q").pack


def _kv8_refuse(c: KV8Cache):
    """Names what is wrong with a cache."""
    k, w = c.k_codes, c.weights
    if k.dtype != _U8 or k.dim() != 4 or not k.is_contiguous():
        raise ValueError("k_codes: expected a contiguous uint8 [pages, heads, page, dim] tensor")
    pages, heads, page, _ = k.shape
    if c.v_codes.dtype != _U8 or c.v_codes.shape != k.shape or not c.v_codes.is_contiguous():
        raise ValueError("v_codes: expected a contiguous uint8 tensor of k_codes' shape")
    for t, nm in ((c.k_scales, "k_scales"), (c.v_scales, "v_scales")):
        if t.dtype != _U8 or t.shape != (pages, heads) or not t.is_contiguous():
            raise ValueError(f"{nm}: expected a contiguous uint8 [{pages}, {heads}] tensor")
    if w is not None and (w.dtype != _F32 or w.shape != (pages, page) or not w.is_contiguous()):
        raise ValueError(f"weights: expected a contiguous float32 [{pages}, {page}] tensor")
    raise ValueError("cache tensors on several devices: expected one device")


def _ckv8(c: KV8Cache):
    """(packed kv8_cache, heads, page, dim, device index)"""
    k, v, ks, vs, w = c.k_codes, c.v_codes, c.k_scales, c.v_scales, c.weights
    shape, dev = k.shape, k.get_device()
    if not (len(shape) == 4 and k.dtype is _U8 and v.dtype is _U8 and ks.dtype is _U8 and vs.dtype is _U8
            and v.shape == shape and ks.shape == vs.shape == shape[:2]
            and k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()
            and v.get_device() == ks.get_device() == vs.get_device() == dev):
        _kv8_refuse(c)
    pages, heads, page, dim = shape
    at = 0
    if w is not None:
        if w.dtype is not _F32 or w.shape != (pages, page) or not w.is_contiguous() or w.get_device() != dev:
            _kv8_refuse(c)
        at = w.data_ptr()
    return _pack_cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), at, pages, heads, dim,
                       page), heads, page, dim, dev


def _ckv8_rows(x: torch.Tensor, name: str, dim: int, heads: int | None = None) -> bytes:
    """A bf16 [rows, heads, dim] array with strides of whole 16-byte pieces."""
    if not isinstance(x, torch.Tensor) or x.dtype is not _BF16 or x.dim() != 3:
        raise ValueError(f"{name}: expected a 3-D bfloat16 tensor [rows, heads, dim]")
    _, h, d = x.shape
    if d != dim or (heads is not None and h != heads):
        raise ValueError(f"{name}: has shape {tuple(x.shape)}, the cache has {heads or 'n'} heads of size {dim}")
    rs, hs, ds = x.stride()
    if ds != 1 or rs % 8 or hs % 8:
        raise ValueError(f"{name}: strides {x.stride()}: expected the last 1, the others multiples of 8")
    return _pack_rows(x.data_ptr(), rs, hs)


def _i32(x, name: str) -> int:
    """A whole number that the C ABI's int32 holds (ctypes would take it modulo 2^32)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name}: {x} does not fit 32 bits")
    return x


def _ckv8_batch(table, lens, starts, rows, max_rows, max_len, page):
    """(packed kv8_batch, seqs)"""
    if table.dtype is not _I32 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table: expected a contiguous int32 [seqs, cols] tensor")
    seqs, cols = table.shape
    if lens.dtype is not _I32 or lens.shape != (seqs,) or not lens.is_contiguous():
        raise ValueError(f"lens: expected a contiguous int32 [{seqs}] tensor")
    at = 0
    if starts is not None:
        if starts.dtype is not _I32 or starts.shape != (seqs + 1,) or not starts.is_contiguous():
            raise ValueError(f"starts: expected a contiguous int32 [{seqs + 1}] tensor")
        at = starts.data_ptr()
        max_rows = rows if max_rows is None else min(int(max_rows), rows)
    else:
        max_rows = rows // seqs if seqs else 0
    return _pack_batch(table.data_ptr(), lens.data_ptr(), at, seqs, cols, rows, max_rows,
                       cols * page if max_len is None else min(int(max_len), cols * page)), seqs


def _kv8_on(dev: int, *tensors):
    """Every tensor on the cache's GPU, which is the current one (checked after the shapes)."""
    if dev < 0:
        raise ValueError("expected GPU tensors")
    if torch._C._cuda_getDevice() != dev:  # (the library's launches and scratch are the current device's)
        raise ValueError(f"tensors on cuda:{dev}, the current device is cuda:{torch._C._cuda_getDevice()}")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {t.device} and cuda:{dev}: expected one device")


def _kv8_stream(stream, dev: int):
    # (the current stream's handle, without building a torch.cuda.Stream)
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _kv8_empty(shape, dtype, device, stream):
    """A tensor of the stream that uses it: memory that the caching allocator
    hands out belongs to the stream it was asked for on, so one of the current
    stream's could be taken for other work, when the caller drops it or before
    its last reader there has ended, while the call's kernels use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def kv8_append(k: torch.Tensor, v: torch.Tensor, cache: KV8Cache, table: torch.Tensor,
               lens: torch.Tensor, starts: torch.Tensor | None = None, *, max_rows: int | None = None,
               stream=None) -> None:
    """Write the rows of k and v (bf16 [rows, heads, dim]) into the cache.

    lens [seqs] counts each sequence's tokens with these; row i of a sequence
    with r rows is its token lens - r + i, on page table[seq, token // page].
    starts [seqs + 1] gives each sequence's rows; without it every sequence
    has rows / seqs.  max_rows bounds one sequence's rows (default: rows)."""
    L = load_library()
    cc, heads, page, dim, dev = _ckv8(cache)
    ck, cv = _ckv8_rows(k, "k", dim, heads), _ckv8_rows(v, "v", dim, heads)
    rows = k.shape[0]
    if v.shape[0] != rows:
        raise ValueError(f"v: {v.shape[0]} rows, k has {rows}")
    cb, _ = _ckv8_batch(table, lens, starts, rows, max_rows, None, page)
    _kv8_on(dev, k, v, table, lens, starts)
    _check(L.kv8_append(ck, cv, cc, cb, _kv8_stream(stream, dev)))


def kv8_workspace(q_heads: int, cache: KV8Cache, table: torch.Tensor, lens: torch.Tensor, rows: int,
                  starts: torch.Tensor | None = None, *, max_rows: int | None = None,
                  max_len: int | None = None) -> torch.Tensor:
    """A workspace for kv8_attention calls of these sizes or smaller ones, for
    one stream (without one, calls share the library's scratch arena)."""
    L = load_library()
    cc, _, page, _, _ = _ckv8(cache)
    n = L.kv8_attention_workspace(_i32(q_heads, "q_heads"), cc, _ckv8_batch(
        table, lens, starts, _i32(rows, "rows"), max_rows, max_len, page)[0])
    if n < 0:
        _check(int(n))
    return torch.zeros((max(n, 256),), dtype=torch.uint8, device=cache.k_codes.device)


def kv8_attention(q: torch.Tensor, cache: KV8Cache, table: torch.Tensor, lens: torch.Tensor,
                  starts: torch.Tensor | None = None, *, scale: float | None = None, window: int = 0,
                  max_rows: int | None = None, max_len: int | None = None, out: torch.Tensor | None = None,
                  lse=None, accumulate: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """Causal attention of the rows of q (bf16 [rows, q_heads, dim]) over the
    cache; rows, lens, starts and table as in kv8_append, whose rows the cache
    already holds.  scale defaults to dim ** -0.5; window > 0 limits a row to
    the last `window` tokens up to its own.  max_rows and max_len bound one
    sequence's rows and tokens (they size the launch; default: from rows and
    the table's width).

    Returns out (bf16 [rows, q_heads, dim]); with lse (True, or a float32
    [rows, q_heads] tensor to write to) returns (out, lse).  accumulate adds
    the attention weight each token receives to cache.weights (of a page that
    several sequences share, what it receives from each of them)."""
    L = load_library()
    cc, _, page, dim, dev = _ckv8(cache)
    cq = _ckv8_rows(q, "q", dim)
    shape = q.shape
    rows, q_heads, _ = shape
    cb, _ = _ckv8_batch(table, lens, starts, rows, max_rows, max_len, page)
    if out is not None and (out.dtype != torch.bfloat16 or out.shape != shape or not out.is_contiguous()):
        raise ValueError(f"out: expected a contiguous bfloat16 [{rows}, {q_heads}, {dim}] tensor")
    give = lse is not None and lse is not False
    make = lse is True or (accumulate and not give)
    if make or not give:
        lse = None
    elif lse.dtype != torch.float32 or lse.shape != (rows, q_heads) or not lse.is_contiguous():
        raise ValueError(f"lse: expected a contiguous float32 [{rows}, {q_heads}] tensor")
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
        raise ValueError("workspace: expected a contiguous uint8 tensor (kv8_workspace)")
    _kv8_on(dev, q, out, lse, workspace, table, lens, starts)
    if out is None:
        out = _kv8_empty(shape, torch.bfloat16, q.device, stream)
    if make:
        lse = _kv8_empty((rows, q_heads), torch.float32, q.device, stream)
    window = max(min(int(window), 2 ** 31 - 1), -1)  # (ctypes would take it modulo 2^32)
    _check(L.kv8_attention(cq, q_heads, dim ** -0.5 if scale is None else float(scale), window, cc, cb,
                           out.data_ptr(), None if lse is None else lse.data_ptr(), 1 if accumulate else 0,
                           None if workspace is None else workspace.data_ptr(),
                           0 if workspace is None else workspace.numel(), _kv8_stream(stream, dev)))
    return (out, lse) if give else out


def kv8_evict_workspace(cache: KV8Cache, table: torch.Tensor, lens: torch.Tensor, *,
                        max_len: int | None = None) -> torch.Tensor:
    """A workspace for kv8_evict calls of these sizes or smaller ones, for one
    stream (without one, calls of more than 32768 tokens share the library's
    scratch arena)."""
    L = load_library()
    cc, _, page, _, _ = _ckv8(cache)
    n = L.kv8_evict_workspace(cc, _ckv8_batch(table, lens, None, 0, None, max_len, page)[0])
    if n < 0:
        _check(int(n))
    return torch.empty((max(n, 256),), dtype=torch.uint8, device=cache.k_codes.device)


def kv8_evict(cache: KV8Cache, table: torch.Tensor, lens: torch.Tensor, new_table: torch.Tensor, keep: int, *,
              recent: int = 0, sink: int = 0, max_len: int | None = None,
              workspace: torch.Tensor | None = None, stream=None):
    """Cut each sequence to at most `keep` tokens -- its first `sink`, its last
    `recent` and of the others those with the largest cache.weights -- and
    write them, in order, to the pages of new_table (int32 [seqs, new_cols],
    none of them a page of table).  Returns (new lens [seqs], kept positions
    [seqs, keep] padded with -1), int32.  workspace: a kv8_evict_workspace,
    for calls that overlap on several streams or are captured."""
    L = load_library()
    cc, _, page, _, dev = _ckv8(cache)
    cb, seqs = _ckv8_batch(table, lens, None, 0, None, max_len, page)
    if new_table.dtype != torch.int32 or new_table.dim() != 2 or new_table.shape[0] != seqs \
            or not new_table.is_contiguous():
        raise ValueError(f"new_table: expected a contiguous int32 [{seqs}, new_cols] tensor")
    keep, recent, sink = _i32(keep, "keep"), _i32(recent, "recent"), _i32(sink, "sink")
    if keep <= 0:
        raise ValueError(f"keep: {keep}, expected at least 1")
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
        raise ValueError("workspace: expected a contiguous uint8 tensor (kv8_evict_workspace)")
    _kv8_on(dev, table, lens, new_table, workspace)
    new_lens = _kv8_empty((seqs,), torch.int32, table.device, stream)
    kept = _kv8_empty((seqs, keep), torch.int32, table.device, stream)
    args = (cc, cb, new_table.data_ptr(), new_table.shape[1], keep, recent, sink, new_lens.data_ptr(),
            kept.data_ptr())
    if workspace is None:
        _check(L.kv8_evict(*args, _kv8_stream(stream, dev)))
    else:
        _check(L.kv8_evict_noalloc(*args, workspace.data_ptr(), workspace.numel(), _kv8_stream(stream, dev)))
    return new_lens, kept
