"""QLoRA linear layer for NVIDIA B200 (sm_100a).

A thin ctypes binding of ``libqlora.so`` (C ABI in ``include/qlora.h``).  The
functions below only marshal arguments: every step of quantisation,
dequantisation, forward and backward runs in the library's CUDA kernels.
PyTorch is used for device memory and streams.  There is no fallback: if the
library is missing or a call fails, a ``QLoRAError`` is raised.

Names follow the C ABI: ``nf4_quantize``, ``nf4_dequantize``,
``qlora_linear_fwd``, ``qlora_linear_bwd``; beside the linear layer, what else a
fine-tuning step runs: ``qlora_layer_norm_fwd`` / ``_bwd``,
``qlora_token_logprobs_fwd`` / ``_bwd``, ``qlora_adamw_step``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora.so")

QLORA_OK = 0
_STATUS = {0: "QLORA_OK", -1: "QLORA_ERR_INVALID_ARG", -2: "QLORA_ERR_UNSUPPORTED", -3: "QLORA_ERR_ALIGNMENT",
           -4: "QLORA_ERR_WORKSPACE", -5: "QLORA_ERR_CUDA", -6: "QLORA_ERR_DEVICE"}

EXPORTS = ("qlora_nf4_sizes", "nf4_quantize", "nf4_quantize_noalloc", "nf4_dequantize", "qlora_lora_merge",
           "qlora_rank_pad", "qlora_linear_workspace_size",
           "qlora_linear_fwd", "qlora_linear_bwd", "qlora_nf4_codebook", "qlora_device_status", "qlora_last_error",
           "qlora_profile_enable", "qlora_profile_read",
           "qlora_dropout_mask", "qlora_linear_dropout_workspace_size", "qlora_linear_fwd_dropout",
           "qlora_linear_bwd_dropout", "qlora_selftest_wait_timeout", "qlora_grouped_workspace_size",
           "qlora_linear_fwd_grouped", "qlora_linear_bwd_grouped",
           "qlora_layer_norm_fwd", "qlora_layer_norm_bwd", "qlora_layer_norm_workspace_size",
           "qlora_adamw_step", "qlora_adamw_state_values",
           "qlora_token_logprobs_fwd", "qlora_token_logprobs_bwd")

KERNEL_CLASSES = ("quant", "dq_const", "dequant", "fwd_gemm", "bwd_gemm", "lora_gemm", "aux")


class QLoRAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_STATUS.get(code, code)}: {msg}")
        self.code = code


class QloraNF4(ctypes.Structure):
    """Mirror of ``qlora_nf4_t``."""
    _fields_ = [("d", ctypes.c_int64), ("k", ctypes.c_int64), ("blocksize", ctypes.c_int32),
                ("double_quant", ctypes.c_int32), ("codes", ctypes.c_void_p), ("absmax", ctypes.c_void_p),
                ("c2", ctypes.c_void_p), ("c1", ctypes.c_void_p), ("mean", ctypes.c_void_p)]


MAX_GROUP = 4


class QloraNF4Group(ctypes.Structure):
    """Mirror of ``qlora_nf4_group_t``."""
    _fields_ = [("n", ctypes.c_int32), ("d", ctypes.c_int64 * MAX_GROUP), ("w", QloraNF4)]


class QloraDropout(ctypes.Structure):
    """Mirror of ``qlora_dropout_t``: adapter dropout probability p and the
    generator's (seed, offset)."""
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64)]


class QloraNorm(ctypes.Structure):
    """Mirror of ``qlora_norm_t``."""
    _fields_ = [("M", ctypes.c_int64), ("D", ctypes.c_int64), ("dtype", ctypes.c_int32), ("wdtype", ctypes.c_int32),
                ("rms", ctypes.c_int32), ("eps", ctypes.c_float)]


class QloraLogits(ctypes.Structure):
    """Mirror of ``qlora_logits_t``."""
    _fields_ = [("N", ctypes.c_int64), ("V", ctypes.c_int64), ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("top", ctypes.c_int32)]


class QloraAdamWTensor(ctypes.Structure):
    """Mirror of ``qlora_adamw_tensor_t``."""
    _fields_ = [("param", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class QloraAdamW(ctypes.Structure):
    """Mirror of ``qlora_adamw_t``."""
    _fields_ = [("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("state_bits", ctypes.c_int32),
                ("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64),
                ("grad_scale", ctypes.c_void_p), ("clock", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libqlora.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise QLoRAError(-5, f"{LIB_PATH} is missing; build it with `python -m bit_quantized_lora_02_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    c_i64, c_i32, c_sz, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p
    L.qlora_nf4_sizes.argtypes = [c_i64, c_i64, c_i32, c_i32, ctypes.POINTER(c_sz), ctypes.POINTER(c_sz)]
    L.nf4_quantize.argtypes = [vp, ctypes.POINTER(QloraNF4), vp, c_sz, vp]
    L.nf4_quantize_noalloc.argtypes = [vp, ctypes.POINTER(QloraNF4), vp]
    L.nf4_dequantize.argtypes = [ctypes.POINTER(QloraNF4), vp, vp]
    L.qlora_lora_merge.argtypes = [ctypes.POINTER(QloraNF4), vp, vp, c_i32, ctypes.c_float, vp, vp]
    L.qlora_rank_pad.argtypes = [c_i32]
    L.qlora_rank_pad.restype = c_i32
    L.qlora_linear_workspace_size.argtypes = [c_i64, c_i64, c_i64, c_i32, c_i32, ctypes.POINTER(c_sz)]
    L.qlora_linear_fwd.argtypes = [vp, c_i64, ctypes.POINTER(QloraNF4), vp, vp, c_i32, ctypes.c_float, vp, vp, vp,
                                   c_sz, vp]
    L.qlora_linear_bwd.argtypes = [vp, vp, c_i64, ctypes.POINTER(QloraNF4), vp, vp, c_i32, ctypes.c_float, vp, vp,
                                   vp, vp, vp, c_sz, vp]
    L.qlora_nf4_codebook.argtypes = [ctypes.POINTER(ctypes.c_float)]
    L.qlora_device_status.argtypes = [vp, ctypes.POINTER(c_i32)]
    L.qlora_dropout_mask.argtypes = [c_i64, c_i64, ctypes.POINTER(QloraDropout), vp, vp]
    L.qlora_linear_dropout_workspace_size.argtypes = [c_i64, c_i64, c_i64, c_i32, c_i32, ctypes.POINTER(c_sz)]
    L.qlora_linear_fwd_dropout.argtypes = [vp, c_i64, ctypes.POINTER(QloraNF4), vp, vp, c_i32, ctypes.c_float,
                                           ctypes.POINTER(QloraDropout), vp, vp, vp, c_sz, vp]
    L.qlora_linear_bwd_dropout.argtypes = [vp, vp, c_i64, ctypes.POINTER(QloraNF4), vp, vp, c_i32, ctypes.c_float,
                                           ctypes.POINTER(QloraDropout), vp, vp, vp, vp, vp, c_sz, vp]
    L.qlora_selftest_wait_timeout.argtypes = [ctypes.c_uint32, vp, vp]
    G = ctypes.POINTER(QloraNF4Group)
    L.qlora_grouped_workspace_size.argtypes = [c_i64, G, c_i32, c_i32, ctypes.POINTER(c_sz)]
    L.qlora_linear_fwd_grouped.argtypes = [vp, c_i64, G, vp, vp, c_i32, ctypes.c_float, vp, vp, vp, c_sz, vp]
    L.qlora_linear_bwd_grouped.argtypes = [vp, vp, c_i64, G, vp, vp, c_i32, ctypes.c_float, vp, vp, vp, vp, vp,
                                           c_sz, vp]
    NP = ctypes.POINTER(QloraNorm)
    L.qlora_layer_norm_fwd.argtypes = [NP, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.qlora_layer_norm_bwd.argtypes = [NP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, c_sz, vp]
    L.qlora_layer_norm_workspace_size.argtypes = [NP, c_i32, ctypes.POINTER(c_sz)]
    LP = ctypes.POINTER(QloraLogits)
    L.qlora_token_logprobs_fwd.argtypes = [LP, vp, vp, vp, vp, vp, vp, vp, vp]
    L.qlora_token_logprobs_bwd.argtypes = [LP, vp, vp, vp, vp, vp, vp, vp, c_i64, c_i64, vp]
    L.qlora_adamw_step.argtypes = [ctypes.POINTER(QloraAdamW), ctypes.POINTER(QloraAdamWTensor), c_i64, vp]
    L.qlora_adamw_state_values.argtypes = [c_i64, vp, vp, vp, vp, vp, vp, vp]
    L.qlora_last_error.restype = ctypes.c_char_p
    L.qlora_profile_enable.argtypes = [c_i32]
    L.qlora_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]
    for name in ("qlora_nf4_sizes", "nf4_quantize", "nf4_quantize_noalloc", "nf4_dequantize", "qlora_lora_merge",
                 "qlora_linear_workspace_size",
                 "qlora_linear_fwd", "qlora_linear_bwd", "qlora_nf4_codebook", "qlora_device_status",
                 "qlora_profile_enable", "qlora_profile_read", "qlora_dropout_mask",
                 "qlora_linear_dropout_workspace_size", "qlora_linear_fwd_dropout", "qlora_linear_bwd_dropout",
                 "qlora_selftest_wait_timeout", "qlora_grouped_workspace_size", "qlora_linear_fwd_grouped",
                 "qlora_linear_bwd_grouped", "qlora_layer_norm_fwd", "qlora_layer_norm_bwd",
                 "qlora_layer_norm_workspace_size", "qlora_adamw_step", "qlora_adamw_state_values",
                 "qlora_token_logprobs_fwd", "qlora_token_logprobs_bwd"):
        getattr(L, name).restype = c_i32
    _lib = L
    return L


def _check(rc: int) -> None:
    if rc != QLORA_OK:
        raise QLoRAError(rc, lib().qlora_last_error().decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _expect(t: Optional[torch.Tensor], name: str, shape, dtype, required: bool = True) -> None:
    """The C ABI sees raw pointers only: check dtype, exact shape and row-major
    contiguity here, so that a mismatched tensor raises instead of being read
    or written past its end."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(int(x) for x in shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")


def _same_device(dev, **tensors) -> None:
    """Every pointer of one call must live on the device the call runs on."""
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the call runs on {dev}")


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


# ---------------------------------------------------------------------------
# quantized weight container
# ---------------------------------------------------------------------------
@dataclass
class NF4Weight:
    """Device buffers of one quantized weight (layout of ``qlora_nf4_t``)."""
    d: int
    k: int
    double_quant: int          # 0: fp32 absmax; 1 (or True): Int8 c2; 2: FP8 E4M3 c2
    codes: torch.Tensor
    absmax: Optional[torch.Tensor] = None
    c2: Optional[torch.Tensor] = None
    c1: Optional[torch.Tensor] = None
    mean: Optional[torch.Tensor] = None
    blocksize: int = 64

    def struct(self, device=None) -> QloraNF4:
        """The C struct, after checking every buffer against the sizes the
        library needs for a d x k weight in this mode: dtype, byte size,
        contiguity and device (``device``: the activations' device, when the
        call has activations).  A short or misplaced buffer raises here instead
        of being read or written past its end."""
        mode = int(self.double_quant)
        if mode not in (0, 1, 2):
            raise ValueError(f"double_quant must be 0, 1 or 2, got {self.double_quant!r}")
        sizes, _ = qlora_nf4_sizes(self.d, self.k, self.blocksize, mode)
        dev = self.codes.device if device is None else torch.device(device)
        want = [("codes", self.codes, sizes[0], (torch.uint8,)),
                ("absmax", self.absmax, sizes[1], (torch.float32,)),
                ("c2", self.c2, sizes[2], (torch.uint8,) if mode == 2 else (torch.int8,)),
                ("c1", self.c1, sizes[3], (torch.float32,)),
                ("mean", self.mean, sizes[4], (torch.float32,))]
        for name, t, need, dtypes in want:
            if need == 0:
                continue
            if t is None:
                raise ValueError(f"NF4Weight.{name} is required for double_quant={mode}")
            if t.dtype not in dtypes:
                raise ValueError(f"NF4Weight.{name}: dtype {t.dtype}, expected {dtypes[0]}")
            if not t.is_contiguous():
                raise ValueError(f"NF4Weight.{name} must be contiguous")
            if t.device != dev:
                raise ValueError(f"NF4Weight.{name} is on {t.device}, the call runs on {dev}")
            if _nbytes(t) < need:
                raise ValueError(f"NF4Weight.{name}: {_nbytes(t)} bytes, a {self.d}x{self.k} weight needs {need}")
        return QloraNF4(self.d, self.k, self.blocksize, mode, _ptr(self.codes), _ptr(self.absmax),
                        _ptr(self.c2), _ptr(self.c1), _ptr(self.mean))

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.absmax, self.c2, self.c1, self.mean)
                   if t is not None)


def qlora_nf4_sizes(d: int, k: int, blocksize: int = 64, double_quant: bool = True):
    """(sizes of codes, absmax, c2, c1, mean in bytes, quantize workspace bytes)."""
    sizes = (ctypes.c_size_t * 5)()
    ws = ctypes.c_size_t()
    _check(lib().qlora_nf4_sizes(d, k, blocksize, int(double_quant), sizes, ctypes.byref(ws)))
    return list(sizes), ws.value


def nf4_alloc(d: int, k: int, double_quant: bool = True, device=None) -> NF4Weight:
    device = device or torch.device("cuda", torch.cuda.current_device())
    sizes, _ = qlora_nf4_sizes(d, k, 64, double_quant)

    def buf(n, dtype, esize):
        # 16 extra bytes of slack keep vector accesses inside the allocation
        return torch.empty(max(n // esize, 1) + 16 // esize, dtype=dtype, device=device)
    codes = buf(sizes[0], torch.uint8, 1)
    mode = int(double_quant)
    if mode:
        c2_dtype = torch.uint8 if mode == 2 else torch.int8   # E4M3 bytes / Int8
        return NF4Weight(d, k, mode, codes, None, buf(sizes[2], c2_dtype, 1), buf(sizes[3], torch.float32, 4),
                         buf(sizes[4], torch.float32, 4))
    return NF4Weight(d, k, 0, codes, buf(sizes[1], torch.float32, 4))


def nf4_quantize(W0: torch.Tensor, double_quant: bool = True, out: Optional[NF4Weight] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> NF4Weight:
    """Blockwise NF4 (+ double quantisation) of a bf16 (d, k) weight."""
    assert W0.dtype == torch.bfloat16 and W0.dim() == 2 and W0.is_contiguous()
    d, k = W0.shape
    q = out or nf4_alloc(d, k, double_quant, W0.device)
    if (q.d, q.k) != (d, k):
        raise ValueError(f"out describes a {q.d}x{q.k} weight, W0 is {d}x{k}")
    _, ws_bytes = qlora_nf4_sizes(d, k, 64, q.double_quant)
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=W0.device)
    if workspace is not None and workspace.device != W0.device:
        raise ValueError(f"workspace is on {workspace.device}, W0 on {W0.device}")
    st = q.struct(W0.device)
    _check(lib().nf4_quantize(W0.data_ptr(), ctypes.byref(st), _ptr(workspace), _nbytes(workspace),
                              _stream(stream)))
    return q


NOALLOC_MAX_WEIGHTS = 1 << 28


def nf4_quantize_noalloc(W0: torch.Tensor, double_quant: bool = True, out: Optional[NF4Weight] = None,
                         stream=None) -> NF4Weight:
    """nf4_quantize without a workspace: for callers that cannot allocate device
    memory, the library uses its own fixed scratch (weights up to 2^28 elements).
    Only `out`'s buffers are the caller's; pass them pre-allocated to allocate
    nothing in this call."""
    assert W0.dtype == torch.bfloat16 and W0.dim() == 2 and W0.is_contiguous()
    d, k = W0.shape
    q = out or nf4_alloc(d, k, double_quant, W0.device)
    if (q.d, q.k) != (d, k):
        raise ValueError(f"out describes a {q.d}x{q.k} weight, W0 is {d}x{k}")
    if int(q.double_quant) != int(double_quant):
        raise ValueError(f"out holds double_quant={int(q.double_quant)} buffers, the call asks for {int(double_quant)}")
    st = q.struct(W0.device)
    _check(lib().nf4_quantize_noalloc(W0.data_ptr(), ctypes.byref(st), _stream(stream)))
    return q


def nf4_dequantize(q: NF4Weight, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """doubleDequant into a bf16 (d, k) tensor."""
    if out is None:
        out = torch.empty(q.d, q.k, dtype=torch.bfloat16, device=q.codes.device)
    _expect(out, "out", (q.d, q.k), torch.bfloat16)
    st = q.struct(out.device)
    _check(lib().nf4_dequantize(ctypes.byref(st), out.data_ptr(), _stream(stream)))
    return out


def qlora_lora_merge(q: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """W_merged = BF16(W^ + (alpha/r) B A) as a bf16 (d, k) tensor."""
    r = A.shape[0]
    if out is None:
        out = torch.empty(q.d, q.k, dtype=torch.bfloat16, device=q.codes.device)
    _expect(A, "A", (r, q.k), torch.bfloat16)
    _expect(B, "B", (q.d, r), torch.bfloat16)
    _expect(out, "out", (q.d, q.k), torch.bfloat16)
    _same_device(out.device, A=A, B=B)
    st = q.struct(out.device)
    _check(lib().qlora_lora_merge(ctypes.byref(st), A.data_ptr(), B.data_ptr(), r, float(alpha), out.data_ptr(),
                                  _stream(stream)))
    return out


# ---------------------------------------------------------------------------
# grouped projections (several weights that share their input X)
# ---------------------------------------------------------------------------
@dataclass
class NF4Group:
    """Stacked NF4 buffers of n projections that share X (layout of
    ``qlora_nf4_group_t``): `w` describes all rows together and `parts[i]` is
    the slice of projection i (quantise W_i into it with nf4_quantize)."""
    ds: tuple
    w: NF4Weight
    parts: list

    def struct(self, device=None) -> QloraNF4Group:
        n = len(self.ds)
        st = QloraNF4Group()
        st.n = n
        for i in range(MAX_GROUP):
            st.d[i] = int(self.ds[i]) if i < n else 0
        st.w = self.w.struct(device)
        if self.w.double_quant and _nbytes(self.w.mean) < 4 * n:
            raise ValueError(f"the group's mean buffer holds {_nbytes(self.w.mean)} bytes, {n} means need {4 * n}")
        return st


def nf4_alloc_group(ds, k: int, double_quant: bool = True, device=None) -> NF4Group:
    """Stacked buffers for projections of ds[i] x k rows (ds[i] % 256 == 0 for
    all but the last) and per-projection slice descriptors."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    ds = tuple(int(x) for x in ds)
    if not 1 <= len(ds) <= MAX_GROUP:
        raise ValueError(f"1..{MAX_GROUP} projections, got {len(ds)}")
    if any(x % 256 for x in ds[:-1]):
        raise ValueError("every projection but the last needs a multiple of 256 rows")
    mode = int(double_quant)
    per = [qlora_nf4_sizes(d, k, 64, mode)[0] for d in ds]
    tot = [sum(sz[j] for sz in per) for j in range(5)]

    def buf(nbytes, dtype, esize):
        return torch.empty(max(nbytes // esize, 1) + 16 // esize, dtype=dtype, device=device)
    codes = buf(tot[0], torch.uint8, 1)
    c2_dtype = torch.uint8 if mode == 2 else torch.int8
    absmax = buf(tot[1], torch.float32, 4) if not mode else None
    c2 = buf(tot[2], c2_dtype, 1) if mode else None
    c1 = buf(tot[3], torch.float32, 4) if mode else None
    mean = buf(4 * len(ds), torch.float32, 4) if mode else None
    w = NF4Weight(sum(ds), k, mode, codes, absmax, c2, c1, mean)
    parts, off = [], [0] * 5
    for i, (d, sz) in enumerate(zip(ds, per)):
        def sl(t, j, esize):
            return None if t is None else t[off[j] // esize: (off[j] + sz[j]) // esize]
        parts.append(NF4Weight(d, k, mode, sl(codes, 0, 1), sl(absmax, 1, 4), sl(c2, 2, 1), sl(c1, 3, 4),
                               None if mean is None else mean[i:i + 1]))
        off = [o + x for o, x in zip(off, sz)]
    return NF4Group(ds, w, parts)


def nf4_quantize_group(Ws, double_quant: bool = True, out: Optional[NF4Group] = None, stream=None) -> NF4Group:
    """Quantise each W_i (d_i x k bf16) on its own into the group's stacked buffers."""
    k = Ws[0].shape[1]
    g = out or nf4_alloc_group([W.shape[0] for W in Ws], k, double_quant, Ws[0].device)
    for W, part in zip(Ws, g.parts):
        nf4_quantize(W, double_quant=part.double_quant, out=part, stream=stream)
    return g


def qlora_grouped_workspace_size(M: int, g: NF4Group, r: int, backward: bool) -> int:
    n = ctypes.c_size_t()
    st = g.struct()
    _check(lib().qlora_grouped_workspace_size(M, ctypes.byref(st), r, int(backward), ctypes.byref(n)))
    return n.value


def qlora_linear_fwd_grouped(X: torch.Tensor, g: NF4Group, A: torch.Tensor, B: torch.Tensor, alpha: float,
                             r: Optional[int] = None, Y: Optional[torch.Tensor] = None,
                             T_save: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                             stream=None, save_T: bool = True):
    """Y = [Y_0 | Y_1 | ...], Y_i = X W_i^T + (alpha/r) (X A_i^T) B_i^T with
    A = stacked A_i ((n r) x k) and B = stacked B_i (sum d_i x r)."""
    n = len(g.ds)
    M, k = X.shape
    r = A.shape[0] // n if r is None else r
    dev = X.device
    dt = g.w.d
    if Y is None:
        Y = torch.empty(M, dt, dtype=torch.bfloat16, device=dev)
    if T_save is None and save_T:
        T_save = torch.empty(M, qlora_rank_pad(n * r), dtype=torch.bfloat16, device=dev)
    _expect(X, "X", (M, g.w.k), torch.bfloat16)
    _expect(A, "A", (n * r, g.w.k), torch.bfloat16)
    _expect(B, "B", (dt, r), torch.bfloat16)
    _expect(Y, "Y", (M, dt), torch.bfloat16)
    _expect(T_save, "T_save", (M, qlora_rank_pad(n * r)), torch.bfloat16, required=False)
    if workspace is None:
        nws = qlora_grouped_workspace_size(M, g, r, False)
        workspace = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev) if nws else None
    _same_device(dev, A=A, B=B, Y=Y, T_save=T_save, workspace=workspace)
    st = g.struct(dev)
    _check(lib().qlora_linear_fwd_grouped(X.data_ptr(), M, ctypes.byref(st), A.data_ptr(), B.data_ptr(), r,
                                          float(alpha), Y.data_ptr(), _ptr(T_save), _ptr(workspace),
                                          _nbytes(workspace), _stream(stream)))
    return Y, T_save


def qlora_linear_bwd_grouped(dY: torch.Tensor, X: torch.Tensor, g: NF4Group, A: torch.Tensor, B: torch.Tensor,
                             alpha: float, r: Optional[int] = None, T_save: Optional[torch.Tensor] = None,
                             dX: Optional[torch.Tensor] = None, dA: Optional[torch.Tensor] = None,
                             dB: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                             stream=None, need_dX: bool = True):
    """Backward of qlora_linear_fwd_grouped; returns (dX, dA stacked, dB stacked)."""
    n = len(g.ds)
    M = dY.shape[0]
    r = A.shape[0] // n if r is None else r
    dev = dY.device
    dt = g.w.d
    if dX is None and need_dX:
        dX = torch.empty(M, g.w.k, dtype=torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty(n * r, g.w.k, dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty(dt, r, dtype=torch.float32, device=dev)
    _expect(dY, "dY", (M, dt), torch.bfloat16)
    _expect(X, "X", (M, g.w.k), torch.bfloat16)
    _expect(A, "A", (n * r, g.w.k), torch.bfloat16)
    _expect(B, "B", (dt, r), torch.bfloat16)
    _expect(T_save, "T_save", (M, qlora_rank_pad(n * r)), torch.bfloat16, required=False)
    _expect(dX, "dX", (M, g.w.k), torch.bfloat16, required=False)
    _expect(dA, "dA", (n * r, g.w.k), torch.float32)
    _expect(dB, "dB", (dt, r), torch.float32)
    if workspace is None:
        nws = qlora_grouped_workspace_size(M, g, r, True)
        workspace = torch.empty(max(nws, 16), dtype=torch.uint8, device=dev) if nws else None
    _same_device(dev, X=X, A=A, B=B, T_save=T_save, dX=dX, dA=dA, dB=dB, workspace=workspace)
    st = g.struct(dev)
    _check(lib().qlora_linear_bwd_grouped(_ptr(dY), _ptr(X), M, ctypes.byref(st), A.data_ptr(), B.data_ptr(), r,
                                          float(alpha), _ptr(T_save), _ptr(dX), dA.data_ptr(), dB.data_ptr(),
                                          _ptr(workspace), _nbytes(workspace), _stream(stream)))
    return dX, dA, dB


def qlora_rank_pad(r: int) -> int:
    return int(lib().qlora_rank_pad(r))


def qlora_linear_workspace_size(M: int, d: int, k: int, r: int, backward: bool) -> int:
    n = ctypes.c_size_t()
    _check(lib().qlora_linear_workspace_size(M, d, k, r, int(backward), ctypes.byref(n)))
    return n.value


def _dropout_struct(dropout) -> Optional[QloraDropout]:
    """(p, seed, offset) -> qlora_dropout_t, or None for no dropout."""
    if dropout is None:
        return None
    p, seed, offset = dropout
    if not (0.0 <= float(p) < 1.0):
        raise ValueError(f"dropout probability {p} outside [0, 1)")
    return QloraDropout(float(p), int(seed) & (2 ** 64 - 1), int(offset) & (2 ** 64 - 1))


def qlora_linear_dropout_workspace_size(M: int, d: int, k: int, r: int, backward: bool) -> int:
    n = ctypes.c_size_t()
    _check(lib().qlora_linear_dropout_workspace_size(M, d, k, r, int(backward), ctypes.byref(n)))
    return n.value


def qlora_dropout_mask(M: int, k: int, p: float, seed: int, offset: int = 0, out: Optional[torch.Tensor] = None,
                       device=None, stream=None) -> torch.Tensor:
    """Keep bitmask of an M x k activation as int32 words (bit b of word w is
    flat element 32 w + b; 1 = kept)."""
    nw = (M * k + 31) // 32
    if out is None:
        device = device or torch.device("cuda", torch.cuda.current_device())
        out = torch.empty(max(nw, 1), dtype=torch.int32, device=device)
    if out.dtype != torch.int32 or out.numel() < nw or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous int32 tensor of at least {nw} words")
    st = _dropout_struct((p, seed, offset))
    _check(lib().qlora_dropout_mask(M, k, ctypes.byref(st), out.data_ptr() if nw else None, _stream(stream)))
    return out


def qlora_linear_fwd_dropout(X: torch.Tensor, q: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float,
                             dropout, **kw):
    """qlora_linear_fwd with adapter dropout; dropout = (p, seed, offset)."""
    return qlora_linear_fwd(X, q, A, B, alpha, dropout=dropout, **kw)


def qlora_linear_bwd_dropout(dY: torch.Tensor, X: torch.Tensor, q: NF4Weight, A: torch.Tensor, B: torch.Tensor,
                             alpha: float, dropout, **kw):
    """qlora_linear_bwd for the dropout forward with the same (p, seed, offset)."""
    return qlora_linear_bwd(dY, X, q, A, B, alpha, dropout=dropout, **kw)


def qlora_linear_fwd(X: torch.Tensor, q: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float,
                     Y: Optional[torch.Tensor] = None, T_save: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None, save_T: bool = True, dropout=None):
    """Y = X W^T + (alpha/r) (X A^T) B^T.  Returns (Y, T_save).  With
    dropout = (p, seed, offset) the adapter sees drop(X) instead of X."""
    M, k = X.shape
    r = A.shape[0]
    dev = X.device
    if Y is None:
        Y = torch.empty(M, q.d, dtype=torch.bfloat16, device=dev)
    if T_save is None and save_T:
        T_save = torch.empty(M, qlora_rank_pad(r), dtype=torch.bfloat16, device=dev)
    _expect(X, "X", (M, q.k), torch.bfloat16)
    _expect(A, "A", (r, q.k), torch.bfloat16)
    _expect(B, "B", (q.d, r), torch.bfloat16)
    _expect(Y, "Y", (M, q.d), torch.bfloat16)
    _expect(T_save, "T_save", (M, qlora_rank_pad(r)), torch.bfloat16, required=False)
    drop = _dropout_struct(dropout)
    if workspace is None:
        n = (qlora_linear_dropout_workspace_size(M, q.d, q.k, r, False) if drop is not None
             else qlora_linear_workspace_size(M, q.d, q.k, r, False))
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev) if n else None
    _same_device(dev, A=A, B=B, Y=Y, T_save=T_save, workspace=workspace)
    st = q.struct(dev)
    if drop is None:
        _check(lib().qlora_linear_fwd(X.data_ptr(), M, ctypes.byref(st), A.data_ptr(), B.data_ptr(), r, float(alpha),
                                      Y.data_ptr(), _ptr(T_save), _ptr(workspace), _nbytes(workspace),
                                      _stream(stream)))
    else:
        _check(lib().qlora_linear_fwd_dropout(X.data_ptr(), M, ctypes.byref(st), A.data_ptr(), B.data_ptr(), r,
                                              float(alpha), ctypes.byref(drop), Y.data_ptr(), _ptr(T_save),
                                              _ptr(workspace), _nbytes(workspace), _stream(stream)))
    return Y, T_save


def qlora_linear_bwd(dY: torch.Tensor, X: torch.Tensor, q: NF4Weight, A: torch.Tensor, B: torch.Tensor,
                     alpha: float, T_save: Optional[torch.Tensor] = None, dX: Optional[torch.Tensor] = None,
                     dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None, need_dX: bool = True, dropout=None):
    """Gradients for the adapters and the input; returns (dX, dA, dB).  With
    dropout = (p, seed, offset), the backward of the dropout forward."""
    M = dY.shape[0]
    r = A.shape[0]
    dev = dY.device
    if dX is None and need_dX:
        dX = torch.empty(M, q.k, dtype=torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty(r, q.k, dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty(q.d, r, dtype=torch.float32, device=dev)
    _expect(dY, "dY", (M, q.d), torch.bfloat16)
    _expect(X, "X", (M, q.k), torch.bfloat16)
    _expect(A, "A", (r, q.k), torch.bfloat16)
    _expect(B, "B", (q.d, r), torch.bfloat16)
    _expect(T_save, "T_save", (M, qlora_rank_pad(r)), torch.bfloat16, required=False)
    _expect(dX, "dX", (M, q.k), torch.bfloat16, required=False)
    _expect(dA, "dA", (r, q.k), torch.float32)
    _expect(dB, "dB", (q.d, r), torch.float32)
    drop = _dropout_struct(dropout)
    if workspace is None:
        n = (qlora_linear_dropout_workspace_size(M, q.d, q.k, r, True) if drop is not None
             else qlora_linear_workspace_size(M, q.d, q.k, r, True))
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev) if n else None
    _same_device(dev, X=X, A=A, B=B, T_save=T_save, dX=dX, dA=dA, dB=dB, workspace=workspace)
    st = q.struct(dev)
    if drop is None:
        _check(lib().qlora_linear_bwd(_ptr(dY), _ptr(X), M, ctypes.byref(st), A.data_ptr(), B.data_ptr(), r,
                                      float(alpha), _ptr(T_save), _ptr(dX), dA.data_ptr(), dB.data_ptr(),
                                      _ptr(workspace), _nbytes(workspace), _stream(stream)))
    else:
        _check(lib().qlora_linear_bwd_dropout(_ptr(dY), _ptr(X), M, ctypes.byref(st), A.data_ptr(), B.data_ptr(),
                                              r, float(alpha), ctypes.byref(drop), _ptr(T_save), _ptr(dX),
                                              dA.data_ptr(), dB.data_ptr(), _ptr(workspace), _nbytes(workspace),
                                              _stream(stream)))
    return dX, dA, dB


# ---------------------------------------------------------------------------
# the operators around the linear layer in a fine-tuning step
# ---------------------------------------------------------------------------
_DT = {torch.bfloat16: 0, torch.float32: 1}     # QLORA_DT_*


def _dt(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _DT:
        raise ValueError(f"{name}: dtype {t.dtype}, expected torch.bfloat16 or torch.float32")
    return _DT[t.dtype]


def _on_cuda(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device, is on {t.device}")
    return t.device


_NO_CONTEXT = contextlib.nullcontext()
# the raw handle of a device's current stream, without building a Stream object where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _enter(dev: int, stream):
    """(raw stream, context for the call's own allocations): the current stream
    of the tensors' device, or the caller's stream, which then also owns what
    the call allocates."""
    if stream is None:
        return _raw_stream(dev), _NO_CONTEXT
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the call runs on cuda:{dev}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _want(t: Optional[torch.Tensor], name: str, shape, dtype, dev: int) -> Optional[int]:
    """The address of an argument that must have this shape and dtype, be
    contiguous and live on CUDA device ``dev`` (-1: the host); None for an
    absent one."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _expect(t, name, shape, dtype)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call runs on {'cpu' if dev < 0 else f'cuda:{dev}'}")
    return t.data_ptr()


@functools.lru_cache(maxsize=256)
def _norm_desc(M: int, D: int, dt: int, wdt: int, rms: bool, eps: float):
    return ctypes.byref(QloraNorm(M, D, dt, wdt, rms, eps))


def _norm_struct(X: torch.Tensor, weight: torch.Tensor, name: str, rms: bool, eps: float):
    if X.dim() != 2:
        raise ValueError(f"{name}: shape {tuple(X.shape)}, expected (rows, values)")
    M, D = X.shape
    return _norm_desc(M, D, _dt(X, name), _dt(weight, "weight"), bool(rms), float(eps))


def qlora_layer_norm_fwd(X: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                         residual: Optional[torch.Tensor] = None, eps: float = 1e-5, rms: bool = False,
                         Y: Optional[torch.Tensor] = None, S: Optional[torch.Tensor] = None,
                         mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None, stream=None):
    """S = X + residual; Y = (S - mean) rstd weight + bias over each row of a
    bf16 or fp32 (M, D) tensor (rms: no mean is subtracted).  Returns
    (Y, S, mean, rstd) for qlora_layer_norm_bwd; S is X without a residual and
    mean is None for rms.  Y and S may be X or residual (in place); where Y is X
    and there is no residual, nothing holds S any more, and None is returned."""
    n = _norm_struct(X, weight, "X", rms, eps)
    shape, dtype, dev, f32 = X.shape, X.dtype, X.get_device(), torch.float32
    M, D = shape
    if S is not None and residual is None:
        raise ValueError("S goes with residual")
    if mean is not None and rms:
        raise ValueError("mean is not used with rms")
    pX = _want(X, "X", shape, dtype, dev)
    pR = _want(residual, "residual", shape, dtype, dev)
    pw = _want(weight, "weight", (D,), weight.dtype, dev)
    pb = _want(bias, "bias", (D,), weight.dtype, dev)
    pY, pS = _want(Y, "Y", shape, dtype, dev), _want(S, "S", shape, dtype, dev)
    pm, pr = _want(mean, "mean", (M,), f32, dev), _want(rstd, "rstd", (M,), f32, dev)
    _on_cuda(X, "X")
    raw, own = _enter(dev, stream)
    with own:
        if Y is None:
            Y = torch.empty_like(X)
            pY = Y.data_ptr()
        if S is None and residual is not None:
            S = torch.empty_like(X)
            pS = S.data_ptr()
        if mean is None and not rms:
            mean = torch.empty(M, dtype=f32, device=X.device)
            pm = mean.data_ptr()
        if rstd is None:
            rstd = torch.empty(M, dtype=f32, device=X.device)
            pr = rstd.data_ptr()
    _check(lib().qlora_layer_norm_fwd(n, pX, pR, pw, pb, pS, pY, pm, pr, raw))
    if S is None and (pY != pX or M == 0):
        S = X
    return Y, S, mean, rstd


@functools.lru_cache(maxsize=256)
def _norm_workspace(M: int, D: int, dt: int, with_dbias: bool, dev: int) -> int:
    size = ctypes.c_size_t()
    # the size goes by the SM count of the current device
    with _NO_CONTEXT if dev < 0 or dev == torch.cuda.current_device() else torch.cuda.device(dev):
        _check(lib().qlora_layer_norm_workspace_size(_norm_desc(M, D, dt, 1, False, 0.0), int(with_dbias),
                                                     ctypes.byref(size)))
    return size.value


def qlora_layer_norm_workspace_size(M: int, D: int, dtype=torch.bfloat16, with_dbias: bool = False) -> int:
    """Bytes of the backward pass's workspace on the current device."""
    if dtype not in _DT:
        raise ValueError(f"dtype {dtype}, expected torch.bfloat16 or torch.float32")
    return _norm_workspace(M, D, _DT[dtype], bool(with_dbias), torch.cuda.current_device() if torch.cuda.is_available() else -1)


def qlora_layer_norm_bwd(dY: torch.Tensor, S: torch.Tensor, weight: torch.Tensor, mean: Optional[torch.Tensor],
                         rstd: torch.Tensor, dS: Optional[torch.Tensor] = None, rms: bool = False,
                         dX: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                         dbias: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         stream=None, need_dbias: bool = False):
    """Backward of qlora_layer_norm_fwd; returns (dX, dweight, dbias).  dX is
    the gradient of X and of the residual alike; dS is the gradient that
    reaches S along the residual stream.  dweight and dbias are fp32; dbias is
    computed with need_dbias or where a tensor for it is given."""
    if S is None:
        raise ValueError("S is required (a forward pass with Y = X and no residual overwrites it)")
    n = _norm_struct(S, weight, "S", rms, 0.0)
    shape, dtype, dev, f32 = S.shape, S.dtype, S.get_device(), torch.float32
    M, D = shape
    if rstd is None or (mean is None and not rms):
        raise ValueError("mean is required" if rstd is not None else "rstd is required")
    pdY, pS = _want(dY, "dY", shape, dtype, dev), _want(S, "S", shape, dtype, dev)
    pw = _want(weight, "weight", (D,), weight.dtype, dev)
    pm, pr = None if rms else _want(mean, "mean", (M,), f32, dev), _want(rstd, "rstd", (M,), f32, dev)
    pdS, pdX = _want(dS, "dS", shape, dtype, dev), _want(dX, "dX", shape, dtype, dev)
    pdw, pdb = _want(dweight, "dweight", (D,), f32, dev), _want(dbias, "dbias", (D,), f32, dev)
    _on_cuda(S, "S")
    if workspace is not None:
        _same_device(S.device, workspace=workspace)
    raw, own = _enter(dev, stream)
    with own:
        if dX is None:
            dX = torch.empty_like(S)
            pdX = dX.data_ptr()
        if dweight is None:
            dweight = torch.empty(D, dtype=f32, device=S.device)
            pdw = dweight.data_ptr()
        if dbias is None and need_dbias:
            dbias = torch.empty(D, dtype=f32, device=S.device)
            pdb = dbias.data_ptr()
        if workspace is None:
            nws = _norm_workspace(M, D, _DT[dtype], dbias is not None, dev)
            workspace = torch.empty(max(nws, 16), dtype=torch.uint8, device=S.device)
    _check(lib().qlora_layer_norm_bwd(n, pdY, pS, pw, pm, pr, pdS, pdX, pdw, pdb, workspace.data_ptr(),
                                      _nbytes(workspace), raw))
    return dX, dweight, dbias


@dataclass
class TokenLogprobs:
    """Results of qlora_token_logprobs_fwd: fp32 (N,) tensors, and (N, top)
    int32 indices and fp32 log probabilities of the largest logits."""
    logp: Optional[torch.Tensor]
    lse: torch.Tensor
    entropy: Optional[torch.Tensor] = None
    top_ids: Optional[torch.Tensor] = None
    top_logp: Optional[torch.Tensor] = None


@functools.lru_cache(maxsize=256)
def _logits_desc(N: int, V: int, ld: int, dt: int, top: int):
    return ctypes.byref(QloraLogits(N, V, ld, dt, top))


def _logits_struct(logits: torch.Tensor, vocab: Optional[int], top: int):
    """Rows may lie further apart than they are long; the values of a row are
    neighbours."""
    if logits.dim() != 2:
        raise ValueError(f"logits: shape {tuple(logits.shape)}, expected (tokens, vocabulary)")
    N, cols = logits.shape
    V = cols if vocab is None else int(vocab)
    if not 0 < V <= cols:
        raise ValueError(f"vocab={V} with {cols} columns of logits")
    sr, sc = logits.stride()
    if cols > 1 and sc != 1 or N > 1 and sr < cols:
        raise ValueError(f"logits: strides {(sr, sc)}, expected rows of neighbouring values that do not overlap")
    return _logits_desc(N, V, sr if N > 1 else cols, _dt(logits, "logits"), int(top))


def qlora_token_logprobs_fwd(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, vocab: Optional[int] = None,
                             top: int = 0, entropy: bool = False, out: Optional[TokenLogprobs] = None,
                             stream=None) -> TokenLogprobs:
    """Log probabilities of the given tokens (int64; a target outside
    [0, vocab) does not count and gives 0) from bf16 or fp32 logits of shape
    (tokens, columns), the first `vocab` columns of which count; with the
    entropy of every row and its `top` (up to 32) most probable tokens, equal
    logits by ascending index.  `out`: tensors of an earlier call to write to."""
    if not 0 <= top <= 32:
        raise ValueError(f"top={top}, expected 0 to 32")
    l = _logits_struct(logits, vocab, top)
    N, dev, f32 = logits.shape[0], logits.get_device(), torch.float32
    pt = _want(targets, "targets", (N,), torch.int64, dev)
    if out is not None:
        have = (out.logp is not None, out.entropy is not None, out.top_ids is not None, out.top_logp is not None)
        if have != (targets is not None, bool(entropy), top > 0, top > 0) or out.lse is None:
            raise ValueError("out holds other results than the call asks for")
        _want(out.logp, "out.logp", (N,), f32, dev), _want(out.lse, "out.lse", (N,), f32, dev)
        _want(out.entropy, "out.entropy", (N,), f32, dev)
        _want(out.top_ids, "out.top_ids", (N, top), torch.int32, dev)
        _want(out.top_logp, "out.top_logp", (N, top), f32, dev)
    _on_cuda(logits, "logits")
    raw, own = _enter(dev, stream)
    if out is None:
        on = logits.device
        with own:
            out = TokenLogprobs(torch.empty(N, dtype=f32, device=on) if targets is not None else None,
                                torch.empty(N, dtype=f32, device=on),
                                torch.empty(N, dtype=f32, device=on) if entropy else None,
                                torch.empty(N, top, dtype=torch.int32, device=on) if top > 0 else None,
                                torch.empty(N, top, dtype=f32, device=on) if top > 0 else None)
    _check(lib().qlora_token_logprobs_fwd(l, logits.data_ptr(), pt, _ptr(out.logp), out.lse.data_ptr(),
                                          _ptr(out.entropy), _ptr(out.top_ids), _ptr(out.top_logp), raw))
    return out


def qlora_token_logprobs_bwd(logits: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor, dlogp: torch.Tensor,
                             entropy: Optional[torch.Tensor] = None, dentropy: Optional[torch.Tensor] = None,
                             vocab: Optional[int] = None, dlogits: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """Gradient of the logits from the gradients of qlora_token_logprobs_fwd's
    logp and (with its entropy) entropy.  Columns from `vocab` on get zeros.
    `dlogits` may be the logits themselves (in place).  Padded logits are best
    passed whole, with `vocab`: a slice of their columns has rows that start at
    other offsets than those of a new gradient tensor, which is then written value
    by value."""
    l = _logits_struct(logits, vocab, 0)
    (N, cols), dev, f32 = logits.shape, logits.get_device(), torch.float32
    for t, name in ((targets, "targets"), (lse, "lse"), (dlogp, "dlogp")):
        if t is None:
            raise ValueError(f"{name} is required")
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs entropy")
    pt, pl = _want(targets, "targets", (N,), torch.int64, dev), _want(lse, "lse", (N,), f32, dev)
    pd = _want(dlogp, "dlogp", (N,), f32, dev)
    pe, ph = _want(entropy, "entropy", (N,), f32, dev), _want(dentropy, "dentropy", (N,), f32, dev)
    if dlogits is not None:
        if dlogits.dtype != logits.dtype or dlogits.shape != logits.shape or dlogits.get_device() != dev:
            raise ValueError("dlogits must have the logits' shape, dtype and device")
        _logits_struct(dlogits, vocab, 0)
    _on_cuda(logits, "logits")
    raw, own = _enter(dev, stream)
    if dlogits is None:
        with own:
            dlogits = torch.empty(N, cols, dtype=logits.dtype, device=logits.device)
    _check(lib().qlora_token_logprobs_bwd(l, logits.data_ptr(), pt, pl, pd, pe, ph, dlogits.data_ptr(),
                                          cols, dlogits.stride(0) if N > 1 else cols, raw))
    return dlogits


ADAMW_BLOCK = 256       # values that share one scale of an 8-bit state


@dataclass
class AdamWState:
    """The tensors of qlora_adamw_step and their moments.  The moments of all
    tensors lie in flat buffers, each tensor's from a multiple of 256 values on
    (`starts`): m and v fp32, or m E4M3 and v uint8 codes with one fp32 scale per
    block of 256.  All zeros is the state before the first step.  The addresses
    of `params`, `grads` and `copies` are read once: the tensors have to stay
    where they are (use `set_grads` for other gradient tensors)."""
    params: list
    grads: list
    copies: Optional[list]
    state_bits: int
    starts: list
    m: torch.Tensor
    v: torch.Tensor
    m_scale: Optional[torch.Tensor]
    v_scale: Optional[torch.Tensor]
    array: object              # qlora_adamw_tensor_t[len(params)]
    device: torch.device

    def set_grads(self, grads) -> None:
        """Take the gradients from these tensors from now on."""
        grads = _adamw_tensors(grads, "grads", self.params, self.device)
        _dt(grads[0], "grads")
        self.grads = grads
        for t, g in zip(self.array, grads):
            t.grad = g.data_ptr()


def _adamw_tensors(ts, name: str, params, dev) -> list:
    ts = list(ts)
    if len(ts) != len(params):
        raise ValueError(f"{name}: {len(ts)} tensors for {len(params)} parameters")
    for i, (t, p) in enumerate(zip(ts, params)):
        _expect(t, f"{name}[{i}]", p.shape, ts[0].dtype)
        if t.device != dev:
            raise ValueError(f"{name}[{i}] is on {t.device}, the parameters on {dev}")
    return ts


def qlora_adamw_alloc(params, grads, state_bits: int = 32, copies=None) -> AdamWState:
    """State for AdamW over many tensors: params (all bf16 or all fp32), their
    gradients (all bf16 or all fp32, the same shapes) and, beside fp32 params,
    bf16 copies that every step writes (the adapters as the linear layer reads
    them).  state_bits: 32, or 8 for block-wise 8-bit moments."""
    params = list(params)
    if state_bits not in (8, 32):
        raise ValueError(f"state_bits must be 8 or 32, got {state_bits!r}")
    if not params:
        raise ValueError("no parameters")
    dev = params[0].device
    params = _adamw_tensors(params, "params", params, dev)
    _dt(params[0], "params")
    grads = _adamw_tensors(grads, "grads", params, dev)
    _dt(grads[0], "grads")
    if copies is not None:
        copies = _adamw_tensors(copies, "copies", params, dev)
        if params[0].dtype != torch.float32 or copies[0].dtype != torch.bfloat16:
            raise ValueError("copies are bf16, beside fp32 parameters")
    spans = sorted((t.data_ptr(), t.data_ptr() + _nbytes(t)) for t in params + (copies or []) if t.numel())
    if any(b[0] < a[1] for a, b in zip(spans, spans[1:])):
        raise ValueError("two parameters (or copies) overlap")
    _on_cuda(params[0], "params")
    starts, at = [], 0
    for p in params:
        starts.append(at)
        at += -(-p.numel() // ADAMW_BLOCK) * ADAMW_BLOCK
    eight = state_bits == 8
    m = torch.zeros(at, dtype=torch.uint8 if eight else torch.float32, device=dev)
    v = torch.zeros_like(m)
    ms = torch.zeros(at // ADAMW_BLOCK, dtype=torch.float32, device=dev) if eight else None
    vs = torch.zeros_like(ms) if eight else None
    if eight:
        m = m.view(torch.float8_e4m3fn)
    array = (QloraAdamWTensor * len(params))()
    for i, (t, p, g, o) in enumerate(zip(array, params, grads, starts)):
        t.param, t.grad, t.n = p.data_ptr(), g.data_ptr(), p.numel()
        t.copy = copies[i].data_ptr() if copies is not None else None
        t.m, t.v = m.data_ptr() + o * m.element_size(), v.data_ptr() + o * v.element_size()
        if eight:
            t.m_scale, t.v_scale = ms.data_ptr() + o // ADAMW_BLOCK * 4, vs.data_ptr() + o // ADAMW_BLOCK * 4
    return AdamWState(params, grads, copies, state_bits, starts, m, v, ms, vs, array, dev)


def qlora_adamw_clock(lr: float, step: int = 0, device=None) -> torch.Tensor:
    """Learning rate (element 0) and steps taken so far (element 1) in device
    memory, for steps that a captured graph replays."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    return torch.tensor([float(lr), float(step), 0, 0, 0, 0, 0, 0], dtype=torch.float64, device=device)


def qlora_adamw_step(state: AdamWState, step: Optional[int] = None, lr: Optional[float] = None, betas=(0.9, 0.999),
                     eps: float = 1e-8, weight_decay: float = 0.0, grad_scale: Optional[torch.Tensor] = None,
                     clock: Optional[torch.Tensor] = None, stream=None) -> None:
    """One AdamW step, in place.  `step` counts from 1; a clock (see
    qlora_adamw_clock) takes the place of `step` and `lr`.  grad_scale: one fp32
    value on the device that multiplies every gradient."""
    dev = state.device.index
    if (clock is None) == (step is None or lr is None) or (clock is not None and (step is not None or lr is not None)):
        raise ValueError("either step and lr, or a clock")
    scale = _want(grad_scale, "grad_scale", (1,), torch.float32, dev) if grad_scale is not None else None
    tick = _want(clock, "clock", (8,), torch.float64, dev) if clock is not None else None
    o = QloraAdamW(_DT[state.params[0].dtype], _DT[state.grads[0].dtype], state.state_bits, float(lr or 0.0),
                   float(betas[0]), float(betas[1]), float(eps), float(weight_decay), int(step or 0), scale, tick)
    raw, _ = _enter(dev, stream)
    _check(lib().qlora_adamw_step(ctypes.byref(o), state.array, len(state.params), raw))


def qlora_adamw_state(state: AdamWState, m: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                      stream=None):
    """The moments as flat fp32 tensors (m, v), laid out as state.starts says:
    the state's own with 32 bits, the values that the codes stand for with 8."""
    if state.state_bits == 32:
        if m is not None or v is not None:
            raise ValueError("32-bit moments are not copied: use the returned tensors")
        return state.m, state.v
    n, dev = state.m.numel(), state.device.index
    pm, pv = _want(m, "m", (n,), torch.float32, dev), _want(v, "v", (n,), torch.float32, dev)
    raw, own = _enter(dev, stream)
    with own:
        if m is None:
            m = torch.empty(n, dtype=torch.float32, device=state.device)
            pm = m.data_ptr()
        if v is None:
            v = torch.empty(n, dtype=torch.float32, device=state.device)
            pv = v.data_ptr()
    _check(lib().qlora_adamw_state_values(n, state.m.data_ptr(), state.m_scale.data_ptr(), state.v.data_ptr(),
                                          state.v_scale.data_ptr(), pm, pv, raw))
    return m, v


def qlora_nf4_codebook():
    buf = (ctypes.c_float * 16)()
    _check(lib().qlora_nf4_codebook(buf))
    return list(buf)


def qlora_device_status(stream=None) -> int:
    """Synchronize and return (and clear) the device status word; 0 = clean."""
    s = ctypes.c_int32()
    rc = lib().qlora_device_status(_stream(stream), ctypes.byref(s))
    if rc not in (QLORA_OK, -6):
        _check(rc)
    return s.value


def qlora_selftest_wait_timeout(limit_us: int = 1000, stream=None) -> int:
    """Run the bounded-wait self-test (a wait nothing ends, given up after
    limit_us); returns the kernel's result word (2: gave up and released its
    TMEM).  The status word then holds code 7 until qlora_device_status()."""
    res = torch.zeros(1, dtype=torch.int32, device=torch.device("cuda", torch.cuda.current_device()))
    _check(lib().qlora_selftest_wait_timeout(int(limit_us), res.data_ptr(), _stream(stream)))
    return int(res.item())


def qlora_profile_enable(on: bool = True) -> None:
    _check(lib().qlora_profile_enable(int(on)))


def qlora_profile_read():
    """Returns ({class: device ms}, {class: launches}) since the last read."""
    ms = (ctypes.c_double * len(KERNEL_CLASSES))()
    n = (ctypes.c_int64 * len(KERNEL_CLASSES))()
    _check(lib().qlora_profile_read(ms, n))
    return dict(zip(KERNEL_CLASSES, list(ms))), dict(zip(KERNEL_CLASSES, list(n)))
