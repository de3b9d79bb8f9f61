"""Python binding of libqlora_nf4.so -- the MI355X QLoRA NF4 linear layer.

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  torch supplies device memory (outputs and workspaces are allocated
as torch tensors) and the current HIP stream.  There is no fallback: if the
library is not built, importing the binding raises.

Functions carry the C ABI's names (include/qlora_nf4.h):

    qlora_nf4_quantize(W0)                    -> NF4Weight
    qlora_nf4_dequantize(w)                   -> bf16 [d, k]
    qlora_linear_fwd(w, x, A, B, alpha)       -> (Y, U)
    qlora_linear_bwd(w, x, dY, A, B, alpha, U=None, need_dx=True) -> (dX, dA, dB)
    qlora_nf4_codebook(), qlora_nf4_thresholds()   (host only, no GPU needed)

and, around the linear layer in a fine-tuning step:

    qlora_layernorm_fwd(x, weight, bias)      -> (y, mean, rstd)
    qlora_layernorm_bwd(x, dy, mean, rstd, weight) -> (dx, dweight, dbias)
    qlora_attention_fwd(q, k, v, cu_seqlens)  -> (o, lse, residual)
    qlora_attention_bwd(q, k, v, o, lse, dout, cu_seqlens) -> (dq, dk, dv)
    qlora_logprob_fwd(logits, targets, top)   -> (logp, entropy, lse, top_logp, top_ids)
    qlora_logprob_bwd(logits, targets, lse, entropy, dlogp, dentropy) -> dlogits
    qlora_adamw_step(AdamWPlan(params, grads, m, v, ...), lr=..., step=...)
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

from .build import LIB_PATH

QLORA_OK, QLORA_EINVAL, QLORA_ENOTSUP, QLORA_EALIGN, QLORA_EWORKSPACE, QLORA_EHIP, QLORA_ESCRATCH = range(7)
BLOCK = 64
DQ_BLOCK = 256
NO_DQ = 0  # dq_block of the format without double quantization (fp32 absmax per block)
C2_INT8, C2_FP8_E4M3 = 0, 1  # c2_format: how the c2 bytes of a double-quantized weight encode values
STATE_BLOCK = 256  # elements that share the scales of 8-bit AdamW states
_TYPES = {torch.bfloat16: 0, torch.float32: 1}  # QLORA_BF16, QLORA_F32

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python bit_nf4_quantized_13_amd/build.py` "
        "(there is no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)


class _CWeight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("absmax_q", ctypes.c_void_p),
                ("absmax_scale", ctypes.c_void_p), ("absmax_mean", ctypes.c_void_p),
                ("d", ctypes.c_int64), ("k", ctypes.c_int64),
                ("block", ctypes.c_int32), ("dq_block", ctypes.c_int32),
                ("c2_format", ctypes.c_int32)]


class _CAdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("n", ctypes.c_int64)]


class _CAdamWConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("step", ctypes.c_int64), ("param_type", ctypes.c_int32), ("grad_type", ctypes.c_int32),
                ("state_type", ctypes.c_int32), ("use_master", ctypes.c_int32)]


class _CAttentionShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("sequences", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("dim", ctypes.c_int32), ("ldq", ctypes.c_int64),
                ("ldk", ctypes.c_int64), ("ldv", ctypes.c_int64), ("scale", ctypes.c_float)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t
_WP = ctypes.POINTER(_CWeight)

_SIGS = {
    "qlora_abi_version": (ctypes.c_int, []),
    "qlora_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "qlora_nf4_codebook": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float)]),
    "qlora_nf4_thresholds": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float)]),
    "qlora_nf4_quantize_workspace": (_SZ, [_I64, _I64, _I32, _I32]),
    "qlora_nf4_quantize": (ctypes.c_int, [_P, _WP, _P, _SZ, _P]),
    "qlora_nf4_dequantize": (ctypes.c_int, [_WP, _P, _P]),
    "qlora_linear_workspace": (_SZ, [_I64, _I64, _I64, _I32]),
    "qlora_linear_fwd": (ctypes.c_int, [_WP, _P, _I64, _P, _P, _I32, ctypes.c_float, _P, _P, _P,
                                        _SZ, _P]),
    "qlora_linear_fwd_noalloc": (ctypes.c_int, [_WP, _P, _I64, _P, _P, _I32, ctypes.c_float, _P, _P, _P]),
    "qlora_linear_bwd": (ctypes.c_int, [_WP, _P, _P, _P, _P, _P, _I64, _I32, ctypes.c_float, _P,
                                        _P, _P, _P, _SZ, _P]),
    "qlora_linear_gemm_only": (ctypes.c_int, [_WP, _I32, _I32, _P, _I64, _I32, _P, _P, _SZ, _P]),
    "qlora_time_next_kernel": (ctypes.c_int, [_I32, _P]),
    "qlora_wall_clock_khz": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int32)]),
    "qlora_adapter_merge": (ctypes.c_int, [_WP, _P, _P, _I32, ctypes.c_float, _P, _P]),
    "qlora_adapter_unmerge": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _I32, ctypes.c_float, _P, _P]),
    "qlora_lora_dropout": (ctypes.c_int, [_P, _I64, _I64, ctypes.c_float, ctypes.c_uint64, _P, _P]),
    "qlora_linear_dropout_workspace": (_SZ, [_I64, _I64, _I64, _I32]),
    "qlora_linear_fwd_dropout": (ctypes.c_int, [_WP, _P, _I64, _P, _P, _I32, ctypes.c_float, ctypes.c_float,
                                                ctypes.c_uint64, _P, _P, _P, _SZ, _P]),
    "qlora_linear_bwd_dropout": (ctypes.c_int, [_WP, _P, _P, _P, _P, _P, _I64, _I32, ctypes.c_float,
                                                ctypes.c_float, ctypes.c_uint64, _P, _P, _P, _P, _SZ, _P]),
    "qlora_layernorm_fwd": (ctypes.c_int, [_P, _I32, _I64, _I64, _I64, _P, _P, _I32, ctypes.c_float, _P, _P, _P, _P]),
    "qlora_layernorm_workspace": (_SZ, [_I64, _I64]),
    "qlora_layernorm_bwd": (ctypes.c_int, [_P, _P, _I32, _I64, _I64, _I64, _P, _P, _P, _I32, _P, _P, _P, _P, _SZ,
                                           _P]),
    "qlora_attention_fwd": (ctypes.c_int, [ctypes.POINTER(_CAttentionShape), _P, _P, _P, _P, _P, _P, _P, _P]),
    "qlora_attention_workspace": (_SZ, [ctypes.POINTER(_CAttentionShape)]),
    "qlora_attention_bwd": (ctypes.c_int, [ctypes.POINTER(_CAttentionShape), _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64,
                                           _P, _I64, _P, _I64, _P, _SZ, _P]),
    "qlora_logprob_workspace": (_SZ, [_I64, _I64, _I32]),
    "qlora_logprob_fwd": (ctypes.c_int, [_P, _I32, _I64, _I64, _I64, _P, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "qlora_logprob_bwd": (ctypes.c_int, [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _I64, _P]),
    "qlora_adamw_step": (ctypes.c_int, [ctypes.POINTER(_CAdamWTensor), _I32, ctypes.POINTER(_CAdamWConfig), _P]),
    "qlora_adamw_moments": (ctypes.c_int, [ctypes.POINTER(_CAdamWTensor), _I32, ctypes.POINTER(_P),
                                           ctypes.POINTER(_P), _P]),
}
for _name, (_res, _args) in _SIGS.items():
    if not hasattr(_lib, _name):
        raise ImportError(f"{LIB_PATH} lacks {_name}: it predates its sources; rebuild it with "
                          "`python bit_nf4_quantized_13_amd/build.py`")
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class QloraError(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call}: {status_str(status)}")
        self.status = status


def status_str(status: int) -> str:
    return _lib.qlora_status_str(int(status)).decode()


def _check(status: int, call: str) -> None:
    if status != QLORA_OK:
        raise QloraError(status, call)


def library() -> ctypes.CDLL:
    """The loaded ctypes handle (for tests that call the C ABI directly)."""
    return _lib


def abi_version() -> int:
    return int(_lib.qlora_abi_version())


def qlora_nf4_codebook() -> list[float]:
    out = (ctypes.c_float * 16)()
    _check(_lib.qlora_nf4_codebook(out), "qlora_nf4_codebook")
    return list(out)


def qlora_nf4_thresholds() -> list[float]:
    out = (ctypes.c_float * 15)()
    _check(_lib.qlora_nf4_thresholds(out), "qlora_nf4_thresholds")
    return list(out)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    """The current device's current stream as a hipStream_t: torch.cuda.current_stream().cuda_stream
    without the Stream object (0.1 against 2.9 us, which short calls notice)."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _dev_tensor(t: torch.Tensor, dtype: torch.dtype, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


@dataclass
class NF4Weight:
    """Device buffers of one quantized W0 [d x k] (see qlora_nf4_weight).

    Double-quantized (dq_block == DQ_BLOCK): absmax_q holds c2, absmax_scale
    c1 per group of 256 blocks and absmax_mean the mean; c2_format says
    whether the c2 bytes are int8 values or OCP FP8 e4m3 bit patterns
    (absmax_q is then uint8; `.view(torch.float8_e4m3fn)` reads them).
    Without double quantization (dq_block == NO_DQ): absmax_scale holds the
    fp32 absmax of every block and absmax_q / absmax_mean are None.
    """
    codes: torch.Tensor                  # uint8 [d*k/2]
    absmax_q: torch.Tensor | None        # int8 or uint8 (e4m3 bits) [nb] (double-quantized only)
    absmax_scale: torch.Tensor           # float32 [G] (double-quantized) or [nb]
    absmax_mean: torch.Tensor | None     # float32 [1] (double-quantized only)
    d: int
    k: int
    block: int = BLOCK
    dq_block: int = DQ_BLOCK
    c2_format: int = C2_INT8

    @staticmethod
    def empty(d: int, k: int, device="cuda", double_quant: bool = True,
              c2_fp8: bool = False, block: int = BLOCK) -> "NF4Weight":
        """Uninitialised buffers for W0 [d, k] in blocks of `block` (64, 128 or 256) weights."""
        nb = (d * k) // block
        codes = torch.empty(d * k // 2, dtype=torch.uint8, device=device)
        if not double_quant:
            return NF4Weight(codes, None, torch.empty(nb, dtype=torch.float32, device=device), None,
                             d, k, block=block, dq_block=NO_DQ)
        g = -(-nb // DQ_BLOCK)
        return NF4Weight(codes, torch.empty(nb, dtype=torch.uint8 if c2_fp8 else torch.int8, device=device),
                         torch.empty(g, dtype=torch.float32, device=device),
                         torch.empty(1, dtype=torch.float32, device=device), d, k, block=block,
                         c2_format=C2_FP8_E4M3 if c2_fp8 else C2_INT8)

    @property
    def double_quant(self) -> bool:
        return self.dq_block != NO_DQ

    def c_struct(self) -> _CWeight:
        return _CWeight(self.codes.data_ptr(), _ptr(self.absmax_q),
                        self.absmax_scale.data_ptr(), _ptr(self.absmax_mean),
                        self.d, self.k, self.block, self.dq_block, self.c2_format)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size()
                   for t in (self.codes, self.absmax_q, self.absmax_scale, self.absmax_mean)
                   if t is not None)


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def quantize_workspace_bytes(d: int, k: int, dq_block: int = DQ_BLOCK, block: int = BLOCK) -> int:
    return int(_lib.qlora_nf4_quantize_workspace(d, k, block, dq_block))


def linear_workspace_bytes(m: int, d: int, k: int, r: int, dropout: bool = False) -> int:
    if dropout:
        return int(_lib.qlora_linear_dropout_workspace(m, d, k, r))
    return int(_lib.qlora_linear_workspace(m, d, k, r))


def qlora_lora_dropout(x: torch.Tensor, p: float, seed: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Xd = dropout of bf16 x [M, k] on the adapter input (Philox keep mask of
    (p, seed); kept values x / (1 - p) rounded to bf16, dropped +0)."""
    _dev_tensor(x, torch.bfloat16, "x")
    m, k = x.shape
    xd = out if out is not None else torch.empty_like(x)
    _check(_lib.qlora_lora_dropout(x.data_ptr(), m, k, float(p), int(seed) & (2**64 - 1), xd.data_ptr(),
                                   _stream()), "qlora_lora_dropout")
    return xd


def qlora_nf4_quantize(w0: torch.Tensor, out: NF4Weight | None = None,
                       workspace: torch.Tensor | None = None,
                       double_quant: bool = True, c2_fp8: bool = False, block: int = BLOCK) -> NF4Weight:
    """NF4 in blocks of `block` weights (64, 128 or 256) (+ double quantization
    of the block absmax, c2 in int8 or, with c2_fp8, OCP FP8 e4m3) of fp32 W0
    [d, k] on the current stream.  With `out` given, its block, dq_block and
    c2_format decide the format."""
    _dev_tensor(w0, torch.float32, "W0")
    d, k = w0.shape
    w = out if out is not None else NF4Weight.empty(d, k, w0.device, double_quant, c2_fp8, block)
    ws_bytes = quantize_workspace_bytes(d, k, w.dq_block, w.block)
    ws = workspace if workspace is not None else _workspace(ws_bytes, w0.device)
    cw = w.c_struct()
    _check(_lib.qlora_nf4_quantize(w0.data_ptr(), ctypes.byref(cw), ws.data_ptr(),
                                   ws.numel(), _stream()), "qlora_nf4_quantize")
    return w


def qlora_nf4_dequantize(w: NF4Weight, out: torch.Tensor | None = None) -> torch.Tensor:
    """doubleDequant of W0 into bf16 [d, k]."""
    y = out if out is not None else torch.empty((w.d, w.k), dtype=torch.bfloat16,
                                                device=w.codes.device)
    cw = w.c_struct()
    _check(_lib.qlora_nf4_dequantize(ctypes.byref(cw), y.data_ptr(), _stream()),
           "qlora_nf4_dequantize")
    return y


def qlora_linear_fwd(w: NF4Weight, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                     alpha: float, save_u: bool = True, out: torch.Tensor | None = None,
                     u_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     dropout: float = 0.0, seed: int = 0):
    """Y = x What^T + (alpha/r) (x A^T) B^T.  Returns (Y bf16 [M, d], U fp32 [M, r] or None).

    dropout > 0: the adapter's input is Xd = drop(x) (qlora_lora_dropout with
    this seed), U = Xd A^T; the backward takes the same dropout and seed."""
    _dev_tensor(x, torch.bfloat16, "x")
    _dev_tensor(a, torch.bfloat16, "A")
    _dev_tensor(b, torch.bfloat16, "B")
    m, r = x.shape[0], a.shape[0]
    y = out if out is not None else torch.empty((m, w.d), dtype=torch.bfloat16, device=x.device)
    if u_out is not None:
        u = _dev_tensor(u_out, torch.float32, "U")
    else:
        u = torch.empty((m, r), dtype=torch.float32, device=x.device) if save_u else None
    ws = workspace if workspace is not None else _workspace(
        linear_workspace_bytes(m, w.d, w.k, r, dropout > 0), x.device)
    cw = w.c_struct()
    if dropout > 0:
        _check(_lib.qlora_linear_fwd_dropout(ctypes.byref(cw), x.data_ptr(), m, a.data_ptr(), b.data_ptr(), r,
                                             float(alpha), float(dropout), int(seed) & (2**64 - 1), y.data_ptr(),
                                             _ptr(u), ws.data_ptr(), ws.numel(), _stream()),
               "qlora_linear_fwd_dropout")
        return y, u
    _check(_lib.qlora_linear_fwd(ctypes.byref(cw), x.data_ptr(), m, a.data_ptr(), b.data_ptr(), r,
                                 float(alpha), y.data_ptr(), _ptr(u), ws.data_ptr(), ws.numel(),
                                 _stream()), "qlora_linear_fwd")
    return y, u


def qlora_linear_fwd_noalloc(w: NF4Weight, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                             alpha: float, out: torch.Tensor, u_out: torch.Tensor | None = None):
    """The decode-shaped forward (M <= 16) through qlora_linear_fwd_noalloc: no
    workspace and no allocation in the call (the caller passes Y, and U if
    wanted).  Returns (Y, U or None)."""
    _dev_tensor(x, torch.bfloat16, "x")
    _dev_tensor(a, torch.bfloat16, "A")
    _dev_tensor(b, torch.bfloat16, "B")
    _dev_tensor(out, torch.bfloat16, "Y")
    if u_out is not None:
        _dev_tensor(u_out, torch.float32, "U")
    cw = w.c_struct()
    _check(_lib.qlora_linear_fwd_noalloc(ctypes.byref(cw), x.data_ptr(), x.shape[0], a.data_ptr(), b.data_ptr(),
                                         a.shape[0], float(alpha), out.data_ptr(), _ptr(u_out), _stream()),
           "qlora_linear_fwd_noalloc")
    return out, u_out


def qlora_linear_bwd(w: NF4Weight, x: torch.Tensor, dy: torch.Tensor, a: torch.Tensor,
                     b: torch.Tensor, alpha: float, u: torch.Tensor | None = None,
                     need_dx: bool = True, workspace: torch.Tensor | None = None,
                     outs: tuple | None = None, dropout: float = 0.0, seed: int = 0):
    """Returns (dX bf16 [M, k] or None, dA fp32 [r, k], dB fp32 [d, r]).  dropout and
    seed: those of the forward."""
    _dev_tensor(x, torch.bfloat16, "x")
    _dev_tensor(dy, torch.bfloat16, "dY")
    _dev_tensor(a, torch.bfloat16, "A")
    _dev_tensor(b, torch.bfloat16, "B")
    if u is not None:
        _dev_tensor(u, torch.float32, "U")
    m, r = x.shape[0], a.shape[0]
    if outs is not None:
        dx, da, db = outs
    else:
        dx = torch.empty((m, w.k), dtype=torch.bfloat16, device=x.device) if need_dx else None
        da = torch.empty((r, w.k), dtype=torch.float32, device=x.device)
        db = torch.empty((w.d, r), dtype=torch.float32, device=x.device)
    ws = workspace if workspace is not None else _workspace(
        linear_workspace_bytes(m, w.d, w.k, r, dropout > 0), x.device)
    cw = w.c_struct()
    if dropout > 0:
        _check(_lib.qlora_linear_bwd_dropout(ctypes.byref(cw), x.data_ptr(), dy.data_ptr(), a.data_ptr(),
                                             b.data_ptr(), _ptr(u), m, r, float(alpha), float(dropout),
                                             int(seed) & (2**64 - 1), _ptr(dx), da.data_ptr(), db.data_ptr(),
                                             ws.data_ptr(), ws.numel(), _stream()), "qlora_linear_bwd_dropout")
        return dx, da, db
    _check(_lib.qlora_linear_bwd(ctypes.byref(cw), x.data_ptr(), dy.data_ptr(), a.data_ptr(),
                                 b.data_ptr(), _ptr(u), m, r, float(alpha), _ptr(dx), da.data_ptr(),
                                 db.data_ptr(), ws.data_ptr(), ws.numel(), _stream()),
           "qlora_linear_bwd")
    return dx, da, db


def qlora_linear_gemm_only(w: NF4Weight, backward: bool, a: torch.Tensor, r: int,
                           out: torch.Tensor, workspace: torch.Tensor, expand: bool = False) -> torch.Tensor:
    """Measurement only: re-run the dequant-GEMM kernel of the preceding
    qlora_linear_fwd (a = x, out = Y) or qlora_linear_bwd (a = dY, out = dX) call
    alone, on the workspace that call prepared; expand=True runs the kernel that
    expands the NF4 codes tile by tile instead (with its block scales)."""
    _dev_tensor(a, torch.bfloat16, "a")
    _dev_tensor(out, torch.bfloat16, "out")
    cw = w.c_struct()
    _check(_lib.qlora_linear_gemm_only(ctypes.byref(cw), 1 if backward else 0, 1 if expand else 0, a.data_ptr(),
                                       a.shape[0], r, out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                       _stream()), "qlora_linear_gemm_only")
    return out


TIMED_KERNELS = {"fwd_gemm": 0, "dx_gemm": 1, "decode": 2}


def qlora_time_next_kernel(kernel: str, span: torch.Tensor | None) -> None:
    """Measurement only: the next launch of `kernel` ("fwd_gemm", "dx_gemm",
    "decode") records its start and end clock readings into `span` (a device
    int64 tensor of 2 elements filled with [-1, 0] beforehand: all bits set
    reads as UINT64_MAX); span_duration_us turns it into microseconds."""
    if span is not None:
        _dev_tensor(span, torch.int64, "span")
    _check(_lib.qlora_time_next_kernel(TIMED_KERNELS[kernel], _ptr(span)), "qlora_time_next_kernel")


def wall_clock_khz() -> int:
    v = ctypes.c_int32(0)
    _check(_lib.qlora_wall_clock_khz(ctypes.byref(v)), "qlora_wall_clock_khz")
    return int(v.value)


def span_duration_us(spans: torch.Tensor, khz: int):
    """Durations in microseconds of [n, 2] spans (read back to the host)."""
    s = spans.detach().cpu().view(-1, 2)
    return ((s[:, 1] - s[:, 0]).double() * 1e3 / khz).tolist()


def qlora_adapter_merge(w: NF4Weight, a: torch.Tensor, b: torch.Tensor, alpha: float,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [d, k] = What + (alpha/r) B A (qlora_adapter_merge's fixed rounding)."""
    _dev_tensor(a, torch.bfloat16, "A")
    _dev_tensor(b, torch.bfloat16, "B")
    y = out if out is not None else torch.empty((w.d, w.k), dtype=torch.bfloat16, device=a.device)
    _dev_tensor(y, torch.bfloat16, "out")
    cw = w.c_struct()
    _check(_lib.qlora_adapter_merge(ctypes.byref(cw), a.data_ptr(), b.data_ptr(), a.shape[0], float(alpha),
                                    y.data_ptr(), _stream()), "qlora_adapter_merge")
    return y


def qlora_adapter_unmerge(w_in: torch.Tensor, a: torch.Tensor, b: torch.Tensor, alpha: float,
                          out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [d, k] = W_in - (alpha/r) B A; out may be w_in (in place)."""
    _dev_tensor(w_in, torch.bfloat16, "W_in")
    _dev_tensor(a, torch.bfloat16, "A")
    _dev_tensor(b, torch.bfloat16, "B")
    d, k = w_in.shape
    y = out if out is not None else torch.empty_like(w_in)
    _dev_tensor(y, torch.bfloat16, "out")
    _check(_lib.qlora_adapter_unmerge(w_in.data_ptr(), d, k, a.data_ptr(), b.data_ptr(), a.shape[0],
                                      float(alpha), y.data_ptr(), _stream()), "qlora_adapter_unmerge")
    return y


def _element_type(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _TYPES:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return _TYPES[t.dtype]


def _rows(t: torch.Tensor, name: str) -> int:
    """The row pitch, in elements, of a device matrix whose rows are dense."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or (shape[1] > 1 and strides[1] != 1):
        raise ValueError(f"{name} must be a matrix with dense rows")
    if shape[0] < 2:
        return shape[1]
    if strides[0] < shape[1]:
        raise ValueError(f"{name} must have rows that do not overlap")
    return strides[0]


def _shaped(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str) -> torch.Tensor:
    if _dev_tensor(t, dtype, name).shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _dense_workspace(ws: torch.Tensor) -> torch.Tensor:
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    return ws


def qlora_layernorm_fwd(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                        eps: float = 1e-5, out: torch.Tensor | None = None, save_stats: bool = True):
    """y = (x - mean) rstd weight + bias over the rows of x [M, n] (bf16 or fp32, rows at any pitch).
    Returns (y like x, mean fp32 [M], rstd fp32 [M]), the statistics None without save_stats."""
    kind, ld = _element_type(x, "x"), _rows(x, "x")
    m, n = x.shape
    ref = weight if weight is not None else bias
    wkind = _element_type(ref, "weight") if ref is not None else 0
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _shaped(t, ref.dtype, (n,), name)
    y = _shaped(out, x.dtype, (m, n), "out") if out is not None else torch.empty(m, n, dtype=x.dtype, device=x.device)
    mean = torch.empty(m, dtype=torch.float32, device=x.device) if save_stats else None
    rstd = torch.empty_like(mean) if save_stats else None
    _check(_lib.qlora_layernorm_fwd(x.data_ptr(), kind, m, n, ld, _ptr(weight), _ptr(bias), wkind, float(eps),
                                    y.data_ptr(), _ptr(mean), _ptr(rstd), _stream()), "qlora_layernorm_fwd")
    return y, mean, rstd


def qlora_layernorm_bwd(x: torch.Tensor, dy: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor | None = None, need_dw: bool = True, need_db: bool = True,
                        workspace: torch.Tensor | None = None, outs: tuple | None = None):
    """Returns (dx like dy, dweight fp32 [n] or None, dbias fp32 [n] or None); mean and rstd are the
    forward's.  outs: the three of them, None in place of a gradient that is not wanted."""
    kind, ld = _element_type(x, "x"), _rows(x, "x")
    m, n = x.shape
    _shaped(dy, x.dtype, (m, n), "dy")
    _shaped(mean, torch.float32, (m,), "mean")
    _shaped(rstd, torch.float32, (m,), "rstd")
    wkind = 0
    if weight is not None:
        wkind = _element_type(weight, "weight")
        _shaped(weight, weight.dtype, (n,), "weight")
    if outs is not None:
        dx, dw, db = outs
        _shaped(dx, x.dtype, (m, n), "dx")
        for t, name in ((dw, "dweight"), (db, "dbias")):
            if t is not None:
                _shaped(t, torch.float32, (n,), name)
    else:
        dx = torch.empty_like(dy)
        dw = torch.empty(n, dtype=torch.float32, device=x.device) if need_dw else None
        db = torch.empty(n, dtype=torch.float32, device=x.device) if need_db else None
    ws = None
    if workspace is not None:
        ws = _dense_workspace(workspace)
    elif dw is not None or db is not None:
        ws = _workspace(layernorm_workspace_bytes(m, n), x.device)
    _check(_lib.qlora_layernorm_bwd(x.data_ptr(), dy.data_ptr(), kind, m, n, ld, mean.data_ptr(), rstd.data_ptr(),
                                    _ptr(weight), wkind, dx.data_ptr(), _ptr(dw), _ptr(db), _ptr(ws),
                                    ws.numel() if ws is not None else 0, _stream()), "qlora_layernorm_bwd")
    return dx, dw, db


def layernorm_workspace_bytes(m: int, n: int) -> int:
    return int(_lib.qlora_layernorm_workspace(m, n))


def _heads(t: torch.Tensor, rows: int, dim: int, name: str) -> int:
    """The row pitch, in elements, of a device bf16 [rows, heads, dim] whose rows are dense."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[0] != rows or shape[2] != dim:
        raise ValueError(f"{name} must have shape [{rows}, heads, {dim}], got {list(shape)}")
    heads, (pitch, head_pitch, step) = shape[1], t.stride()
    if (dim > 1 and step != 1) or (heads > 1 and head_pitch != dim):
        raise ValueError(f"{name} must have its heads side by side in dense rows")
    if rows < 2:
        return heads * dim
    if pitch < heads * dim:
        raise ValueError(f"{name} must have rows that do not overlap")
    return pitch


def _attention_shape(q, k, v, cu_seqlens, scale) -> _CAttentionShape:
    if q.dim() != 3:
        raise ValueError("q must have shape [rows, heads, dim]")
    rows, heads, dim = q.shape
    ldq, ldk, ldv = _heads(q, rows, dim, "q"), _heads(k, rows, dim, "k"), _heads(v, rows, dim, "v")
    kv_heads = k.shape[1]
    if kv_heads != v.shape[1]:
        raise ValueError("k and v must have the same heads")
    _dev_tensor(cu_seqlens, torch.int32, "cu_seqlens")
    return _CAttentionShape(rows, cu_seqlens.numel() - 1, heads, kv_heads, dim, ldq, ldk, ldv,
                            dim ** -0.5 if scale is None else scale)


def qlora_attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                        scale: float | None = None, save_residual: bool = False, out: torch.Tensor | None = None):
    """Causal attention over packed sequences: q bf16 [T, heads, dim], k and v [T, kv_heads, dim] (rows at
    any pitch of a multiple of 8), sequence s in the rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1 (int32).
    Returns (o like q, lse fp32 [heads, T], residual like o or None); the residual is what the backward
    takes to be exact in o.  scale: dim ** -0.5 if not given."""
    shape = _attention_shape(q, k, v, cu_seqlens, scale)
    rows, heads, dim = q.shape
    o = _shaped(out, torch.bfloat16, q.shape, "out") if out is not None else torch.empty(
        rows, heads, dim, dtype=torch.bfloat16, device=q.device)
    res = torch.empty_like(o) if save_residual else None
    lse = torch.empty(heads, rows, dtype=torch.float32, device=q.device)
    _check(_lib.qlora_attention_fwd(ctypes.byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                    cu_seqlens.data_ptr(), o.data_ptr(), _ptr(res), lse.data_ptr(), _stream()),
           "qlora_attention_fwd")
    return o, lse, res


def qlora_attention_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                        dout: torch.Tensor, cu_seqlens: torch.Tensor, scale: float | None = None,
                        residual: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        outs: tuple | None = None):
    """(dq, dk, dv) like q, k, v from the forward's o, lse (and residual) and dout; outs may be slices
    of one matrix."""
    shape = _attention_shape(q, k, v, cu_seqlens, scale)
    _shaped(o, torch.bfloat16, q.shape, "o")
    _shaped(dout, torch.bfloat16, q.shape, "dout")
    _shaped(lse, torch.float32, (q.shape[1], q.shape[0]), "lse")
    if residual is not None:
        _shaped(residual, torch.bfloat16, q.shape, "residual")
    rows, heads, dim = q.shape
    if outs is None:
        kv_heads, device = k.shape[1], q.device
        dq = torch.empty_like(o)
        dk = torch.empty(rows, kv_heads, dim, dtype=torch.bfloat16, device=device)
        dv = torch.empty_like(dk)
        pitches = heads * dim, kv_heads * dim, kv_heads * dim
    else:
        dq, dk, dv = outs
        pitches = []
        for t, like, name in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
            if t.shape != like.shape:
                raise ValueError(f"{name} must have shape {list(like.shape)}")
            pitches.append(_heads(t, rows, dim, name))
    ws = _dense_workspace(workspace) if workspace is not None else _workspace(
        int(_lib.qlora_attention_workspace(ctypes.byref(shape))), q.device)
    _check(_lib.qlora_attention_bwd(ctypes.byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                    _ptr(residual), lse.data_ptr(), dout.data_ptr(), cu_seqlens.data_ptr(),
                                    dq.data_ptr(), pitches[0], dk.data_ptr(), pitches[1], dv.data_ptr(), pitches[2],
                                    ws.data_ptr(), ws.numel(), _stream()), "qlora_attention_bwd")
    return dq, dk, dv


def logprob_workspace_bytes(m: int, v: int, top: int = 0) -> int:
    return int(_lib.qlora_logprob_workspace(m, v, top))


def qlora_logprob_fwd(logits: torch.Tensor, targets: torch.Tensor, top: int = 0,
                      workspace: torch.Tensor | None = None):
    """Log-probabilities of the targets (int64 [M]; outside [0, V): no target, 0) under logits [M, V]
    (bf16 or fp32, rows at any pitch, -inf for tokens that are ruled out).  Returns fp32 [M] logp, entropy
    and lse, and the `top` best alternatives: fp32 [M, top] log-probabilities and int32 [M, top] ids
    (None, None with top = 0)."""
    kind, ld = _element_type(logits, "logits"), _rows(logits, "logits")
    m, v = logits.shape
    _shaped(targets, torch.int64, (m,), "targets")
    device = logits.device
    logp, entropy, lse = torch.empty(3, m, dtype=torch.float32, device=device).unbind(0)
    top_logp = torch.empty(m, top, dtype=torch.float32, device=device) if top > 0 else None
    top_ids = torch.empty_like(top_logp, dtype=torch.int32) if top > 0 else None
    ws = _dense_workspace(workspace) if workspace is not None else _workspace(logprob_workspace_bytes(m, v, top), device)
    _check(_lib.qlora_logprob_fwd(logits.data_ptr(), kind, m, v, ld, targets.data_ptr(), int(top), logp.data_ptr(),
                                  entropy.data_ptr(), lse.data_ptr(), _ptr(top_logp), _ptr(top_ids), ws.data_ptr(),
                                  ws.numel(), _stream()), "qlora_logprob_fwd")
    return logp, entropy, lse, top_logp, top_ids


def qlora_logprob_bwd(logits: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor, entropy: torch.Tensor | None,
                      dlogp: torch.Tensor, dentropy: torch.Tensor | None = None,
                      out: torch.Tensor | None = None) -> torch.Tensor:
    """dlogits [M, V] (like logits) from the gradients of logp and, if given, entropy; out may be the
    logits themselves (in place)."""
    kind, ld = _element_type(logits, "logits"), _rows(logits, "logits")
    m, v = logits.shape
    _shaped(targets, torch.int64, (m,), "targets")
    for t, name in ((lse, "lse"), (entropy, "entropy"), (dlogp, "dlogp"), (dentropy, "dentropy")):
        if t is not None:
            _shaped(t, torch.float32, (m,), name)
    if out is None:
        out = torch.empty(m, v, dtype=logits.dtype, device=logits.device)
    elif out.dtype != logits.dtype or out.shape != logits.shape:
        raise ValueError("out must have the logits' type and shape")
    _check(_lib.qlora_logprob_bwd(logits.data_ptr(), kind, m, v, ld, targets.data_ptr(), _ptr(lse), _ptr(entropy),
                                  _ptr(dlogp), _ptr(dentropy), out.data_ptr(), _rows(out, "out"), _stream()),
           "qlora_logprob_bwd")
    return out


class AdamWPlan:
    """The tensors of an AdamW step, checked and laid out once: params (bf16 or fp32), grads (bf16 or
    fp32) and states of the same sizes.  States are fp32 m and v, or int8 m and uint8 v with fp32
    scales (one for each 256 elements, the last block possibly shorter); masters are fp32 weights
    beside bf16 params.  The plan keeps the tensors: every step reads and updates these buffers, so
    gradients have to arrive in the same ones (qlora_linear_bwd's outs)."""

    def __init__(self, params, grads, m, v, m_scales=None, v_scales=None, masters=None):
        params, grads, m, v = list(params), list(grads), list(m), list(v)
        count = len(params)
        if not count:
            raise ValueError("an AdamW plan needs at least one tensor")
        self.bits8 = m_scales is not None
        if self.bits8 != (v_scales is not None):
            raise ValueError("8-bit states need m_scales and v_scales")
        none = [None] * count
        m_scales, v_scales = (list(m_scales), list(v_scales)) if self.bits8 else (none, none)
        self.master = masters is not None
        masters = list(masters) if self.master else none
        for name, ts in (("grads", grads), ("m", m), ("v", v), ("m_scales", m_scales), ("v_scales", v_scales),
                         ("masters", masters)):
            if len(ts) != count:
                raise ValueError(f"{count} params and {len(ts)} {name}")
        self.param_type = _element_type(params[0], "params")
        self.grad_type = _element_type(grads[0], "grads")
        f32 = torch.float32
        mt, vt = (torch.int8, torch.uint8) if self.bits8 else (f32, f32)
        self.count = count
        self.table = (_CAdamWTensor * count)()
        self.tensors = (params, grads, m, v, m_scales, v_scales, masters)
        self.sizes = [p.numel() for p in params]
        for i, (p, g, mi, vi, ms, vs, w) in enumerate(zip(*self.tensors)):
            n = p.numel()
            for t, dtype, size, name in ((p, params[0].dtype, n, "params"), (g, grads[0].dtype, n, "grads"),
                                         (mi, mt, n, "m"), (vi, vt, n, "v"), (ms, f32, -(-n // STATE_BLOCK), "m_scales"),
                                         (vs, f32, -(-n // STATE_BLOCK), "v_scales"), (w, f32, n, "masters")):
                if t is None and name not in ("params", "grads", "m", "v"):
                    continue
                if _dev_tensor(t, dtype, f"{name}[{i}]").numel() != size:
                    raise ValueError(f"{name}[{i}] must have {size} elements, got {t.numel()}")
            self.table[i] = _CAdamWTensor(_ptr(p), _ptr(g), _ptr(mi), _ptr(vi), _ptr(ms), _ptr(vs), _ptr(w), n)

    @staticmethod
    def zeros(params, grads, bits8: bool = True, master: bool = False) -> "AdamWPlan":
        """A plan with new states (zeros) for params, and with `master` fp32 copies of them."""
        params = list(params)
        mt, vt = (torch.int8, torch.uint8) if bits8 else (torch.float32, torch.float32)
        scales = (lambda: [torch.zeros(-(-p.numel() // STATE_BLOCK), dtype=torch.float32, device=p.device)
                           for p in params]) if bits8 else (lambda: None)
        return AdamWPlan(params, grads, [torch.zeros(p.shape, dtype=mt, device=p.device) for p in params],
                         [torch.zeros(p.shape, dtype=vt, device=p.device) for p in params], scales(), scales(),
                         [p.float() for p in params] if master else None)


def qlora_adamw_step(plan: AdamWPlan, lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999,
                     eps: float = 1e-8, weight_decay: float = 0.0, grad_scale: float = 1.0) -> None:
    """One AdamW step on the plan's tensors, on the current stream; `step` counts from 1."""
    config = _CAdamWConfig(lr, beta1, beta2, eps, weight_decay, grad_scale, step, plan.param_type, plan.grad_type,
                           int(plan.bits8), int(plan.master))
    _check(_lib.qlora_adamw_step(plan.table, plan.count, ctypes.byref(config), _stream()), "qlora_adamw_step")


def qlora_adamw_moments(plan: AdamWPlan, m_out=None, v_out=None):
    """The fp32 values of the plan's 8-bit states: (list of m, list of v)."""
    if not plan.bits8:
        raise ValueError("the plan's states are not in 8 bits")
    outs = []
    for given, name in ((m_out, "m_out"), (v_out, "v_out")):
        ts = list(given) if given is not None else [torch.empty(t.shape, dtype=torch.float32, device=t.device)
                                                     for t in plan.tensors[2]]
        if len(ts) != plan.count:
            raise ValueError(f"{plan.count} tensors and {len(ts)} {name}")
        for i, (t, n) in enumerate(zip(ts, plan.sizes)):
            if t.is_cuda and t.dtype == torch.float32 and t.is_contiguous() and t.numel() == n:
                continue
            _dev_tensor(t, torch.float32, f"{name}[{i}]")
            raise ValueError(f"{name}[{i}] must have {n} elements, got {t.numel()}")
        outs.append(ts)
    ptrs = [(_P * plan.count)(*[t.data_ptr() for t in ts]) for ts in outs]
    _check(_lib.qlora_adamw_moments(plan.table, plan.count, ptrs[0], ptrs[1], _stream()), "qlora_adamw_moments")
    return outs[0], outs[1]


__all__ = [
    "qlora_layernorm_fwd", "qlora_layernorm_bwd", "layernorm_workspace_bytes",
    "qlora_attention_fwd", "qlora_attention_bwd",
    "qlora_logprob_fwd", "qlora_logprob_bwd", "logprob_workspace_bytes",
    "AdamWPlan", "qlora_adamw_step", "qlora_adamw_moments", "STATE_BLOCK",
    "NF4Weight", "QloraError", "qlora_nf4_quantize", "qlora_nf4_dequantize", "qlora_linear_fwd",
    "qlora_linear_fwd_noalloc",
    "qlora_linear_bwd", "qlora_linear_gemm_only", "qlora_time_next_kernel", "wall_clock_khz",
    "span_duration_us", "qlora_adapter_merge", "qlora_adapter_unmerge",
    "qlora_lora_dropout",
    "qlora_nf4_codebook", "qlora_nf4_thresholds", "status_str", "library",
    "abi_version", "quantize_workspace_bytes", "linear_workspace_bytes",
    "BLOCK", "DQ_BLOCK", "NO_DQ", "C2_INT8", "C2_FP8_E4M3",
]
