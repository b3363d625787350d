"""dense_gemm_tiled_amd -- MI355X (gfx950) dense GEMM, Python binding.

A thin ctypes layer over libtcgemm.so (C ABI in include/tcgemm.h).  PyTorch is
used only for device memory and streams: every GEMM runs in the library's HIP
kernels, enqueued on torch's current stream.  There is no fallback path: if
the library is not built, every call raises.

    import dense_gemm_tiled_amd as tg
    tg.gemm(a, b, c, alpha=1.0, beta=0.0, transpose_a=False, transpose_b=False)

computes c = alpha * op(a) @ op(b) + beta * c in place (tensorcore "GEMM",
section "Surface"), where a is stored [M,K] or, transposed, [K,M]; b is
stored [K,N] or, transposed, [N,K]; c is [M,N].  3-D tensors make a batched
call (one launch for all problems).
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, NamedTuple, Optional, Tuple

__all__ = [
    "gemm", "w4_quantize", "w4_dequantize", "w4_pack", "w4_gemm", "moe_route", "moe", "W4Weight",
    "cross_entropy", "cross_entropy_backward", "moe_balance", "moe_route_backward",
    "plan", "TcGemmError", "last_kernel", "dispatch_count", "time_next_gemm", "library_path",
    "load_library", "F32", "F16", "BF16", "I8", "I32", "status_name", "DescT",
    "BatchedDescT", "PlanInfoT",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libtcgemm.so")

# tc_dtype_t
F32, F16, BF16, I8, I32 = 0, 1, 2, 3, 4
_NAMES = {F32: "f32", F16: "f16", BF16: "bf16", I8: "i8", I32: "i32"}

# tc_status_t
_STATUS = {0: "TC_OK", 1: "TC_ERR_INVALID_ARGUMENT", 2: "TC_ERR_UNSUPPORTED",
           3: "TC_ERR_OVERFLOW", 4: "TC_ERR_ALIASING", 5: "TC_ERR_OUT_OF_MEMORY",
           6: "TC_ERR_DEVICE"}


def status_name(code: int) -> str:
    return _STATUS.get(int(code), "TC_ERR_UNKNOWN(%d)" % code)


class TcGemmError(RuntimeError):
    """A libtcgemm call returned an error status."""

    def __init__(self, status: int, message: str):
        self.status = int(status)
        self.message = message
        super().__init__("%s: %s" % (status_name(status), message))


class DescT(ctypes.Structure):
    """tc_gemm_desc"""
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("a_dtype", ctypes.c_int), ("b_dtype", ctypes.c_int),
                ("c_dtype", ctypes.c_int), ("accum_dtype", ctypes.c_int),
                ("transpose_a", ctypes.c_bool), ("transpose_b", ctypes.c_bool),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("lda", ctypes.c_int32), ("ldb", ctypes.c_int32), ("ldc", ctypes.c_int32)]


class BatchedDescT(ctypes.Structure):
    """tc_gemm_batched_desc"""
    _fields_ = [("base", DescT), ("batch", ctypes.c_int32),
                ("stride_a", ctypes.c_int64), ("stride_b", ctypes.c_int64),
                ("stride_c", ctypes.c_int64)]


class EpilogueT(ctypes.Structure):
    """tc_epilogue"""
    _fields_ = [("bias", ctypes.c_void_p), ("bias_stride", ctypes.c_int64),
                ("activation", ctypes.c_int), ("col_scale", ctypes.c_void_p),
                ("scale_stride", ctypes.c_int64)]


class QWeightDescT(ctypes.Structure):
    """tc_qweight_desc"""
    _fields_ = [("batch", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("group", ctypes.c_int32), ("scale_dtype", ctypes.c_int),
                ("has_zeros", ctypes.c_bool)]


class QWeightT(ctypes.Structure):
    """tc_qweight"""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p)]


class QGemmDescT(ctypes.Structure):
    """tc_qgemm_desc"""
    _fields_ = [("M", ctypes.c_int32), ("x_dtype", ctypes.c_int), ("y_dtype", ctypes.c_int),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("ldx", ctypes.c_int32), ("ldy", ctypes.c_int32)]


class RouteDescT(ctypes.Structure):
    """tc_route_desc"""
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("ld", ctypes.c_int32), ("renormalize", ctypes.c_bool),
                ("scale", ctypes.c_float)]


class MoeDescT(ctypes.Structure):
    """tc_moe_desc"""
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("top_k", ctypes.c_int32), ("x_dtype", ctypes.c_int),
                ("y_dtype", ctypes.c_int), ("ldx", ctypes.c_int32), ("ldy", ctypes.c_int32),
                ("gate", ctypes.c_int), ("group", ctypes.c_int32), ("has_zeros", ctypes.c_bool)]


class CeDescT(ctypes.Structure):
    """tc_ce_desc"""
    _fields_ = [("T", ctypes.c_int32), ("V", ctypes.c_int32), ("H", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("ldx", ctypes.c_int32), ("ldw", ctypes.c_int32),
                ("targets64", ctypes.c_bool), ("scale", ctypes.c_float)]


class CeGradsT(ctypes.Structure):
    """tc_ce_grads"""
    _fields_ = [("grad", ctypes.c_void_p), ("grad_stride", ctypes.c_int64),
                ("dx", ctypes.c_void_p), ("dx_dtype", ctypes.c_int), ("lddx", ctypes.c_int32),
                ("dw", ctypes.c_void_p), ("dw_dtype", ctypes.c_int), ("lddw", ctypes.c_int32),
                ("beta", ctypes.c_float)]


# tc_gate_t
GATES = {"silu": 0, "gelu_tanh": 1}

# tc_activation_t
ACTIVATIONS = {"none": 0, "relu": 1, "gelu_tanh": 2}


class PlanInfoT(ctypes.Structure):
    """tc_plan_info"""
    _fields_ = [("kernel", ctypes.c_char * 128),
                ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("tile_k", ctypes.c_int32), ("threads", ctypes.c_int32),
                ("tiles_m", ctypes.c_int32), ("tiles_n", ctypes.c_int32),
                ("splits", ctypes.c_int32), ("k_per_split", ctypes.c_int32),
                ("grid", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("launches", ctypes.c_int32), ("band", ctypes.c_int32)]


# Every symbol include/tcgemm.h declares, with its ctypes signature.
_VP = ctypes.c_void_p
_SIGNATURES = {
    "tc_context_create": (ctypes.c_int, [ctypes.POINTER(_VP)]),
    "tc_context_destroy": (None, [_VP]),
    "tc_stream_create": (ctypes.c_int, [_VP, ctypes.POINTER(_VP)]),
    "tc_stream_wrap": (ctypes.c_int, [_VP, _VP, ctypes.POINTER(_VP)]),
    "tc_stream_sync": (ctypes.c_int, [_VP]),
    "tc_stream_destroy": (None, [_VP]),
    "tc_gemm": (ctypes.c_int, [_VP, ctypes.POINTER(DescT), _VP, _VP, _VP]),
    "tc_gemm_async": (ctypes.c_int, [_VP, ctypes.POINTER(DescT), _VP, _VP, _VP, _VP]),
    "tc_gemm_batched": (ctypes.c_int, [_VP, ctypes.POINTER(BatchedDescT), _VP, _VP, _VP]),
    "tc_gemm_batched_async": (ctypes.c_int,
                              [_VP, ctypes.POINTER(BatchedDescT), _VP, _VP, _VP, _VP]),
    "tc_gemm_batched_async_noalloc": (ctypes.c_int,
                                      [_VP, ctypes.POINTER(BatchedDescT), _VP, _VP, _VP, _VP]),
    "tc_gemm_epilogue": (ctypes.c_int, [_VP, ctypes.POINTER(BatchedDescT),
                                        ctypes.POINTER(EpilogueT), _VP, _VP, _VP]),
    "tc_gemm_epilogue_async": (ctypes.c_int, [_VP, ctypes.POINTER(BatchedDescT),
                                              ctypes.POINTER(EpilogueT), _VP, _VP, _VP, _VP]),
    "tc_gemm_plan": (ctypes.c_int, [_VP, ctypes.POINTER(BatchedDescT),
                                    ctypes.POINTER(PlanInfoT)]),
    "tc_set_autotune": (ctypes.c_int, [_VP, ctypes.c_int]),
    "tc_autotune_entries": (ctypes.c_int64, [_VP]),
    "tc_last_kernel": (ctypes.c_char_p, [_VP]),
    "tc_dispatch_count": (ctypes.c_uint64, [_VP]),
    "tc_time_next_gemm": (ctypes.c_int, [_VP, _VP, _VP]),
    "tc_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "tc_last_error": (ctypes.c_char_p, [_VP]),
    "tc_tile_of_workgroup": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                            ctypes.c_int32, ctypes.c_int64,
                                            ctypes.POINTER(ctypes.c_int32),
                                            ctypes.POINTER(ctypes.c_int32),
                                            ctypes.POINTER(ctypes.c_int32)]),
    "tc_version": (ctypes.c_char_p, []),
    "tc_qweight_sizes": (ctypes.c_int, [ctypes.POINTER(QWeightDescT), ctypes.POINTER(ctypes.c_int64),
                                        ctypes.POINTER(ctypes.c_int64),
                                        ctypes.POINTER(ctypes.c_int64)]),
    "tc_quantize_async": (ctypes.c_int, [_VP, ctypes.POINTER(QWeightDescT), _VP, ctypes.c_int,
                                         ctypes.c_int64, ctypes.c_int64,
                                         ctypes.POINTER(QWeightT), _VP]),
    "tc_dequantize_async": (ctypes.c_int, [_VP, ctypes.POINTER(QWeightDescT),
                                           ctypes.POINTER(QWeightT), _VP, ctypes.c_int,
                                           ctypes.c_int64, ctypes.c_int64, _VP]),
    "tc_qweight_pack_async": (ctypes.c_int, [_VP, ctypes.POINTER(QWeightDescT),
                                             ctypes.POINTER(QWeightT), ctypes.POINTER(QWeightT),
                                             _VP]),
    "tc_qgemm_async": (ctypes.c_int, [_VP, ctypes.POINTER(QGemmDescT),
                                      ctypes.POINTER(QWeightDescT), _VP, ctypes.POINTER(QWeightT),
                                      _VP, ctypes.POINTER(EpilogueT), _VP]),
    "tc_moe_route_async": (ctypes.c_int, [_VP, ctypes.POINTER(RouteDescT), _VP, _VP, _VP, _VP]),
    "tc_moe_workspace": (ctypes.c_int, [ctypes.POINTER(MoeDescT), ctypes.POINTER(ctypes.c_int64)]),
    "tc_moe_async": (ctypes.c_int, [_VP, ctypes.POINTER(MoeDescT), _VP, ctypes.POINTER(RouteDescT),
                                    _VP, _VP, _VP, ctypes.POINTER(QWeightT),
                                    ctypes.POINTER(QWeightT), _VP, _VP, ctypes.c_int64, _VP]),
    "tc_cross_entropy_workspace": (ctypes.c_int, [ctypes.POINTER(CeDescT), _VP, _VP,
                                                  ctypes.POINTER(ctypes.c_int64)]),
    "tc_cross_entropy_async": (ctypes.c_int, [_VP, ctypes.POINTER(CeDescT), _VP, _VP, _VP, _VP, _VP,
                                              _VP, ctypes.c_int64, _VP]),
    "tc_cross_entropy_backward_workspace": (ctypes.c_int, [ctypes.POINTER(CeDescT),
                                                           ctypes.POINTER(CeGradsT), _VP, _VP,
                                                           ctypes.POINTER(ctypes.c_int64)]),
    "tc_cross_entropy_backward_async": (ctypes.c_int, [_VP, ctypes.POINTER(CeDescT),
                                                       ctypes.POINTER(CeGradsT), _VP, _VP, _VP, _VP,
                                                       _VP, ctypes.c_int64, _VP]),
    "tc_moe_balance_workspace": (ctypes.c_int, [ctypes.POINTER(RouteDescT),
                                                ctypes.POINTER(ctypes.c_int64)]),
    "tc_moe_balance_async": (ctypes.c_int, [_VP, ctypes.POINTER(RouteDescT), _VP, _VP,
                                            ctypes.c_float, _VP, _VP, _VP, _VP, ctypes.c_int64, _VP]),
    "tc_moe_route_backward_async": (ctypes.c_int, [_VP, ctypes.POINTER(RouteDescT), _VP, _VP, _VP, _VP,
                                                   _VP, _VP, ctypes.c_int, ctypes.c_int32, _VP]),
}

_lib = None


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libtcgemm.so (built in-tree by dense_gemm_tiled_amd.build).

    Raises RuntimeError if it is missing: there is no other implementation.
    """
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            "libtcgemm.so is not built (%s); run `python -m dense_gemm_tiled_amd.build` "
            "or __graft_entry__.build()" % _LIB_PATH)
    lib = ctypes.CDLL(_LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


# ------------------------------------------------------------------ context / streams
_ctx: Dict[int, int] = {}                       # device -> tc_context*
_streams: Dict[Tuple[int, int], int] = {}      # (device, hipStream_t) -> tc_stream*


def _check(status: int, ctx: Optional[int]) -> None:
    if status != 0:
        msg = load_library().tc_last_error(ctx)
        raise TcGemmError(status, (msg or b"").decode())


def _context(device: int) -> int:
    h = _ctx.get(device)
    if h is None:
        out = _VP()
        _check(load_library().tc_context_create(ctypes.byref(out)), None)
        h = _ctx.setdefault(device, out.value)     # (another thread may have been first)
    return h


def _current_raw_stream(device: int) -> int:
    """torch's current stream on `device` as a hipStream_t (an int)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return int(raw(device))
    return int(torch.cuda.current_stream(device).cuda_stream)


def _torch_stream(device: int, stream=None) -> Tuple[int, int]:
    handle = _current_raw_stream(device) if stream is None else int(stream.cuda_stream)
    key = (device, handle)
    s = _streams.get(key)
    ctx = _context(device)
    if s is None:
        import torch
        out = _VP()
        with torch.cuda.device(device):
            _check(load_library().tc_stream_wrap(ctx, _VP(handle), ctypes.byref(out)), ctx)
        s = _streams.setdefault(key, out.value)
    return ctx, s


def last_kernel(device: int = 0) -> str:
    return (load_library().tc_last_kernel(_context(device)) or b"").decode()


def dispatch_count(device: int = 0) -> int:
    return int(load_library().tc_dispatch_count(_context(device)))


def time_next_gemm(start, end, device: int = 0) -> None:
    """Have the next GEMM call record torch.cuda.Event `start` and `end` on
    its stream right around its main GEMM kernel (see tc_time_next_gemm).
    The events must already exist on the device (recorded once)."""
    ctx = _context(device)
    _check(load_library().tc_time_next_gemm(ctx, _VP(start.cuda_event), _VP(end.cuda_event)), ctx)


# ------------------------------------------------------------------ descriptors
def _dtype_code(t) -> int:
    import torch
    table = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16,
             torch.int8: I8, torch.int32: I32}
    if t.dtype not in table:
        raise TcGemmError(2, "unsupported tensor dtype %s" % t.dtype)
    return table[t.dtype]


def _ld(t) -> int:
    """Leading dimension (elements) of the last two dims of a row-major view."""
    if t.stride(-1) != 1 and t.size(-1) > 1:
        raise TcGemmError(1, "the last dimension must be contiguous (stride 1)")
    if t.size(-2) <= 1:
        return int(t.size(-1))
    return int(t.stride(-2))


def _i32(**sizes):
    """The values of sizes that a descriptor holds in 32 bits (ctypes would
    keep the lower half of a longer one)."""
    for name, v in sizes.items():
        if not -2 ** 31 <= v < 2 ** 31:
            raise TcGemmError(3, "%s=%d does not fit 32 bits" % (name, v))
    return tuple(sizes.values())


def make_desc(a, b, c, alpha: float = 1.0, beta: float = 0.0,
              transpose_a: bool = False, transpose_b: bool = False) -> BatchedDescT:
    """Build the batched descriptor for tensors a, b, c (2-D or 3-D)."""
    if a.dim() not in (2, 3) or b.dim() not in (2, 3) or c.dim() not in (2, 3):
        raise TcGemmError(1, "operands must be 2-D or 3-D tensors")
    M, N = int(c.size(-2)), int(c.size(-1))
    K = int(a.size(-2) if transpose_a else a.size(-1))
    a_m = int(a.size(-1) if transpose_a else a.size(-2))
    b_k, b_n = (int(b.size(-1)), int(b.size(-2))) if transpose_b else (int(b.size(-2)), int(b.size(-1)))
    if a_m != M or b_n != N or b_k != K:
        raise TcGemmError(1, "shape mismatch: op(a) %dx%d, op(b) %dx%d, c %dx%d"
                          % (a_m, K, b_k, b_n, M, N))
    batch = int(c.size(0)) if c.dim() == 3 else 1
    for t in (a, b):
        if t.dim() == 3 and int(t.size(0)) != batch:
            raise TcGemmError(1, "batch sizes differ")
    ad, bd, cd = _dtype_code(a), _dtype_code(b), _dtype_code(c)
    accum = I32 if ad == I8 else F32
    desc = BatchedDescT()
    base = desc.base
    base.M, base.N, base.K = _i32(M=M, N=N, K=K)
    base.a_dtype, base.b_dtype, base.c_dtype, base.accum_dtype = ad, bd, cd, accum
    base.transpose_a, base.transpose_b = bool(transpose_a), bool(transpose_b)
    base.alpha, base.beta = float(alpha), float(beta)
    base.lda, base.ldb, base.ldc = _i32(lda=_ld(a), ldb=_ld(b), ldc=_ld(c))
    desc.batch, = _i32(batch=batch)
    desc.stride_a = int(a.stride(0)) if a.dim() == 3 else 0
    desc.stride_b = int(b.stride(0)) if b.dim() == 3 else 0
    desc.stride_c = int(c.stride(0)) if c.dim() == 3 else 0
    return desc


# ------------------------------------------------------------------ API
def _column_vector(c, t, name: str, dtype) -> Tuple[int, int]:
    """(pointer, per-problem stride) of a [N] or [batch, N] GPU tensor."""
    N = int(c.size(-1))
    if not t.is_cuda or t.dtype != dtype:
        raise TcGemmError(1, "%s must be a GPU tensor of dtype %s" % (name, dtype))
    if int(t.size(-1)) != N or (t.size(-1) > 1 and t.stride(-1) != 1):
        raise TcGemmError(1, "%s must hold N contiguous values per problem" % name)
    stride = 0
    if t.dim() == 2:
        batch = int(c.size(0)) if c.dim() == 3 else 1
        if int(t.size(0)) != batch:
            raise TcGemmError(1, "%s has %d rows for %d problems" % (name, t.size(0), batch))
        stride = int(t.stride(0))
    elif t.dim() != 1:
        raise TcGemmError(1, "%s must be 1-D or 2-D" % name)
    return t.data_ptr(), stride


def make_epilogue(c, bias=None, activation: Optional[str] = None, col_scale=None) -> EpilogueT:
    """tc_epilogue for output c: bias is a GPU tensor of c's dtype and
    col_scale a float32 GPU tensor, each holding N values per problem ([N],
    shared by a batch, or [batch, N] with contiguous rows); activation is
    None, "none", "relu" or "gelu_tanh"."""
    import torch
    ep = EpilogueT()
    act = "none" if activation is None else activation
    if act not in ACTIVATIONS:
        raise TcGemmError(1, "unknown activation %r" % (activation,))
    ep.activation = ACTIVATIONS[act]
    ep.bias, ep.bias_stride, ep.col_scale, ep.scale_stride = None, 0, None, 0
    if bias is not None:
        ep.bias, ep.bias_stride = _column_vector(c, bias, "bias", c.dtype)
    if col_scale is not None:
        ep.col_scale, ep.scale_stride = _column_vector(c, col_scale, "col_scale", torch.float32)
    return ep


# Descriptors of the shapes seen so far (a call rebuilds none: its fields
# depend only on the key), bounded.
_desc_cache: Dict[tuple, BatchedDescT] = {}


def _desc_of(a, b, c, alpha, beta, transpose_a, transpose_b):
    """The descriptor of a call and a ctypes reference to it, cached per
    (types, shapes, strides, scalars, transposes)."""
    key = (a.dtype, b.dtype, c.dtype, a.shape, b.shape, c.shape, a.stride(), b.stride(),
           c.stride(), alpha, beta, transpose_a, transpose_b)
    d = _desc_cache.get(key)
    if d is None:
        desc = make_desc(a, b, c, alpha, beta, transpose_a, transpose_b)
        d = (desc, ctypes.byref(desc))
        if len(_desc_cache) < 4096:
            _desc_cache[key] = d
    return d


def gemm(a, b, c, *, alpha: float = 1.0, beta: float = 0.0, transpose_a: bool = False,
         transpose_b: bool = False, stream=None, bias=None, activation: Optional[str] = None,
         col_scale=None):
    """c = activation(alpha * (op(a) @ op(b)) * col_scale + beta * c + bias) on
    c's device, enqueued on torch's current stream (or `stream`).  Without
    bias, activation and col_scale this is the plain product
    (tc_gemm_batched_async), with any of them the fused epilogue
    (tc_gemm_epilogue_async); int8 a and b with a float c need col_scale
    (per-column dequantization).  Returns c."""
    if not (a.is_cuda and b.is_cuda and c.is_cuda):
        raise TcGemmError(1, "a, b and c must be GPU tensors")
    device = c.get_device()
    desc, dref = _desc_of(a, b, c, alpha, beta, transpose_a, transpose_b)
    lib = _lib if _lib is not None else load_library()
    ctx, s = _torch_stream(device, stream)
    if bias is None and activation is None and col_scale is None:
        st = lib.tc_gemm_batched_async(ctx, dref, a.data_ptr(), b.data_ptr(), c.data_ptr(), s)
    else:
        ep = make_epilogue(c, bias, activation, col_scale)
        st = lib.tc_gemm_epilogue_async(ctx, dref, ctypes.byref(ep), a.data_ptr(), b.data_ptr(),
                                        c.data_ptr(), s)
    if st != 0:
        _check(st, ctx)
    return c


# ------------------------------------------------------------------ weights in 4 bits
class _W4Arrays(NamedTuple):
    codes: "torch.Tensor"
    scales: "torch.Tensor"
    zeros: "Optional[torch.Tensor]" = None


class W4Weight(_W4Arrays):
    """Matrices held in 4 bits with a scale (and zero point) per group of K
    (the layout is in include/tcgemm.h): codes uint8 [.., ceil(N/16),
    ceil(K/128), 1024], scales f16 or bf16 [.., ceil(N/16), ceil(K/128), 16,
    128/group], zeros uint8 of the scales' shape or None.  Contiguous; the
    leading dims, if any, count matrices.  Functions that take one accept a
    plain tuple of the three (or two) too.  N and K, the matrices' own sizes,
    are known where w4_quantize or w4_pack made the weight or the constructor
    was told them, else None."""
    N: Optional[int] = None
    K: Optional[int] = None

    def __new__(cls, codes, scales, zeros=None, *, N: Optional[int] = None, K: Optional[int] = None):
        self = super().__new__(cls, codes, scales, zeros)
        if N is not None:
            self.N = int(N)
        if K is not None:
            self.K = int(K)
        return self


def _float_code(t, name: str, types=(F32, F16, BF16)) -> int:
    code = _dtype_code(t)
    if code not in types:
        raise TcGemmError(2, "%s must be one of %s (got %s)"
                          % (name, "/".join(_NAMES[c] for c in types), _NAMES[code]))
    return code


def _same_device(first, *others) -> int:
    """The device index all tensors share."""
    if not first.is_cuda:
        raise TcGemmError(1, "the operands must be GPU tensors")
    device = first.get_device()
    for t in others:
        if t is not None and (not t.is_cuda or t.get_device() != device):
            raise TcGemmError(1, "the operands must be on one GPU")
    return device


# Descriptors of the calls seen so far, as _desc_cache, bounded.
_op_cache: Dict[tuple, tuple] = {}


def _cached(key, make):
    v = _op_cache.get(key)
    if v is None:
        v = make()
        if len(_op_cache) < 4096:
            _op_cache[key] = v
    return v


def _w4_desc(w, N: int, K: int, lead=()):
    """tc_qweight_desc of w, checked to hold matrices [N, K], one per index
    of the leading shape `lead`."""
    codes, scales, zeros = w
    import torch
    nb, kb = (N + 15) // 16, (K + 127) // 128
    per = int(scales.size(-1)) if scales.dim() else 0
    if per not in (1, 2, 4):
        raise TcGemmError(1, "the scales' last dimension must be 128/group: 1, 2 or 4 (got %d)" % per)
    lead = tuple(lead)
    if codes.dtype != torch.uint8 or tuple(codes.shape) != lead + (nb, kb, 1024):
        raise TcGemmError(1, "codes must be uint8 of shape %s (got %s %s)"
                          % (lead + (nb, kb, 1024), codes.dtype, tuple(codes.shape)))
    if tuple(scales.shape) != lead + (nb, kb, 16, per):
        raise TcGemmError(1, "scales must have shape %s (got %s)"
                          % (lead + (nb, kb, 16, per), tuple(scales.shape)))
    if zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != scales.shape):
        raise TcGemmError(1, "zeros must be uint8 of the scales' shape")
    if not (codes.is_contiguous() and scales.is_contiguous()
            and (zeros is None or zeros.is_contiguous())):
        raise TcGemmError(1, "codes, scales and zeros must be contiguous")
    batch = 1
    for n in lead:
        batch *= n
    return QWeightDescT(*_i32(batch=batch, N=N, K=K), 128 // per, _float_code(scales, "scales", (F16, BF16)),
                        zeros is not None)


def _w4_ptrs(w) -> QWeightT:
    codes, scales, zeros = w
    return QWeightT(codes.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr())


def _w4_key(w) -> tuple:
    codes, scales, zeros = w
    return (codes.shape, codes.dtype, codes.is_contiguous(), scales.shape, scales.dtype,
            scales.is_contiguous(), None if zeros is None else
            (zeros.shape, zeros.dtype, zeros.is_contiguous()))


def _as_w4(w):
    """(codes, scales, zeros) of a W4Weight or a tuple of two or three."""
    if not isinstance(w, (tuple, list)) or len(w) not in (2, 3):
        raise TcGemmError(1, "the weight must be (codes, scales, zeros or None)")
    return tuple(w) if len(w) == 3 else (w[0], w[1], None)


def _on_stream(device: int, stream):
    """Context under which torch allocates for the stream a call runs on."""
    import torch
    return torch.cuda.stream(stream) if stream is not None else torch.cuda.device(device)


def _w4_new(lead, N: int, K: int, group: int, zeros: bool, scale_dtype):
    """Descriptor of a new W4Weight, a reference to it, the shapes of its
    arrays, N and K."""
    import torch
    if group not in (32, 64, 128):
        raise TcGemmError(1, "group must be 32, 64 or 128 (got %r)" % (group,))
    batch = 1
    for n in lead:
        batch *= n
    nb, kb = (N + 15) // 16, (K + 127) // 128
    code = F16 if scale_dtype is torch.float16 else BF16
    d = QWeightDescT(*_i32(batch=batch, N=N, K=K), group, code, zeros)
    return d, ctypes.byref(d), (*lead, nb, kb, 1024), (*lead, nb, kb, 16, 128 // group), N, K


def _w4_empty(new, zeros: bool, scale_dtype, where, device: int, stream) -> W4Weight:
    import torch
    if stream is not None:
        with _on_stream(device, stream):
            return _w4_empty(new, zeros, scale_dtype, where, device, None)
    return W4Weight(torch.empty(new[2], dtype=torch.uint8, device=where),
                    torch.empty(new[3], dtype=scale_dtype, device=where),
                    torch.empty(new[3], dtype=torch.uint8, device=where) if zeros else None,
                    N=new[4], K=new[5])


def _pitch(t, name: str) -> int:
    """_ld of a tensor whose rows are apart: 0, which a broadcast tensor has,
    means contiguous to the library."""
    ld = _ld(t)
    if ld == 0 and t.size(-2) > 1:
        raise TcGemmError(1, "the rows of %s must not be broadcast" % name)
    return ld


def _dense_batch(t, name: str):
    """(leading shape, N, K, row pitch, matrix stride) of a [.., N, K] tensor
    whose matrices are evenly spaced."""
    if t.dim() < 2:
        raise TcGemmError(1, "%s must have at least 2 dimensions" % name)
    lead, N, K = tuple(t.shape[:-2]), int(t.size(-2)), int(t.size(-1))
    ld = _pitch(t, name)
    stride, expect = 0, None
    for d in range(len(lead) - 1, -1, -1):
        if lead[d] == 1:
            continue
        if expect is None:
            stride = int(t.stride(d))
            if stride == 0:
                raise TcGemmError(1, "the matrices of %s must not be broadcast" % name)
        elif int(t.stride(d)) != expect:
            raise TcGemmError(1, "the matrices of %s must be evenly spaced" % name)
        expect = int(t.stride(d)) * lead[d]
    return lead, N, K, ld, stride


def _make_quantize(w, group, zeros, scale_dtype):
    import torch
    code = _float_code(w, "w")
    if scale_dtype is None:
        scale_dtype = torch.bfloat16 if code == F32 else w.dtype
    if scale_dtype not in (torch.float16, torch.bfloat16):
        raise TcGemmError(2, "scale_dtype must be torch.float16 or torch.bfloat16")
    lead, N, K, ld, stride = _dense_batch(w, "w")
    if w.numel() == 0:
        raise TcGemmError(1, "dims must be >= 1 (shape %s)" % (tuple(w.shape),))
    return _w4_new(lead, N, K, group, zeros, scale_dtype), code, ld, stride, scale_dtype


def w4_quantize(w, *, group: int = 128, zeros: bool = False, scale_dtype=None, stream=None) -> W4Weight:
    """w [.., N, K] (f32, f16 or bf16) in 4 bits, with a scale per `group`
    values of K (32, 64 or 128) and, with zeros, a zero point
    (tc_quantize_async has the formulas).  scale_dtype: torch.float16 or
    torch.bfloat16, the type of the activations it will meet; by default w's,
    bfloat16 for f32."""
    device = _same_device(w)
    zeros = bool(zeros)
    key = ("quantize", w.shape, w.stride(), w.dtype, group, zeros, scale_dtype)
    new, code, ld, stride, scale_dtype = _cached(key, lambda: _make_quantize(w, group, zeros, scale_dtype))
    lib = _lib if _lib is not None else load_library()
    ctx, s = _torch_stream(device, stream)
    out = _w4_empty(new, zeros, scale_dtype, w.device, device, stream)
    q = _w4_ptrs(out)
    st = lib.tc_quantize_async(ctx, new[1], w.data_ptr(), code, ld, stride, ctypes.byref(q), s)
    if st != 0:
        _check(st, ctx)
    return out


def _make_dequantize(w, out):
    code = _float_code(out, "out")
    lead, N, K, ld, stride = _dense_batch(out, "out")
    d = _w4_desc(w, N, K, lead)
    return d, ctypes.byref(d), code, ld, stride


def w4_dequantize(w, out, *, stream=None):
    """The values a W4Weight stands for into out [.., N, K] (f32, f16 or
    bf16), rounded once.  Returns out."""
    w = _as_w4(w)
    device = _same_device(out, *w)
    key = ("dequantize", out.shape, out.stride(), out.dtype, _w4_key(w))
    _, d, code, ld, stride = _cached(key, lambda: _make_dequantize(w, out))
    lib = _lib if _lib is not None else load_library()
    ctx, s = _torch_stream(device, stream)
    q = _w4_ptrs(w)
    st = lib.tc_dequantize_async(ctx, d, ctypes.byref(q), out.data_ptr(), code, ld, stride, s)
    if st != 0:
        _check(st, ctx)
    return out


def w4_pack(codes, scales, zeros=None, *, K: Optional[int] = None, group: int = 128,
            stream=None) -> W4Weight:
    """Lay out what another quantizer made: codes uint8 [.., N, ceil(K/2)],
    two per byte, the even k in the low nibble; scales f16 or bf16 and zeros
    uint8 [.., N, ceil(K/group)]; all contiguous.  W = scale * (code - zero),
    zero 8 without zeros.  K: by default twice the codes' last dimension."""
    import torch
    device = _same_device(codes, scales, zeros)
    _float_code(scales, "scales", (F16, BF16))
    if codes.dim() < 2 or codes.dtype != torch.uint8 or codes.numel() == 0:
        raise TcGemmError(1, "codes must be uint8 [.., N, ceil(K/2)]")
    lead, N = tuple(codes.shape[:-2]), int(codes.size(-2))
    K = 2 * int(codes.size(-1)) if K is None else int(K)
    if group not in (32, 64, 128):
        raise TcGemmError(1, "group must be 32, 64 or 128 (got %r)" % (group,))
    if (K + 1) // 2 != codes.size(-1):
        raise TcGemmError(1, "K=%d does not fit %d bytes of codes per row" % (K, codes.size(-1)))
    shape = lead + (N, (K + group - 1) // group)
    if tuple(scales.shape) != shape:
        raise TcGemmError(1, "scales must have shape %s (got %s)" % (shape, tuple(scales.shape)))
    if zeros is not None and (zeros.dtype != torch.uint8 or tuple(zeros.shape) != shape):
        raise TcGemmError(1, "zeros must be uint8 of the scales' shape")
    if not all(t is None or t.is_contiguous() for t in (codes, scales, zeros)):
        raise TcGemmError(1, "codes, scales and zeros must be contiguous")
    ctx, s = _torch_stream(device, stream)
    new = _w4_new(lead, N, K, group, zeros is not None, scales.dtype)
    out = _w4_empty(new, zeros is not None, scales.dtype, codes.device, device, stream)
    q, src = _w4_ptrs(out), _w4_ptrs((codes, scales, zeros))
    _check(load_library().tc_qweight_pack_async(ctx, new[1], ctypes.byref(src), ctypes.byref(q), s), ctx)
    return out


def _make_qgemm(x, w, y, alpha, beta):
    if x.dim() != 2 or y.dim() != 2 or x.size(0) != y.size(0):
        raise TcGemmError(1, "x must be [M, K] and y [M, N] (got %s and %s)"
                          % (tuple(x.shape), tuple(y.shape)))
    wd = _w4_desc(w, int(y.size(1)), int(x.size(1)))
    M, ldx, ldy = _i32(M=int(x.size(0)), ldx=_pitch(x, "x"), ldy=_pitch(y, "y"))
    g = QGemmDescT(M, _dtype_code(x), _dtype_code(y), float(alpha), float(beta), ldx, ldy)
    return g, wd, ctypes.byref(g), ctypes.byref(wd)


def w4_gemm(x, w, y, *, alpha: float = 1.0, beta: float = 0.0, bias=None,
            activation: Optional[str] = None, stream=None):
    """y = activation(alpha * (x @ W^T) + beta * y + bias) for a weight held
    in 4 bits: x [M, K] of the scales' type, W [N, K] as a W4Weight, y [M, N]
    of x's type or f32, bias [N] of y's type; activation None, "none", "relu"
    or "gelu_tanh".  Runs on torch's current stream (or `stream`), needs no
    workspace.  Returns y."""
    codes, scales, zeros = w = _as_w4(w)
    # (numbers: a tensor as a key would keep the value of its first call)
    alpha, beta = float(alpha), float(beta)
    device = y.get_device()
    if (device < 0 or x.get_device() != device or codes.get_device() != device
            or scales.get_device() != device
            or (zeros is not None and zeros.get_device() != device)
            or (bias is not None and bias.get_device() != device)):
        raise TcGemmError(1, "the operands must be on one GPU")
    key = (x.shape, x.stride(), x.dtype, y.shape, y.stride(), y.dtype, alpha, beta, codes.shape,
           codes.dtype, codes.is_contiguous(), scales.shape, scales.dtype, scales.is_contiguous(),
           None if zeros is None else (zeros.shape, zeros.dtype, zeros.is_contiguous()))
    d = _op_cache.get(key)
    if d is None:
        d = _cached(key, lambda: _make_qgemm(x, w, y, alpha, beta))
    g, wd = d[2], d[3]
    lib = _lib if _lib is not None else load_library()
    ctx, s = _torch_stream(device, stream)
    q = _w4_ptrs(w)
    ep = None
    if bias is not None or activation not in (None, "none"):
        ep = ctypes.byref(make_epilogue(y, bias, activation))
    st = lib.tc_qgemm_async(ctx, g, wd, x.data_ptr(), ctypes.byref(q), y.data_ptr(), ep, s)
    if st != 0:
        _check(st, ctx)
    return y


# ------------------------------------------------------------------ mixture of experts
def _make_route(logits, top_k, renormalize, scale):
    if logits.dim() != 2:
        raise TcGemmError(1, "logits must be [T, E] (got %s)" % (tuple(logits.shape),))
    T, E, k, ld = _i32(T=int(logits.size(0)), E=int(logits.size(1)), top_k=int(top_k),
                       ld=_pitch(logits, "the logits"))
    r = RouteDescT(T, E, k, _dtype_code(logits), ld, bool(renormalize), float(scale))
    return r, ctypes.byref(r)


def moe_route(logits, top_k: int, *, renormalize: bool = True, scale: float = 1.0, stream=None):
    """(ids int32 [T, top_k], weights f32 [T, top_k]): the experts with the
    largest of the router's logits [T, E] (f32, f16 or bf16), the largest
    first, ties to the lowest index, and scale times their softmax weights,
    over the chosen ones (renormalize) or over all E.  Experts whose logit is
    -inf or NaN are never chosen; places left over hold id -1, weight 0.  Not
    recorded by autograd: moe_route_backward has the weights' gradient."""
    import torch
    device = _same_device(logits)
    if not (isinstance(top_k, int) and top_k >= 1):
        raise TcGemmError(1, "top_k must be a whole number >= 1 (got %r)" % (top_k,))
    renormalize, scale = bool(renormalize), float(scale)
    key = ("route", logits.shape, logits.stride(), logits.dtype, top_k, renormalize, scale)
    d, r = _cached(key, lambda: _make_route(logits, top_k, renormalize, scale))
    lib = _lib if _lib is not None else load_library()
    ctx, s = _torch_stream(device, stream)
    shape, where = (d.T, d.top_k), logits.device
    if stream is None:
        ids = torch.empty(shape, dtype=torch.int32, device=where)
        weights = torch.empty(shape, dtype=torch.float32, device=where)
    else:
        with _on_stream(device, stream):
            ids = torch.empty(shape, dtype=torch.int32, device=where)
            weights = torch.empty(shape, dtype=torch.float32, device=where)
    st = lib.tc_moe_route_async(ctx, r, logits.data_ptr(), ids.data_ptr(), weights.data_ptr(), s)
    if st != 0:
        _check(st, ctx)
    return ids, weights


def _make_moe(x, route, gate_up, down, y, top_k, activation, renormalize, scale, intermediate):
    import torch
    if activation not in GATES:
        raise TcGemmError(1, "unknown activation %r" % (activation,))
    if x.dim() != 2 or x.shape != y.shape:
        raise TcGemmError(1, "x and y must be [T, H] (got %s and %s)" % (tuple(x.shape), tuple(y.shape)))
    T, H = int(x.size(0)), int(x.size(1))
    held = isinstance(gate_up, tuple)
    if held != isinstance(down, tuple):
        raise TcGemmError(2, "gate_up and down must both be held in 4 bits or both in 16")
    if held:
        if down[0].dim() != 4 or gate_up[0].dim() != 5:
            raise TcGemmError(1, "gate_up must hold [E, 2] matrices and down [E]")
        E = int(down[0].size(0))
        I = 16 * int(gate_up[0].size(2)) if intermediate is None else int(intermediate)
        up, dn = _w4_desc(gate_up, I, H, (E, 2)), _w4_desc(down, H, I, (E,))
        if (up.group, up.has_zeros, up.scale_dtype) != (dn.group, dn.has_zeros, dn.scale_dtype):
            raise TcGemmError(2, "gate_up and down must be held alike")
        if up.scale_dtype != _dtype_code(x):
            raise TcGemmError(2, "the scales must have x's dtype %s" % x.dtype)
        group, zeros = up.group, up.has_zeros
    else:
        if down.dim() != 3 or gate_up.dim() not in (3, 4):
            raise TcGemmError(1, "gate_up must be [E, 2, I, H] or [E, 2 I, H], down [E, H, I]")
        E, I = int(down.size(0)), int(down.size(2))
        if (tuple(gate_up.shape) not in ((E, 2, I, H), (E, 2 * I, H)) or int(down.size(1)) != H
                or intermediate not in (None, I)):
            raise TcGemmError(1, "shapes of gate_up %s, down %s and x %s do not fit"
                              % (tuple(gate_up.shape), tuple(down.shape), tuple(x.shape)))
        if gate_up.dtype != x.dtype or down.dtype != x.dtype:
            raise TcGemmError(2, "gate_up and down must have x's dtype %s" % x.dtype)
        if not (gate_up.is_contiguous() and down.is_contiguous()):
            raise TcGemmError(1, "gate_up and down must be contiguous")
        group, zeros = 0, False
    r = rref = None
    if isinstance(route, tuple):
        ids, weights = route
        if top_k is not None and int(top_k) != int(ids.size(-1)):
            raise TcGemmError(1, "top_k=%d, but ids have %d columns" % (top_k, ids.size(-1)))
        k = int(ids.size(-1))
        if (tuple(ids.shape) != (T, k) or weights.shape != ids.shape or ids.dtype != torch.int32
                or weights.dtype != torch.float32):
            raise TcGemmError(1, "ids must be int32 and weights float32 [T, top_k]")
        if not (ids.is_contiguous() and weights.is_contiguous()):
            raise TcGemmError(1, "ids and weights must be contiguous")
    else:
        if top_k is None:
            raise TcGemmError(1, "top_k must be given with logits")
        k = int(top_k)
        if tuple(route.shape) != (T, E):
            raise TcGemmError(1, "logits must be [T, E] = %s (got %s)" % ((T, E), tuple(route.shape)))
        r, rref = _make_route(route, k, renormalize, scale)
    d = MoeDescT(*_i32(T=T, H=H, I=I, E=E, top_k=k), _dtype_code(x), _dtype_code(y),
                 *_i32(ldx=_pitch(x, "x"), ldy=_pitch(y, "y")), GATES[activation], group, zeros)
    need = ctypes.c_int64()
    st = load_library().tc_moe_workspace(ctypes.byref(d), ctypes.byref(need))
    # (a descriptor the library refuses is refused again, with its text, by the call)
    return d, ctypes.byref(d), r, rref, need.value if st == 0 else 0


def _intermediate(gate_up, down) -> Optional[int]:
    """The intermediate size that 4-bit experts know of themselves: gate_up's
    rows, down's columns; None where neither knows."""
    rows, cols = getattr(gate_up, "N", None), getattr(down, "K", None)
    if rows is not None and cols is not None and rows != cols:
        raise TcGemmError(1, "gate_up has %d rows and down %d columns" % (rows, cols))
    return cols if rows is None else rows


def _weights_key(w) -> tuple:
    return _w4_key(w) if isinstance(w, tuple) else (w.shape, w.dtype, w.is_contiguous())


def moe(x, route, gate_up, down, y, *, top_k: Optional[int] = None, activation: str = "silu",
        renormalize: bool = True, scale: float = 1.0, intermediate: Optional[int] = None,
        stream=None):
    """A layer of gated experts for few tokens (tc_moe_async):

        y[t] = sum_j p[t, j] * down[e] (act(gate[e] x[t]) * (up[e] x[t])),  e = ids[t, j]

    x and y [T, H], y of x's type or f32.  route: the router's logits [T, E]
    (then top_k, renormalize and scale choose as moe_route does) or a tuple
    (ids int32, weights float32), both [T, top_k]; an id outside [0, E) adds
    nothing.  gate_up [E, 2, I, H] (gate, then up; [E, 2 I, H] is the same
    memory) and down [E, H, I]: tensors of x's type, or both in 4 bits
    (W4Weight of leading shapes (E, 2) and (E,)); then I is `intermediate`,
    by default the size that one of the weights knows (W4Weight.N, .K).  Plain
    tuples know none: without `intermediate` they are taken to hold whole
    blocks of 16 rows, all of them used.  activation: "silu" or
    "gelu_tanh".  Scratch memory comes from torch's allocator, for this call
    alone.  Returns y."""
    import torch
    if isinstance(gate_up, (tuple, list)):
        if intermediate is None:
            intermediate = _intermediate(gate_up, down)
        gate_up = _as_w4(gate_up)
    if isinstance(down, (tuple, list)):
        down = _as_w4(down)
    held = gate_up if isinstance(gate_up, tuple) else (gate_up,)
    held = held + (down if isinstance(down, tuple) else (down,))
    given = tuple(route) if isinstance(route, (tuple, list)) else (route,)
    if isinstance(route, (tuple, list)):
        if len(given) != 2:
            raise TcGemmError(1, "route must be logits or (ids, weights)")
        route = given
    device = _same_device(y, x, *given, *held)
    renormalize, scale = bool(renormalize), float(scale)
    top_k = None if top_k is None else int(top_k)
    intermediate = None if intermediate is None else int(intermediate)
    key = ("moe", x.shape, x.stride(), x.dtype, y.shape, y.stride(), y.dtype,
           tuple((g.shape, g.stride(), g.dtype) for g in given), _weights_key(gate_up),
           _weights_key(down), top_k, activation, renormalize, scale, intermediate)
    _, d, _, r, need = _cached(key, lambda: _make_moe(x, route, gate_up, down, y, top_k, activation,
                                                      renormalize, scale, intermediate))
    lib = _lib if _lib is not None else load_library()
    ctx, s = _torch_stream(device, stream)
    if stream is None:
        space = torch.empty(need, dtype=torch.uint8, device=y.device)
    else:
        with _on_stream(device, stream):
            space = torch.empty(need, dtype=torch.uint8, device=y.device)
    up = _w4_ptrs(gate_up) if isinstance(gate_up, tuple) else QWeightT(gate_up.data_ptr(), None, None)
    dn = _w4_ptrs(down) if isinstance(down, tuple) else QWeightT(down.data_ptr(), None, None)
    if len(given) == 2:
        logits, ids, weights = None, given[0].data_ptr(), given[1].data_ptr()
    else:
        logits, ids, weights = given[0].data_ptr(), None, None
    st = lib.tc_moe_async(ctx, d, x.data_ptr(), r, logits, ids, weights, ctypes.byref(up),
                          ctypes.byref(dn), y.data_ptr(), space.data_ptr(), need, s)
    if st != 0:
        _check(st, ctx)
    return y


# ------------------------------------------------------------------ losses
def _scratch(need: int, like, device: int, stream):
    """Scratch memory for one call on the stream it runs on."""
    import torch
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    with _on_stream(device, stream):
        return torch.empty(need, dtype=torch.uint8, device=like.device)


def _new(shapes, like, device: int, stream):
    """New tensors of the given (shape, dtype)s, made for the stream a call
    runs on."""
    import torch
    empty, where = torch.empty, like.device
    if stream is None:
        return [empty(shape, dtype=dtype, device=where) for shape, dtype in shapes]
    with _on_stream(device, stream):
        return [empty(shape, dtype=dtype, device=where) for shape, dtype in shapes]


def _make_ce(x, weight, targets, scale):
    import torch
    if x.dim() != 2 or weight.dim() != 2 or x.size(1) != weight.size(1):
        raise TcGemmError(1, "x must be [T, H] and the weight [V, H] (got %s and %s)"
                          % (tuple(x.shape), tuple(weight.shape)))
    code = _float_code(x, "x")
    if weight.dtype != x.dtype:
        raise TcGemmError(2, "the weight must have x's dtype %s (got %s)" % (x.dtype, weight.dtype))
    if targets.dtype not in (torch.int32, torch.int64):
        raise TcGemmError(2, "targets must be int32 or int64 (got %s)" % targets.dtype)
    T, V, H, ldx, ldw = _i32(T=int(x.size(0)), V=int(weight.size(0)), H=int(x.size(1)),
                             ldx=_pitch(x, "x"), ldw=_pitch(weight, "the weight"))
    if tuple(targets.shape) != (T,) or not targets.is_contiguous():
        raise TcGemmError(1, "targets must be [T] = [%d], contiguous (got %s)" % (T, tuple(targets.shape)))
    return CeDescT(T, V, H, code, ldx, ldw, targets.dtype == torch.int64, scale)


def _make_ce_forward(x, weight, targets, scale):
    d = _make_ce(x, weight, targets, scale)
    need = ctypes.c_int64()
    st = load_library().tc_cross_entropy_workspace(ctypes.byref(d), x.data_ptr(), weight.data_ptr(),
                                                   ctypes.byref(need))
    # (a descriptor the library refuses is refused again, with its text, by the call)
    return d, ctypes.byref(d), need.value if st == 0 else 0


def _ce_key(x, weight, targets) -> tuple:
    return (x.shape, x.stride(), x.dtype, x.data_ptr() % 16, weight.shape, weight.stride(), weight.dtype,
            weight.data_ptr() % 16, targets.shape, targets.stride(), targets.dtype)


def cross_entropy(x, weight, targets, *, scale: float = 1.0, stream=None):
    """(loss, lse), float32 [T]: the softmax cross entropy of the linear layer
    scale * (x @ weight^T) against targets, and the log of each token's sum of
    exponentials (tc_cross_entropy_async).  x [T, H] and weight [V, H], f32,
    f16 or bf16; targets [T] int32 or int64.  A token whose target is outside
    [0, V), -100 for instance, is ignored: its loss is 0.  The [T, V] products
    are not kept.  Scratch memory comes from torch's allocator, for this call
    alone.  Not recorded by autograd: the results never require grad, also where
    x or the weight does, and the caller passes on what cross_entropy_backward
    gives."""
    import torch
    device = _same_device(x, weight, targets)
    scale = float(scale)
    d, dref, need = _cached(("ce", scale) + _ce_key(x, weight, targets),
                            lambda: _make_ce_forward(x, weight, targets, scale))
    lib = _lib if _lib is not None else load_library()
    ctx, s = _torch_stream(device, stream)
    (loss, lse), space = _new([(d.T, torch.float32)] * 2, x, device, stream), _scratch(need, x, device, stream)
    st = lib.tc_cross_entropy_async(ctx, dref, x.data_ptr(), weight.data_ptr(), targets.data_ptr(),
                                    loss.data_ptr(), lse.data_ptr(), space.data_ptr(), need, s)
    if st != 0:
        _check(st, ctx)
    return loss, lse


def _make_ce_backward(x, weight, targets, lse, grad, dx, dweight, scale, beta):
    import torch
    d = _make_ce(x, weight, targets, scale)
    g = CeGradsT()
    if lse.dtype != torch.float32 or tuple(lse.shape) != (d.T,) or not lse.is_contiguous():
        raise TcGemmError(1, "lse must be float32 [T] = [%d], contiguous" % d.T)
    if grad.dtype != torch.float32 or tuple(grad.shape) not in ((), (1,), (d.T,)):
        raise TcGemmError(1, "grad must be float32, one number or [T] = [%d] (got %s %s)"
                          % (d.T, grad.dtype, tuple(grad.shape)))
    g.grad_stride = int(grad.stride(0)) if grad.numel() > 1 else 0
    for name, t, like in (("dx", dx, x), ("dweight", dweight, weight)):
        if t is not None and t.shape != like.shape:
            raise TcGemmError(1, "%s must be %s (got %s)" % (name, tuple(like.shape), tuple(t.shape)))
    if dx is not None:
        g.dx_dtype, (g.lddx,) = _float_code(dx, "dx"), _i32(lddx=_pitch(dx, "dx"))
    if dweight is not None:
        g.dw_dtype, (g.lddw,) = _float_code(dweight, "dweight"), _i32(lddw=_pitch(dweight, "dweight"))
    g.beta = beta
    # (any address of the right alignment: the size does not depend on more)
    g.grad = 16
    g.dx, g.dw = (None if dx is None else dx.data_ptr()), (None if dweight is None else dweight.data_ptr())
    need = ctypes.c_int64()
    st = load_library().tc_cross_entropy_backward_workspace(ctypes.byref(d), ctypes.byref(g), x.data_ptr(),
                                                            weight.data_ptr(), ctypes.byref(need))
    return d, ctypes.byref(d), g, need.value if st == 0 else 0


def cross_entropy_backward(x, weight, targets, lse, grad, dx=None, dweight=None, *, scale: float = 1.0,
                           beta: float = 0.0, stream=None):
    """The gradients of cross_entropy's losses (tc_cross_entropy_backward_async):
    dx [T, H] and dweight = beta * dweight + .. [V, H], either one None or of
    x's type or f32.  lse: what cross_entropy returned for the same x, weight
    and scale; grad float32: the losses' gradient, [T] of any stride or one
    number for all of them.  Ignored tokens add nothing to dweight and have
    dx = 0.  An f32 gradient from 16-bit inputs is as exact as fp32 sums and
    takes two or three times the products, which are stored on the way; one in
    x's type comes from softmax gradients that are rounded to it.  Returns (dx,
    dweight)."""
    outs = [t for t in (dx, dweight) if t is not None]
    if not outs:
        raise TcGemmError(1, "dx and dweight must not both be None")
    device = _same_device(x, weight, targets, lse, grad, *outs)
    scale, beta = float(scale), float(beta)
    key = ("ceb", scale, beta, lse.shape, lse.stride(), lse.dtype, grad.shape, grad.stride(), grad.dtype,
           None if dx is None else (dx.shape, dx.stride(), dx.dtype),
           None if dweight is None else (dweight.shape, dweight.stride(), dweight.dtype))
    _, dref, made, need = _cached(key + _ce_key(x, weight, targets),
                                  lambda: _make_ce_backward(x, weight, targets, lse, grad, dx, dweight, scale,
                                                            beta))
    # (a copy: threads may share the cached one)
    g = CeGradsT.from_buffer_copy(made)
    g.grad = grad.data_ptr()
    g.dx, g.dw = (None if dx is None else dx.data_ptr()), (None if dweight is None else dweight.data_ptr())
    lib = _lib if _lib is not None else load_library()
    ctx, s = _torch_stream(device, stream)
    space = _scratch(need, x, device, stream)
    st = lib.tc_cross_entropy_backward_async(ctx, dref, ctypes.byref(g), x.data_ptr(), weight.data_ptr(),
                                             targets.data_ptr(), lse.data_ptr(), space.data_ptr(), need, s)
    if st != 0:
        _check(st, ctx)
    return dx, dweight


def _make_balance(logits, ids):
    import torch
    if ids.dim() != 2 or ids.dtype != torch.int32 or not ids.is_contiguous():
        raise TcGemmError(1, "ids must be int32 [T, top_k], contiguous")
    r, rref = _make_route(logits, int(ids.size(1)), True, 1.0)
    if int(ids.size(0)) != r.T:
        raise TcGemmError(1, "ids must have a row per token: %d (got %d)" % (r.T, ids.size(0)))
    need = ctypes.c_int64()
    st = load_library().tc_moe_balance_workspace(rref, ctypes.byref(need))
    return r, rref, need.value if st == 0 else 0


def moe_balance(logits, ids, *, coef: float = 1.0, stream=None):
    """(loss float32 [], counts int32 [E], slope float32 [E]): the balance loss
    of a router, coef * E * sum_e (share of the choices)[e] * (mean
    probability)[e], the choices of each expert, and what moe_route_backward
    needs for its gradient (tc_moe_balance_async has the formulas).  logits [T,
    E] f32, f16 or bf16; ids int32 [T, top_k] as moe_route gives them; a token
    with no id inside [0, E), padding for instance, does not count.  Not recorded
    by autograd: moe_route_backward has the gradient."""
    import torch
    device = _same_device(logits, ids)
    r, rref, need = _cached(("balance", logits.shape, logits.stride(), logits.dtype, ids.shape, ids.stride(),
                             ids.dtype), lambda: _make_balance(logits, ids))
    lib = _lib if _lib is not None else load_library()
    ctx, s = _torch_stream(device, stream)
    loss, counts, slope = _new([((), torch.float32), (r.E, torch.int32), (r.E, torch.float32)], logits, device,
                               stream)
    space = _scratch(need, logits, device, stream) if need else None
    st = lib.tc_moe_balance_async(ctx, rref, logits.data_ptr(), ids.data_ptr(), float(coef), loss.data_ptr(),
                                  counts.data_ptr(), slope.data_ptr(), space.data_ptr() if need else None, need, s)
    if st != 0:
        _check(st, ctx)
    return loss, counts, slope


def _make_route_backward(logits, ids, dweights, dlogits, renormalize, scale, slope, dloss):
    import torch
    if ids.dim() != 2 or ids.dtype != torch.int32 or not ids.is_contiguous():
        raise TcGemmError(1, "ids must be int32 [T, top_k], contiguous")
    r, rref = _make_route(logits, int(ids.size(1)), renormalize, scale)
    if int(ids.size(0)) != r.T:
        raise TcGemmError(1, "ids must have a row per token: %d (got %d)" % (r.T, ids.size(0)))
    if dweights is not None and (dweights.dtype != torch.float32 or dweights.shape != ids.shape
                                 or not dweights.is_contiguous()):
        raise TcGemmError(1, "dweights must be float32 of ids' shape %s, contiguous" % (tuple(ids.shape),))
    if (slope is None) != (dloss is None):
        raise TcGemmError(1, "slope and dloss go together")
    if slope is not None:
        if slope.dtype != torch.float32 or tuple(slope.shape) != (r.E,) or not slope.is_contiguous():
            raise TcGemmError(1, "slope must be float32 [E] = [%d], contiguous" % r.E)
        if dloss.dtype != torch.float32 or dloss.numel() != 1:
            raise TcGemmError(1, "dloss must be one float32 number")
    if dlogits.shape != logits.shape:
        raise TcGemmError(1, "dlogits must be %s (got %s)" % (tuple(logits.shape), tuple(dlogits.shape)))
    code = _float_code(dlogits, "dlogits")
    ldd, = _i32(ldd=_pitch(dlogits, "dlogits"))
    return r, rref, code, ldd


def moe_route_backward(logits, ids, dweights, dlogits, *, renormalize: bool = True, scale: float = 1.0,
                       slope=None, dloss=None, stream=None):
    """The gradient of a router's logits into dlogits [T, E] (of the logits'
    type or f32), in one pass (tc_moe_route_backward_async): through the
    weights that moe_route gave for ids with the same renormalize and scale,
    whose gradient is dweights (float32 [T, top_k], or None), and through
    moe_balance's loss, with its slope and the loss's gradient dloss (one
    float32 number on the GPU), or neither.  Returns dlogits."""
    device = _same_device(logits, ids, dweights, dlogits, slope, dloss)
    renormalize, scale = bool(renormalize), float(scale)
    sig = lambda t: None if t is None else (t.shape, t.stride(), t.dtype)  # noqa: E731
    _, rref, code, ldd = _cached(
        ("routeb", sig(logits), sig(ids), sig(dweights), sig(dlogits), renormalize, scale, sig(slope),
         sig(dloss)),
        lambda: _make_route_backward(logits, ids, dweights, dlogits, renormalize, scale, slope, dloss))
    lib = _lib if _lib is not None else load_library()
    ctx, s = _torch_stream(device, stream)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = lib.tc_moe_route_backward_async(ctx, rref, logits.data_ptr(), ids.data_ptr(), ptr(dweights),
                                         ptr(slope), ptr(dloss), dlogits.data_ptr(), code, ldd, s)
    if st != 0:
        _check(st, ctx)
    return dlogits


def gemm_sync(a, b, c, *, alpha: float = 1.0, beta: float = 0.0, transpose_a: bool = False,
              transpose_b: bool = False):
    """Synchronous form: runs on the library context's own stream after
    synchronizing the device, and returns when c holds the result."""
    import torch
    device = c.device.index if c.device.index is not None else 0
    desc = make_desc(a, b, c, alpha, beta, transpose_a, transpose_b)
    torch.cuda.synchronize(device)
    lib = load_library()
    ctx = _context(device)
    with torch.cuda.device(device):
        st = lib.tc_gemm_batched(ctx, ctypes.byref(desc), _VP(a.data_ptr()), _VP(b.data_ptr()),
                                 _VP(c.data_ptr()))
    _check(st, ctx)
    return c


def set_autotune(enable: bool, device: int = 0) -> None:
    """Turn first-call autotuning on or off for the device's context (see
    tc_set_autotune)."""
    ctx = _context(device)
    _check(load_library().tc_set_autotune(ctx, int(bool(enable))), ctx)


def autotune_entries(device: int = 0) -> int:
    return int(load_library().tc_autotune_entries(_context(device)))


def plan(desc: BatchedDescT) -> dict:
    """Validate and plan a descriptor on the host (no GPU needed)."""
    lib = load_library()
    info = PlanInfoT()
    st = lib.tc_gemm_plan(None, ctypes.byref(desc), ctypes.byref(info))
    _check(st, None)
    out = {name: getattr(info, name) for name, _ in PlanInfoT._fields_}
    out["kernel"] = info.kernel.decode()
    return out
