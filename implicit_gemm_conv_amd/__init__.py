"""Python binding of libigc (include/igc.h): argument marshalling only.

Every function here forwards to the C entry point of the same name in
implicit_gemm_conv_amd/libigc.so and returns its igc_status_t as an int.
Tensor arguments may be torch tensors (their data_ptr() is passed) on the GPU
or in pinned memory -- others raise ValueError, since the GPU would fault on a
host address -- or plain integer device addresses.  `stream` defaults to
torch's current HIP stream.
All computation happens in the HIP kernels; there is no fallback: if the
library is not built, every call raises.

Build it with `python -m implicit_gemm_conv_amd.build` (or __graft_entry__.build()).
"""
import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libigc.so")

IGC_OK, IGC_ERR_INVALID_VALUE, IGC_ERR_MISALIGNED, IGC_ERR_UNSUPPORTED, IGC_ERR_HIP = range(5)
ROW_MAJOR, COL_MAJOR = 0, 1
OUT_F32, OUT_BF16, OUT_F16 = 0, 1, 2
OUT_CODES = {"f32": OUT_F32, "bf16": OUT_BF16, "f16": OUT_F16}
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)
ACT_CODES = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "silu": ACT_SILU}
OP_GEMM, OP_CONV_FPROP, OP_CONV_DGRAD, OP_CONV_WGRAD = range(4)

# Every exported entry point (include/igc.h), for the load check.
EXPORTS = (
    "gemm_bf16", "gemm_fp16", "gemm_bf16_ex", "gemm_fp16_ex", "gemm_bf16_noalloc",
    "conv2d_nhwc_implicit_gemm", "conv2d_nhwc_implicit_gemm_fp16", "conv2d_nhwc_implicit_gemm_ex",
    "conv2d_nhwc_implicit_gemm_fp16_ex",
    "conv2d_nhwc_dgrad_implicit_gemm", "conv2d_nhwc_dgrad_implicit_gemm_fp16", "conv2d_nhwc_dgrad_implicit_gemm_ex",
    "conv2d_nhwc_dgrad_implicit_gemm_fp16_ex",
    "conv2d_nhwc_wgrad_implicit_gemm", "conv2d_nhwc_wgrad_implicit_gemm_fp16", "conv2d_nhwc_wgrad_implicit_gemm_ex",
    "conv2d_nhwc_wgrad_implicit_gemm_fp16_ex",
    "gemm_bf16_epilogue", "gemm_fp16_epilogue", "gemm_bf16_epilogue_ex", "gemm_fp16_epilogue_ex",
    "conv2d_nhwc_implicit_gemm_epilogue", "conv2d_nhwc_implicit_gemm_epilogue_fp16",
    "conv2d_nhwc_implicit_gemm_epilogue_ex", "conv2d_nhwc_implicit_gemm_epilogue_fp16_ex",
    "igc_epilogue_workspace_bytes", "igc_epilogue_default_tune",
    "epilogue_backward_bf16", "epilogue_backward_fp16", "epilogue_backward_bf16_ex", "epilogue_backward_fp16_ex",
    "igc_epilogue_backward_workspace_bytes",
    "group_norm_nhwc_bf16", "group_norm_nhwc_fp16", "group_norm_nhwc_bf16_ex", "group_norm_nhwc_fp16_ex",
    "group_norm_nhwc_backward_bf16", "group_norm_nhwc_backward_fp16", "group_norm_nhwc_backward_bf16_ex",
    "group_norm_nhwc_backward_fp16_ex", "igc_group_norm_workspace_bytes",
    "gemm_int8", "gemm_int8_ex", "igc_gemm_int8_workspace_bytes", "igc_gemm_int8_default_tune",
    "rms_norm_bf16", "rms_norm_fp16", "rms_norm_int8_bf16", "rms_norm_int8_fp16",
    "rms_norm_backward_bf16", "rms_norm_backward_fp16", "rms_norm_backward_bf16_ex", "rms_norm_backward_fp16_ex",
    "igc_rms_norm_backward_workspace_bytes", "quantize_rows_int8_bf16", "quantize_rows_int8_fp16",
    "igc_workspace_bytes", "igc_tune_supported", "igc_default_tune", "igc_tune_count", "igc_tune_get",
    "igc_tune_scope", "igc_tune_lds_bytes", "igc_status_string", "igc_take_device_error", "igc_debug_stream_k",
    "igc_pool_allocations", "igc_ring_schedule", "igc_lds_chunk", "igc_stage_slot",
)


class IgcError(RuntimeError):
    def __init__(self, status):
        self.status = status
        super().__init__(status_string(status))


class Tune(ctypes.Structure):
    _fields_ = [("bm", ctypes.c_int), ("bn", ctypes.c_int), ("bk", ctypes.c_int), ("pipe_depth", ctypes.c_int),
                ("waves", ctypes.c_int), ("mfma", ctypes.c_int), ("half_stage", ctypes.c_int),
                ("loader_waves", ctypes.c_int), ("k_splits", ctypes.c_int), ("stream_k", ctypes.c_int),
                ("ring_sync", ctypes.c_int), ("sk_hybrid", ctypes.c_int)]

    def astuple(self):
        """(bm, bn, bk, pipe_depth, waves, mfma, half_stage, loader_waves, ring_sync): the compiled configuration."""
        return (self.bm, self.bn, self.bk, self.pipe_depth, self.waves, self.mfma or 32, self.half_stage,
                self.loader_waves or self.waves, self.ring_sync)


def tune(cfg, k_splits=0, stream_k=0, sk_hybrid=0):
    """A Tune from a compiled configuration tuple (bm, bn, bk, pipe_depth, waves, mfma, half_stage, loader_waves
    [, ring_sync]) and a schedule."""
    cfg = tuple(cfg)
    ring_sync = cfg[8] if len(cfg) > 8 else 0
    return Tune(*cfg[:8], k_splits, stream_k, ring_sync, sk_hybrid)


class CEpilogue(ctypes.Structure):
    """igc_epilogue_t."""
    _fields_ = [("act", ctypes.c_int), ("backward", ctypes.c_int), ("bias", ctypes.c_void_p),
                ("bias_type", ctypes.c_int), ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("residual_type", ctypes.c_int), ("pre", ctypes.c_void_p), ("ldp", ctypes.c_int64),
                ("pre_type", ctypes.c_int)]


def act_code(act):
    """The code of an activation given by name ("none", "relu", "gelu", "gelu_tanh", "silu") or by code."""
    return ACT_CODES[act] if isinstance(act, str) else int(act)


_DTYPE_CODES = {}


def out_code(dtype):
    """The OUT_ code of a torch dtype."""
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        code = {"torch.float32": OUT_F32, "torch.bfloat16": OUT_BF16, "torch.float16": OUT_F16}.get(str(dtype))
        if code is None:
            raise TypeError(f"{dtype}: float32, bfloat16 or float16 wanted")
        _DTYPE_CODES[dtype] = code
    return code


_EPILOGUE = struct.Struct("@iiPiPqiPqi0q")  # igc_epilogue_t, the layout of CEpilogue
assert _EPILOGUE.size == ctypes.sizeof(CEpilogue)


def _on_host(x):
    """Whether a tensor that is not a GPU's lies where the GPU cannot reach it.  (Plain addresses cannot be told apart.)"""
    return x.data_ptr() != 0 and x.nbytes != 0 and not x.is_pinned()


def _refuse_host(what):
    raise ValueError(f"{what} is in host memory, where the GPU cannot reach it")


def _bias(x, code):
    try:
        ptr = x.data_ptr()
    except AttributeError:
        if code is None:
            raise TypeError("a raw address needs its type") from None
        return int(x), code
    if not x.is_contiguous() and x.shape[-1] > 1 and x.stride(-1) != 1:
        raise ValueError("values of a row must lie together")
    return ptr, out_code(x.dtype) if code is None else code


def _matrix(x, code, ld):
    try:
        ptr, strides = x.data_ptr(), x.stride()
    except AttributeError:
        if code is None or ld is None:
            raise TypeError("a raw address needs its type and leading dimension") from None
        return int(x), ld, code
    if strides and strides[-1] != 1 and x.shape[-1] > 1:
        raise ValueError("values of a row must lie together")
    if ld is None:
        if len(strides) > 2 and not x.is_contiguous():
            raise ValueError("an epilogue's tensor of more than two dimensions is taken as dense, and this one is not")
        ld = strides[0] if len(strides) == 2 else 0
    return ptr, ld, out_code(x.dtype) if code is None else code


class Epilogue:
    """A fused epilogue (igc_epilogue_t) from tensors: types come from their dtypes, the leading dimensions of a
    `residual` and `pre` of two dimensions from their first stride unless given, and the tensors are kept alive with it.
    Those of more dimensions and no given leading dimension, and all of a convolution's, have to be dense (ValueError).  A raw device address needs its type (bias_type, residual_type, pre_type:
    an OUT_ code) and leading dimension.  `raw` holds the packed C structure: calls take it as it is, and refuse one
    whose tensors are in host memory."""
    __slots__ = ("raw", "_keep", "_host")

    def __init__(self, act="none", bias=None, residual=None, pre=None, backward=False, ldr=None, ldp=None,
                 bias_type=None, residual_type=None, pre_type=None):
        self._keep = (bias, residual, pre)
        self._host = None
        for name, x in (("bias", bias), ("residual", residual), ("pre", pre)):
            if x is not None and not getattr(x, "is_cuda", True) and _on_host(x):
                self._host = name
        self.raw = _EPILOGUE.pack(act_code(act), backward, *((0, 0) if bias is None else _bias(bias, bias_type)),
                                  *((0, 0, 0) if residual is None else _matrix(residual, residual_type, ldr)),
                                  *((0, 0, 0) if pre is None else _matrix(pre, pre_type, ldp)))

    @property
    def c(self):
        """A copy of the C structure."""
        return CEpilogue.from_buffer_copy(self.raw)


_lib = None


def lib():
    """The loaded libigc.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m implicit_gemm_conv_amd.build`")
        # torch ships its own copy of the HIP runtime; load it first so that the
        # library binds to the same runtime that allocated the tensors passed in
        # (with two runtimes in one process, launches on torch's memory fail).
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        L = ctypes.CDLL(LIB_PATH)
        i64, i32, p = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
        tp = ctypes.POINTER(Tune)
        gemm = [i64, i64, i64, p, i64, i32, p, i64, i32, p, i64, i32]
        conv = [i32] * 13 + [p, p, p, i32]
        protos = {"gemm_bf16": gemm + [p], "gemm_fp16": gemm + [p], "gemm_bf16_noalloc": gemm + [p],
                  "gemm_bf16_ex": gemm + [tp, p, i64, p], "gemm_fp16_ex": gemm + [tp, p, i64, p]}
        for base in ("conv2d_nhwc_implicit_gemm", "conv2d_nhwc_dgrad_implicit_gemm", "conv2d_nhwc_wgrad_implicit_gemm"):
            protos[base] = conv + [p]
            protos[base + "_fp16"] = conv + [p]
            protos[base + "_ex"] = conv + [tp, p, i64, p]
            protos[base + "_fp16_ex"] = conv + [tp, p, i64, p]
        ep, f32 = p, ctypes.c_float  # (a packed igc_epilogue_t)
        for base in ("gemm_bf16_epilogue", "gemm_fp16_epilogue"):
            protos[base] = gemm + [ep, p]
            protos[base + "_ex"] = gemm + [ep, tp, p, i64, p]
        for base in ("conv2d_nhwc_implicit_gemm_epilogue", "conv2d_nhwc_implicit_gemm_epilogue_fp16"):
            protos[base] = conv + [ep, p]
            protos[base + "_ex"] = conv + [ep, tp, p, i64, p]
        for t in ("bf16", "fp16"):
            back = [i64, i64, i32, p, i64, p, i64, p, i64, p, i32]
            protos["epilogue_backward_" + t] = back + [p]
            protos["epilogue_backward_" + t + "_ex"] = back + [p, i64, p]
            norm = [i32] * 5 + [p, i64, p, p, i32, f32, i32, p, i64, p, p]
            protos["group_norm_nhwc_" + t] = norm + [p]
            protos["group_norm_nhwc_" + t + "_ex"] = norm + [p, i64, p]
            grad = [i32] * 5 + [p, i64, p, p, i32, p, p, i32, p, i64, p, i64, p, p]
            protos["group_norm_nhwc_backward_" + t] = grad + [p]
            protos["group_norm_nhwc_backward_" + t + "_ex"] = grad + [p, i64, p]
            rows = [i64, i64, p, i64, p, i64, p, i64, p, i32, f32, p, i64, p, p]
            protos["rms_norm_" + t] = rows
            protos["rms_norm_int8_" + t] = rows
            grad = [i64, i64, p, i64, p, i32, p, p, i64, p, i64, p, i64, p]
            protos["rms_norm_backward_" + t] = grad + [p]
            protos["rms_norm_backward_" + t + "_ex"] = grad + [p, i64, p]
            protos["quantize_rows_int8_" + t] = [i64, i64, i32, p, i64, p, i64, p, i64, p, p]
        int8 = [i64, i64, i64, p, i64, p, p, i64, p, p, i64, i32, ep]
        protos["gemm_int8"] = int8 + [p]
        protos["gemm_int8_ex"] = int8 + [tp, p, i64, p]
        for name, args, res in (("igc_gemm_int8_workspace_bytes", [i64, i64, i64, tp], i64),
                                ("igc_gemm_int8_default_tune", [i64, i64, i64, tp], i32),
                                ("igc_rms_norm_backward_workspace_bytes", [i64, i64], i64),
                                ("igc_epilogue_workspace_bytes", [i32, i64, i64, i64, tp], i64),
                                ("igc_epilogue_default_tune", [i32, i64, i64, i64, i32, i32, tp], i32),
                                ("igc_epilogue_backward_workspace_bytes", [i64, i64], i64),
                                ("igc_group_norm_workspace_bytes", [i32] * 5, i64)):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = res
        for name, args in protos.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = i32
        L.igc_workspace_bytes.argtypes = [i32, i64, i64, i64, tp]
        L.igc_workspace_bytes.restype = i64
        L.igc_tune_supported.argtypes = [tp]
        L.igc_tune_supported.restype = i32
        L.igc_default_tune.argtypes = [i32, i64, i64, i64, tp]
        L.igc_default_tune.restype = i32
        L.igc_tune_count.argtypes = []
        L.igc_tune_count.restype = i32
        L.igc_tune_get.argtypes = [i32, tp]
        L.igc_tune_get.restype = i32
        L.igc_tune_scope.argtypes = [i32]
        L.igc_tune_scope.restype = i32
        L.igc_tune_lds_bytes.argtypes = [tp]
        L.igc_tune_lds_bytes.restype = i64
        L.igc_status_string.argtypes = [i32]
        L.igc_status_string.restype = ctypes.c_char_p
        L.igc_take_device_error.argtypes = [ctypes.POINTER(ctypes.c_int)]
        L.igc_take_device_error.restype = i32
        L.igc_debug_stream_k.argtypes = [i32, i32]
        L.igc_debug_stream_k.restype = None
        L.igc_pool_allocations.argtypes = []
        L.igc_pool_allocations.restype = i64
        L.igc_ring_schedule.argtypes = [i32, i32, i32, ctypes.POINTER(ctypes.c_int), i32]
        L.igc_ring_schedule.restype = i32
        L.igc_lds_chunk.argtypes = [i32, i32, i32, i32]
        L.igc_lds_chunk.restype = i32
        L.igc_stage_slot.argtypes = [i32, i32, i32]
        L.igc_stage_slot.restype = i32
        _lib = L
    return _lib


def _ptr(x):
    """A tensor's device address, or an address as it is."""
    if x is None:
        return None
    try:
        if x.is_cuda:  # (one attribute, 0.07 us, before the common return)
            return x.data_ptr()
    except AttributeError:
        return x.data_ptr() if hasattr(x, "data_ptr") else int(x)
    if _on_host(x):
        _refuse_host("a tensor")
    return x.data_ptr()


def _nbytes(x):
    if x is None:
        return 0
    if hasattr(x, "nbytes"):
        return x.nbytes
    raise TypeError("pass workspace_bytes with a raw workspace address")


_current_handle = None


def _stream(stream):
    """The handle of `stream`, or of torch's current one, as an integer.  (torch.cuda.current_stream() builds a Stream
    object, 2.8 us a call; torch's own generated code asks for the handle alone, 0.2 us.)"""
    if stream is None:
        global _current_handle
        if _current_handle is None:
            import torch
            raw, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
            torch.cuda.init()
            _current_handle = (lambda: raw(device())) if raw and device else \
                (lambda: torch.cuda.current_stream().cuda_stream)
        return _current_handle()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _tune(t):
    if t is None:
        return None
    if isinstance(t, Tune):
        return ctypes.byref(t)
    t = tuple(t)
    return ctypes.byref(Tune(*t) if len(t) >= 10 else tune(t))


def gemm_bf16(M, N, K, A, lda, la, B, ldb, lb, C, ldc, c_type, stream=None):
    return lib().gemm_bf16(M, N, K, _ptr(A), lda, la, _ptr(B), ldb, lb, _ptr(C), ldc, c_type, _stream(stream))


def gemm_fp16(M, N, K, A, lda, la, B, ldb, lb, C, ldc, c_type, stream=None):
    return lib().gemm_fp16(M, N, K, _ptr(A), lda, la, _ptr(B), ldb, lb, _ptr(C), ldc, c_type, _stream(stream))


def gemm_bf16_noalloc(M, N, K, A, lda, la, B, ldb, lb, C, ldc, c_type, stream=None):
    return lib().gemm_bf16_noalloc(M, N, K, _ptr(A), lda, la, _ptr(B), ldb, lb, _ptr(C), ldc, c_type,
                                   _stream(stream))


def gemm_bf16_ex(M, N, K, A, lda, la, B, ldb, lb, C, ldc, c_type, tune=None, workspace=None, workspace_bytes=None,
                 stream=None):
    wsb = workspace_bytes if workspace_bytes is not None else _nbytes(workspace)
    return lib().gemm_bf16_ex(M, N, K, _ptr(A), lda, la, _ptr(B), ldb, lb, _ptr(C), ldc, c_type, _tune(tune),
                              _ptr(workspace), wsb, _stream(stream))


def gemm_fp16_ex(M, N, K, A, lda, la, B, ldb, lb, C, ldc, c_type, tune=None, workspace=None, workspace_bytes=None,
                 stream=None):
    wsb = workspace_bytes if workspace_bytes is not None else _nbytes(workspace)
    return lib().gemm_fp16_ex(M, N, K, _ptr(A), lda, la, _ptr(B), ldb, lb, _ptr(C), ldc, c_type, _tune(tune),
                              _ptr(workspace), wsb, _stream(stream))


def _conv_plain(name):
    def call(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, in0, in1, out, out_type,
             stream=None):
        return getattr(lib(), name)(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, _ptr(in0),
                                    _ptr(in1), _ptr(out), out_type, _stream(stream))
    call.__name__ = name
    return call


def _conv_ex(name):
    def call(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, in0, in1, out, out_type,
             tune=None, workspace=None, workspace_bytes=None, stream=None):
        wsb = workspace_bytes if workspace_bytes is not None else _nbytes(workspace)
        return getattr(lib(), name)(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, _ptr(in0),
                                    _ptr(in1), _ptr(out), out_type, _tune(tune), _ptr(workspace), wsb,
                                    _stream(stream))
    call.__name__ = name
    return call


# forward: (x, w) -> y;  data gradient: (dy, w) -> dx;  filter gradient: (x, dy) -> dw
conv2d_nhwc_implicit_gemm = _conv_plain("conv2d_nhwc_implicit_gemm")
conv2d_nhwc_implicit_gemm_fp16 = _conv_plain("conv2d_nhwc_implicit_gemm_fp16")
conv2d_nhwc_implicit_gemm_ex = _conv_ex("conv2d_nhwc_implicit_gemm_ex")
conv2d_nhwc_implicit_gemm_fp16_ex = _conv_ex("conv2d_nhwc_implicit_gemm_fp16_ex")
conv2d_nhwc_dgrad_implicit_gemm = _conv_plain("conv2d_nhwc_dgrad_implicit_gemm")
conv2d_nhwc_dgrad_implicit_gemm_fp16 = _conv_plain("conv2d_nhwc_dgrad_implicit_gemm_fp16")
conv2d_nhwc_dgrad_implicit_gemm_ex = _conv_ex("conv2d_nhwc_dgrad_implicit_gemm_ex")
conv2d_nhwc_dgrad_implicit_gemm_fp16_ex = _conv_ex("conv2d_nhwc_dgrad_implicit_gemm_fp16_ex")
conv2d_nhwc_wgrad_implicit_gemm = _conv_plain("conv2d_nhwc_wgrad_implicit_gemm")
conv2d_nhwc_wgrad_implicit_gemm_fp16 = _conv_plain("conv2d_nhwc_wgrad_implicit_gemm_fp16")
conv2d_nhwc_wgrad_implicit_gemm_ex = _conv_ex("conv2d_nhwc_wgrad_implicit_gemm_ex")
conv2d_nhwc_wgrad_implicit_gemm_fp16_ex = _conv_ex("conv2d_nhwc_wgrad_implicit_gemm_fp16_ex")


def _epi(e):
    if isinstance(e, Epilogue):
        if e._host:
            _refuse_host("the epilogue's " + e._host)
        return e.raw
    return None if e is None else bytes(e)


def _conv_epi(e):
    """The same for a convolution, whose residual and pre are dense NPQK whatever their leading dimensions say."""
    if isinstance(e, Epilogue):
        for x in e._keep[1:]:
            if hasattr(x, "is_contiguous") and not x.is_contiguous():
                raise ValueError("a convolution's residual and pre have to be dense, and one of them is not")
    return _epi(e)


def _entry(name):
    """The C function, looked up once, at the first call."""
    found = []

    def get():
        if not found:
            found.append(getattr(lib(), name))
        return found[0]
    return get


# The calls of small operators are bound by their host side, so these look their C function up once.

def _gemm_epilogue(name):
    plain, ex = _entry(name), _entry(name + "_ex")

    def call(M, N, K, A, lda, la, B, ldb, lb, D, ldd, d_type, epilogue, stream=None):
        return plain()(M, N, K, _ptr(A), lda, la, _ptr(B), ldb, lb, _ptr(D), ldd, d_type, _epi(epilogue),
                       _stream(stream))

    def call_ex(M, N, K, A, lda, la, B, ldb, lb, D, ldd, d_type, epilogue, tune=None, workspace=None,
                workspace_bytes=None, stream=None):
        wsb = workspace_bytes if workspace_bytes is not None else _nbytes(workspace)
        return ex()(M, N, K, _ptr(A), lda, la, _ptr(B), ldb, lb, _ptr(D), ldd, d_type, _epi(epilogue),
                    _tune(tune), _ptr(workspace), wsb, _stream(stream))
    call.__name__, call_ex.__name__ = name, name + "_ex"
    return call, call_ex


def _conv_epilogue(name):
    plain, ex = _entry(name), _entry(name + "_ex")

    def call(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, x, w, y, y_type, epilogue,
             stream=None):
        return plain()(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, _ptr(x), _ptr(w),
                       _ptr(y), y_type, _conv_epi(epilogue), _stream(stream))

    def call_ex(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, x, w, y, y_type, epilogue,
                tune=None, workspace=None, workspace_bytes=None, stream=None):
        wsb = workspace_bytes if workspace_bytes is not None else _nbytes(workspace)
        return ex()(N, H, W, C, K, R, S, stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, _ptr(x), _ptr(w),
                    _ptr(y), y_type, _conv_epi(epilogue), _tune(tune), _ptr(workspace), wsb, _stream(stream))
    call.__name__, call_ex.__name__ = name, name + "_ex"
    return call, call_ex


def _epilogue_backward(name):
    plain, ex = _entry(name), _entry(name + "_ex")

    def call(M, N, act, dD, ldd, pre, ldp, dz, ldz, dbias, dbias_type, stream=None):
        return plain()(M, N, act_code(act), _ptr(dD), ldd, _ptr(pre), ldp, _ptr(dz), ldz, _ptr(dbias),
                       dbias_type, _stream(stream))

    def call_ex(M, N, act, dD, ldd, pre, ldp, dz, ldz, dbias, dbias_type, workspace=None, workspace_bytes=None,
                stream=None):
        wsb = workspace_bytes if workspace_bytes is not None else _nbytes(workspace)
        return ex()(M, N, act_code(act), _ptr(dD), ldd, _ptr(pre), ldp, _ptr(dz), ldz, _ptr(dbias),
                    dbias_type, _ptr(workspace), wsb, _stream(stream))
    call.__name__, call_ex.__name__ = name, name + "_ex"
    return call, call_ex


def _group_norm(name):
    plain, ex = _entry(name), _entry(name + "_ex")

    def call(N, H, W, C, G, x, ldx, gamma, beta, param_type, eps, act, y, ldy, mean=None, rstd=None, stream=None):
        return plain()(N, H, W, C, G, _ptr(x), ldx, _ptr(gamma), _ptr(beta), param_type, eps,
                       act_code(act), _ptr(y), ldy, _ptr(mean), _ptr(rstd), _stream(stream))

    def call_ex(N, H, W, C, G, x, ldx, gamma, beta, param_type, eps, act, y, ldy, mean=None, rstd=None,
                workspace=None, workspace_bytes=None, stream=None):
        wsb = workspace_bytes if workspace_bytes is not None else _nbytes(workspace)
        return ex()(N, H, W, C, G, _ptr(x), ldx, _ptr(gamma), _ptr(beta), param_type, eps, act_code(act),
                    _ptr(y), ldy, _ptr(mean), _ptr(rstd), _ptr(workspace), wsb, _stream(stream))
    call.__name__, call_ex.__name__ = name, name + "_ex"
    return call, call_ex


def _group_norm_backward(name):
    plain, ex = _entry(name), _entry(name + "_ex")

    def call(N, H, W, C, G, x, ldx, gamma, beta, param_type, mean, rstd, act, dy, lddy, dx, lddx, dgamma=None,
             dbeta=None, stream=None):
        return plain()(N, H, W, C, G, _ptr(x), ldx, _ptr(gamma), _ptr(beta), param_type, _ptr(mean),
                       _ptr(rstd), act_code(act), _ptr(dy), lddy, _ptr(dx), lddx, _ptr(dgamma),
                       _ptr(dbeta), _stream(stream))

    def call_ex(N, H, W, C, G, x, ldx, gamma, beta, param_type, mean, rstd, act, dy, lddy, dx, lddx, dgamma=None,
                dbeta=None, workspace=None, workspace_bytes=None, stream=None):
        wsb = workspace_bytes if workspace_bytes is not None else _nbytes(workspace)
        return ex()(N, H, W, C, G, _ptr(x), ldx, _ptr(gamma), _ptr(beta), param_type, _ptr(mean),
                    _ptr(rstd), act_code(act), _ptr(dy), lddy, _ptr(dx), lddx, _ptr(dgamma),
                    _ptr(dbeta), _ptr(workspace), wsb, _stream(stream))
    call.__name__, call_ex.__name__ = name, name + "_ex"
    return call, call_ex


def _rms_norm(name):
    entry = _entry(name)

    def call(M, C, x, ldx, residual, ldr, h, ldh, gamma, param_type, eps, y, ldy, rstd=None, stream=None):
        return entry()(M, C, _ptr(x), ldx, _ptr(residual), ldr, _ptr(h), ldh, _ptr(gamma), param_type, eps, _ptr(y), ldy,
                       _ptr(rstd), _stream(stream))
    call.__name__ = name
    return call


def _rms_norm_int8(name):
    entry = _entry(name)

    def call(M, C, x, ldx, residual, ldr, h, ldh, gamma, param_type, eps, q, ldq, scale, stream=None):
        return entry()(M, C, _ptr(x), ldx, _ptr(residual), ldr, _ptr(h), ldh, _ptr(gamma), param_type, eps, _ptr(q), ldq,
                       _ptr(scale), _stream(stream))
    call.__name__ = name
    return call


def _rms_norm_backward(name):
    plain, ex = _entry(name), _entry(name + "_ex")

    def call(M, C, h, ldh, gamma, param_type, rstd, dy, lddy, dh, lddh, dx, lddx, dgamma=None, stream=None):
        return plain()(M, C, _ptr(h), ldh, _ptr(gamma), param_type, _ptr(rstd), _ptr(dy), lddy, _ptr(dh), lddh, _ptr(dx),
                       lddx, _ptr(dgamma), _stream(stream))

    def call_ex(M, C, h, ldh, gamma, param_type, rstd, dy, lddy, dh, lddh, dx, lddx, dgamma=None, workspace=None,
                workspace_bytes=None, stream=None):
        wsb = workspace_bytes if workspace_bytes is not None else _nbytes(workspace)
        return ex()(M, C, _ptr(h), ldh, _ptr(gamma), param_type, _ptr(rstd), _ptr(dy), lddy, _ptr(dh), lddh, _ptr(dx),
                    lddx, _ptr(dgamma), _ptr(workspace), wsb, _stream(stream))
    call.__name__, call_ex.__name__ = name, name + "_ex"
    return call, call_ex


def _quantize_rows(name):
    entry = _entry(name)

    def call(M, C, act, x, ldx, gate, ldg, q, ldq, scale, stream=None):
        return entry()(M, C, act_code(act), _ptr(x), ldx, _ptr(gate), ldg, _ptr(q), ldq, _ptr(scale), _stream(stream))
    call.__name__ = name
    return call


_gemm_int8, _gemm_int8_ex = _entry("gemm_int8"), _entry("gemm_int8_ex")


def gemm_int8(M, N, K, A, lda, scale_a, B, ldb, scale_b, D, ldd, d_type, epilogue=None, stream=None):
    return _gemm_int8()(M, N, K, _ptr(A), lda, _ptr(scale_a), _ptr(B), ldb, _ptr(scale_b), _ptr(D), ldd, d_type,
                        _epi(epilogue), _stream(stream))


def gemm_int8_ex(M, N, K, A, lda, scale_a, B, ldb, scale_b, D, ldd, d_type, epilogue=None, tune=None, workspace=None,
                 workspace_bytes=None, stream=None):
    wsb = workspace_bytes if workspace_bytes is not None else _nbytes(workspace)
    return _gemm_int8_ex()(M, N, K, _ptr(A), lda, _ptr(scale_a), _ptr(B), ldb, _ptr(scale_b), _ptr(D), ldd, d_type,
                           _epi(epilogue), _tune(tune), _ptr(workspace), wsb, _stream(stream))


gemm_bf16_epilogue, gemm_bf16_epilogue_ex = _gemm_epilogue("gemm_bf16_epilogue")
gemm_fp16_epilogue, gemm_fp16_epilogue_ex = _gemm_epilogue("gemm_fp16_epilogue")
conv2d_nhwc_implicit_gemm_epilogue, conv2d_nhwc_implicit_gemm_epilogue_ex = \
    _conv_epilogue("conv2d_nhwc_implicit_gemm_epilogue")
conv2d_nhwc_implicit_gemm_epilogue_fp16, conv2d_nhwc_implicit_gemm_epilogue_fp16_ex = \
    _conv_epilogue("conv2d_nhwc_implicit_gemm_epilogue_fp16")
epilogue_backward_bf16, epilogue_backward_bf16_ex = _epilogue_backward("epilogue_backward_bf16")
epilogue_backward_fp16, epilogue_backward_fp16_ex = _epilogue_backward("epilogue_backward_fp16")
group_norm_nhwc_bf16, group_norm_nhwc_bf16_ex = _group_norm("group_norm_nhwc_bf16")
group_norm_nhwc_fp16, group_norm_nhwc_fp16_ex = _group_norm("group_norm_nhwc_fp16")
group_norm_nhwc_backward_bf16, group_norm_nhwc_backward_bf16_ex = _group_norm_backward("group_norm_nhwc_backward_bf16")
group_norm_nhwc_backward_fp16, group_norm_nhwc_backward_fp16_ex = _group_norm_backward("group_norm_nhwc_backward_fp16")

rms_norm_bf16, rms_norm_fp16 = _rms_norm("rms_norm_bf16"), _rms_norm("rms_norm_fp16")
rms_norm_int8_bf16, rms_norm_int8_fp16 = _rms_norm_int8("rms_norm_int8_bf16"), _rms_norm_int8("rms_norm_int8_fp16")
rms_norm_backward_bf16, rms_norm_backward_bf16_ex = _rms_norm_backward("rms_norm_backward_bf16")
rms_norm_backward_fp16, rms_norm_backward_fp16_ex = _rms_norm_backward("rms_norm_backward_fp16")
quantize_rows_int8_bf16 = _quantize_rows("quantize_rows_int8_bf16")
quantize_rows_int8_fp16 = _quantize_rows("quantize_rows_int8_fp16")


def igc_gemm_int8_workspace_bytes(M, N, K, tune=None):
    return lib().igc_gemm_int8_workspace_bytes(M, N, K, _tune(tune))


def igc_gemm_int8_default_tune(M, N, K):
    """The Tune that gemm_int8 takes; bm = 0 where it runs on the kernel of few rows."""
    t = Tune()
    if not lib().igc_gemm_int8_default_tune(M, N, K, ctypes.byref(t)):
        raise ValueError("bad arguments, or a schedule that is not compiled")
    return t


def igc_rms_norm_backward_workspace_bytes(M, C):
    return lib().igc_rms_norm_backward_workspace_bytes(M, C)


def igc_epilogue_workspace_bytes(op, M, N, K, tune=None):
    return lib().igc_epilogue_workspace_bytes(op, M, N, K, _tune(tune))


def igc_epilogue_default_tune(M, N, K, op=OP_GEMM, la=ROW_MAJOR, lb=COL_MAJOR):
    """The Tune that a call with an epilogue takes; bm = 0 where a product runs on the kernel of few rows."""
    t = Tune()
    if not lib().igc_epilogue_default_tune(op, M, N, K, la, lb, ctypes.byref(t)):
        raise ValueError("bad arguments, or a schedule that is not compiled")
    return t


def igc_epilogue_backward_workspace_bytes(M, N):
    return lib().igc_epilogue_backward_workspace_bytes(M, N)


def igc_group_norm_workspace_bytes(N, H, W, C, G):
    return lib().igc_group_norm_workspace_bytes(N, H, W, C, G)


def conv_out_hw(H, W, R, S, sh=1, sw=1, ph=0, pw=0, dh=1, dw=1):
    """Output size (P, Q) of the forward convolution."""
    return (H + 2 * ph - dh * (R - 1) - 1) // sh + 1, (W + 2 * pw - dw * (S - 1) - 1) // sw + 1


def conv_gemm_view(op, N, H, W, C, K, R, S, sh=1, sw=1, ph=0, pw=0, dh=1, dw=1):
    """(M, N_gemm, K_gemm) of a convolution operation, as include/igc.h defines them."""
    P, Q = conv_out_hw(H, W, R, S, sh, sw, ph, pw, dh, dw)
    if op == OP_CONV_FPROP:
        return N * P * Q, K, R * S * C
    if op == OP_CONV_DGRAD:
        return N * H * W, C, R * S * K
    return K, R * S * C, N * P * Q


def igc_workspace_bytes(op, M, N, K, tune=None):
    return lib().igc_workspace_bytes(op, M, N, K, _tune(tune))


def igc_tune_supported(t):
    return lib().igc_tune_supported(_tune(t))


def igc_default_tune(M, N, K, op=OP_GEMM):
    """The Tune the library picks for operation `op` with GEMM view M x N x K."""
    t = Tune()
    if not lib().igc_default_tune(op, M, N, K, ctypes.byref(t)):
        raise ValueError("bad shape")
    return t


def igc_tune_count():
    return lib().igc_tune_count()


def igc_tune_get(i):
    t = Tune()
    return t if lib().igc_tune_get(i, ctypes.byref(t)) else None


SCOPE_ALL, SCOPE_STREAM_K, SCOPE_CONV_FPROP, SCOPE_EPILOGUE = 1, 2, 4, 8


def igc_tune_scope(i):
    return lib().igc_tune_scope(i)


def igc_tune_lds_bytes(t):
    return lib().igc_tune_lds_bytes(_tune(t))


def tunes(scope=0):
    """Compiled (bm, bn, bk, pipe_depth, waves, mfma, half_stage, loader_waves, ring_sync) configurations whose
    scope includes every bit of `scope` (SCOPE_ALL: every type, layout and operation; SCOPE_STREAM_K;
    SCOPE_CONV_FPROP: the complete forward convolution; SCOPE_EPILOGUE: the fused epilogue)."""
    return [igc_tune_get(i).astuple() for i in range(igc_tune_count()) if igc_tune_scope(i) & scope == scope]


def igc_status_string(status):
    return lib().igc_status_string(int(status)).decode()


status_string = igc_status_string


def igc_take_device_error():
    """The current device's error word (then cleared); synchronises the device."""
    v = ctypes.c_int(0)
    check(lib().igc_take_device_error(ctypes.byref(v)))
    return v.value


def igc_debug_stream_k(spin_limit=0, drop_workgroup=-1):
    lib().igc_debug_stream_k(spin_limit, drop_workgroup)


def igc_pool_allocations():
    return lib().igc_pool_allocations()


def igc_ring_schedule(pipe_depth, k_tiles, half_stage=0):
    """The mainloop's event list [(kind, tile, operand, x), ...] (see include/igc.h)."""
    n = lib().igc_ring_schedule(pipe_depth, half_stage, k_tiles, None, 0)
    if n < 0:
        raise ValueError("bad ring parameters")
    buf = (ctypes.c_int * (4 * max(n, 1)))()
    lib().igc_ring_schedule(pipe_depth, half_stage, k_tiles, buf, n)
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(n)]


def igc_lds_chunk(k_contiguous, chunks_per_row, row, logical_chunk):
    return lib().igc_lds_chunk(k_contiguous, chunks_per_row, row, logical_chunk)


def igc_stage_slot(row, slot, slots_per_row):
    return lib().igc_stage_slot(row, slot, slots_per_row)


def check(status):
    """Raises IgcError unless status is IGC_OK."""
    if status != IGC_OK:
        raise IgcError(status)
