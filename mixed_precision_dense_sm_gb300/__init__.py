"""Python binding for libgemm_sm103.so, the GB300 mixed-precision GEMM and
row softmax.

Argument marshalling only: every step of C = alpha*op(A)*op(B) + beta*C runs in
the library's CUDA kernels.  PyTorch is used for device memory and streams.
If the compiled library is missing, importing this package raises -- there is
no fallback implementation.

The entry points mirror include/gemm_sm103.h one to one:
``gemm_create``, ``gemm_run``, ``gemm_sync``, ``gemm_destroy``,
``gemm_status_string``, ``gemm_check_args``, ``gemm_plan_query``,
``gemm_run_ex`` (fused bias/activation epilogue), ``gemm_run_layernorm``
and ``gemm_layernorm_plan_query`` (LayerNorm after the linear layer),
``gemm_debug_set`` and ``gemm_run_noalloc``; and include/softmax_sm103.h: ``softmax_rows``,
``softmax_plan_query``, ``softmax_sync``, ``softmax_debug_set``; and
include/conv_sm103.h: ``conv2d_fprop``, ``conv2d_plan_query``,
``conv2d_output_dims``; include/glu_sm103.h (the gated linear layer):
``glu_forward``, ``glu_backward``, ``glu_plan_query``; include/norm_sm103.h
(norms around a block): ``norm_block_forward``, ``norm_block_backward``,
``norm_block_backward_workspace``; include/grad_sm103.h (gradient norm and
clipping): ``grad_clip_raw``, ``grad_clip_workspace``; include/expert_sm103.h
(tokens sorted by expert and back): ``expert_sort_raw`` and ``expert_rows_raw``;
include/ortho_sm103.h (the orthogonalised update): ``ortho_update``,
``ortho_workspace``.
``Gemm`` wraps a handle and adds ``__call__``, ``layernorm``, ``glu``,
``glu_backward`` and ``orthogonalize`` for torch tensors; ``softmax``, ``norm_block``,
``norm_block_backward``, ``grad_clip``, ``expert_sort``, ``expert_gather``,
``expert_combine``, ``expert_gather_backward`` and ``expert_combine_backward``
do the same for the others.
"""
from __future__ import annotations

import array
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgemm_sm103.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "gemm_sm103.h")
HEADERS = [HEADER, os.path.join(os.path.dirname(HERE), "include", "softmax_sm103.h"),
           os.path.join(os.path.dirname(HERE), "include", "conv_sm103.h"),
           os.path.join(os.path.dirname(HERE), "include", "glu_sm103.h"),
           os.path.join(os.path.dirname(HERE), "include", "norm_sm103.h"),
           os.path.join(os.path.dirname(HERE), "include", "grad_sm103.h"),
           os.path.join(os.path.dirname(HERE), "include", "expert_sm103.h"),
           os.path.join(os.path.dirname(HERE), "include", "ortho_sm103.h")]

GEMM_F16, GEMM_BF16, GEMM_F32 = 0, 1, 2
STATUS = {0: "GEMM_OK", 1: "GEMM_ERR_INVALID_VALUE", 2: "GEMM_ERR_NOT_SUPPORTED",
          3: "GEMM_ERR_ALLOC", 4: "GEMM_ERR_LAUNCH", 5: "GEMM_ERR_DEVICE_TIMEOUT"}
PATHS = {0: "noop", 1: "scale", 2: "tiled_1sm", 3: "tiled_2sm", 4: "skinny",
         5: "dot"}


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class Dtypes(ctypes.Structure):
    _fields_ = [("a", ctypes.c_int32), ("b", ctypes.c_int32), ("c", ctypes.c_int32)]


class Epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("bias_dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


class LayerNorm(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("bias_dtype", ctypes.c_int32),
                ("gamma", ctypes.c_void_p), ("shift", ctypes.c_void_p),
                ("ln_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class GluForward(ctypes.Structure):
    _fields_ = [("activation", ctypes.c_int32), ("bias", ctypes.c_void_p),
                ("bias_dtype", ctypes.c_int32), ("P", ctypes.c_void_p), ("ldp", ctypes.c_int64)]


class GluBackward(ctypes.Structure):
    _fields_ = [("activation", ctypes.c_int32), ("p_dtype", ctypes.c_int32),
                ("dP", ctypes.c_void_p), ("lddp", ctypes.c_int64),
                ("dX", ctypes.c_void_p), ("lddx", ctypes.c_int64), ("dx_dtype", ctypes.c_int32),
                ("dW", ctypes.c_void_p), ("lddw", ctypes.c_int64), ("dw_dtype", ctypes.c_int32),
                ("beta_w", ctypes.c_float),
                ("dbias", ctypes.c_void_p), ("dbias_dtype", ctypes.c_int32)]


NORM_KINDS = {None: 0, "none": 0, "rms": 1, "layer": 2}
NORM_MAX_N = 16384


class NormBlock(ctypes.Structure):
    _fields_ = [("pre", ctypes.c_int32), ("post", ctypes.c_int32),
                ("pre_weight", ctypes.c_void_p), ("pre_bias", ctypes.c_void_p),
                ("post_weight", ctypes.c_void_p), ("post_bias", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("ld_gate", ctypes.c_int64),
                ("gate_rows", ctypes.c_int64), ("vec_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float)]


class NormBlockGrads(ctypes.Structure):
    _fields_ = [("d_pre_weight", ctypes.c_void_p), ("d_pre_bias", ctypes.c_void_p),
                ("d_post_weight", ctypes.c_void_p), ("d_post_bias", ctypes.c_void_p),
                ("d_gate", ctypes.c_void_p), ("grad_dtype", ctypes.c_int32)]


class ExpertWeights(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("ldw", ctypes.c_int64),
                ("weight_dtype", ctypes.c_int32), ("dweight", ctypes.c_void_p),
                ("lddw", ctypes.c_int64), ("dweight_dtype", ctypes.c_int32)]


EXPERT_MAX = 1024


class OrthoUpdate(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("coefficients", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("scale", ctypes.c_float)]


ORTHO_MAX_STEPS, ORTHO_MAX_SIDE = 32, 65536
ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU = 0, 1, 2, 3
ACTIVATIONS = {None: ACT_NONE, "none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU,
               "silu": ACT_SILU}


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "path", "block_m", "block_n", "block_k", "stages", "split_k", "grid", "num_tiles",
        "pack_a", "pack_b", "a_mn_major", "b_mn_major", "swap_ab", "c_vector", "sk_len",
        "sk_max_seg", "k_blocks", "tiles_m", "tiles_n", "transpose_ab", "c_tma")] + \
        [("workspace_bytes", ctypes.c_int64), ("conv_rows", ctypes.c_int32),
         ("conv_pitch", ctypes.c_int32)]

    def as_dict(self):
        d = {n: getattr(self, n) for n, _ in self._fields_}
        d["path_name"] = PATHS.get(self.path, "?")
        return d


SOFTMAX_MODES = {0: "noop", 1: "warp", 2: "cta", 3: "stream"}


class SoftmaxPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "mode", "threads", "cluster", "slice", "vec", "grid", "depth", "group_warps", "unit_rows",
        "kv")] + \
        [("hbm_bytes", ctypes.c_int64)]

    def as_dict(self):
        d = {n: getattr(self, n) for n, _ in self._fields_}
        d["mode_name"] = SOFTMAX_MODES.get(self.mode, "?")
        return d


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -c \"import __graft_entry__ as g; g.build()\"` "
            "(the CUDA library is required; there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    i64, vp, c = ctypes.c_int64, ctypes.c_void_p, ctypes.c_char
    run_args = [c, c, i64, i64, i64, ctypes.c_float, vp, i64, vp, i64, ctypes.c_float, vp, i64,
                Dtypes]
    lib.gemm_create.restype = ctypes.c_int
    lib.gemm_create.argtypes = [ctypes.POINTER(vp)]
    lib.gemm_run.restype = ctypes.c_int
    lib.gemm_run.argtypes = [vp] + run_args + [vp]
    lib.gemm_run_ex.restype = ctypes.c_int
    lib.gemm_run_ex.argtypes = [vp] + run_args + [ctypes.POINTER(Epilogue), vp]
    lib.gemm_run_layernorm.restype = ctypes.c_int
    lib.gemm_run_layernorm.argtypes = [vp] + run_args + [ctypes.POINTER(LayerNorm), vp]
    lib.gemm_layernorm_plan_query.restype = ctypes.c_int
    lib.gemm_layernorm_plan_query.argtypes = run_args + [
        ctypes.POINTER(LayerNorm), ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(Plan),
        ctypes.POINTER(ctypes.c_int32)]
    lib.gemm_run_noalloc.restype = ctypes.c_int
    lib.gemm_run_noalloc.argtypes = run_args + [vp]
    lib.gemm_debug_set.restype = ctypes.c_int
    lib.gemm_debug_set.argtypes = [vp, ctypes.c_uint32, ctypes.c_uint64]
    lib.gemm_sync.restype = ctypes.c_int
    lib.gemm_sync.argtypes = [vp, vp]
    lib.gemm_destroy.restype = ctypes.c_int
    lib.gemm_destroy.argtypes = [vp]
    lib.gemm_status_string.restype = ctypes.c_char_p
    lib.gemm_status_string.argtypes = [ctypes.c_int]
    lib.gemm_check_args.restype = ctypes.c_int
    lib.gemm_check_args.argtypes = run_args
    lib.gemm_plan_query.restype = ctypes.c_int
    lib.gemm_plan_query.argtypes = run_args + [ctypes.c_int32, ctypes.c_int32,
                                               ctypes.POINTER(Plan)]
    i32 = ctypes.c_int32
    smx_args = [i64, i64, vp, i64, i32, vp, i64, i32]
    lib.softmax_rows.restype = ctypes.c_int
    lib.softmax_rows.argtypes = smx_args + [vp]
    lib.softmax_plan_query.restype = ctypes.c_int
    lib.softmax_plan_query.argtypes = smx_args + [i32, i32, ctypes.POINTER(SoftmaxPlan)]
    conv_geo = [i64] * 13
    lib.conv2d_output_dims.restype = ctypes.c_int
    lib.conv2d_output_dims.argtypes = [i64] * 10 + [ctypes.POINTER(i64)] * 2
    lib.conv2d_fprop.restype = ctypes.c_int
    lib.conv2d_fprop.argtypes = [vp] + conv_geo + [ctypes.c_float, vp, vp, ctypes.c_float, vp,
                                                   Dtypes, ctypes.POINTER(Epilogue), vp]
    lib.conv2d_plan_query.restype = ctypes.c_int
    lib.conv2d_plan_query.argtypes = conv_geo + [ctypes.c_float, vp, vp, ctypes.c_float, vp,
                                                 Dtypes, i32, i32, ctypes.POINTER(Plan)]
    glu_args = [i64, i64, i64, vp, i64, vp, i64, vp, i64, Dtypes, ctypes.POINTER(GluForward)]
    lib.glu_forward.restype = ctypes.c_int
    lib.glu_forward.argtypes = [vp] + glu_args + [vp]
    lib.glu_plan_query.restype = ctypes.c_int
    lib.glu_plan_query.argtypes = glu_args + [i32, i32, ctypes.POINTER(Plan)]
    lib.glu_backward.restype = ctypes.c_int
    lib.glu_backward.argtypes = [vp, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32,
                                 ctypes.POINTER(GluBackward), vp]
    lib.norm_block_forward.restype = ctypes.c_int
    lib.norm_block_forward.argtypes = [i64, i64] + [vp, i64] * 4 + [
        i32, i32, ctypes.POINTER(NormBlock), vp]
    lib.norm_block_backward.restype = ctypes.c_int
    lib.norm_block_backward.argtypes = [i64, i64] + [vp, i64] * 6 + [
        i32, i32, ctypes.POINTER(NormBlock), ctypes.POINTER(NormBlockGrads), vp, i64, vp]
    lib.norm_block_backward_workspace.restype = i64
    lib.norm_block_backward_workspace.argtypes = [i64, i64, i64, i32]
    lib.grad_clip.restype = ctypes.c_int
    lib.grad_clip.argtypes = [i64, vp, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp, vp, i64, vp]
    lib.grad_clip_workspace.restype = i64
    lib.grad_clip_workspace.argtypes = [i64, i32]
    lib.expert_sort.restype = ctypes.c_int
    lib.expert_sort.argtypes = [i64, i64, i64, vp, i64, i32, vp, vp, vp, vp]
    for f in (lib.expert_gather, lib.expert_combine):
        f.restype = ctypes.c_int
        f.argtypes = [i64] * 4 + [vp, i64, vp, vp, i64, i32, ctypes.POINTER(ExpertWeights), vp]
    for f in (lib.expert_gather_backward, lib.expert_combine_backward):
        f.restype = ctypes.c_int
        f.argtypes = [i64] * 4 + [vp, i64, vp, i64, vp, vp, i64, i32,
                                  ctypes.POINTER(ExpertWeights), vp]
    lib.ortho_update.restype = ctypes.c_int
    lib.ortho_update.argtypes = [vp, i64, i64, i64, vp, i64, i64, i32, vp, i64, i64,
                                 ctypes.POINTER(OrthoUpdate), vp]
    lib.ortho_workspace.restype = i64
    lib.ortho_workspace.argtypes = [i64, i64, i64]
    lib.softmax_sync.restype = ctypes.c_int
    lib.softmax_sync.argtypes = [vp]
    lib.softmax_debug_set.restype = ctypes.c_int
    lib.softmax_debug_set.argtypes = [ctypes.c_uint32, ctypes.c_uint64]
    return lib


lib = _load()


def _tr(t: str) -> bytes:
    return t.encode() if isinstance(t, str) else bytes(t)


def gemm_status_string(status: int) -> str:
    return lib.gemm_status_string(status).decode()


def gemm_create() -> int:
    h = ctypes.c_void_p()
    st = lib.gemm_create(ctypes.byref(h))
    if st != 0:
        raise GemmError(st, "gemm_create")
    return h.value


def gemm_destroy(h) -> int:
    return lib.gemm_destroy(h)


GEMM_DEBUG_SKIP_FIRST_LOAD = 1


def gemm_debug_set(h, flags: int, wait_limit_ns: int = 0) -> int:
    """Test hook of the failure path (see include/gemm_sm103.h)."""
    return lib.gemm_debug_set(h, flags, wait_limit_ns)


def gemm_sync(h, stream=0) -> int:
    return lib.gemm_sync(h, stream)


def gemm_run(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
             dtypes, stream=0) -> int:
    """Raw C-ABI call: A, B, C are device addresses (ints), dtypes a
    (a, b, c) tuple of GEMM_F16/GEMM_BF16/GEMM_F32, stream a cudaStream_t
    value.  Returns the gemm_status_t code."""
    return lib.gemm_run(h, _tr(transA), _tr(transB), M, N, K, float(alpha), A, lda, B, ldb,
                        float(beta), C, ldc, Dtypes(*dtypes), stream)


def gemm_run_ex(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtypes,
                bias=0, bias_dtype=GEMM_F32, act=ACT_NONE, stream=0) -> int:
    """Raw C-ABI call with a fused epilogue: act(alpha*AB + beta*C + bias[n]).
    bias is a device address (0 for none)."""
    ep = Epilogue(bias or None, bias_dtype, act)
    return lib.gemm_run_ex(h, _tr(transA), _tr(transB), M, N, K, float(alpha), A, lda, B, ldb,
                           float(beta), C, ldc, Dtypes(*dtypes), ctypes.byref(ep), stream)


def gemm_run_layernorm(h, transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtypes,
                       bias=0, bias_dtype=GEMM_F32, gamma=0, shift=0, ln_dtype=GEMM_F32,
                       eps=1e-5, stream=0) -> int:
    """Raw C-ABI call of LayerNorm after the linear layer: C <- LayerNorm(
    round_C(alpha*AB + beta*C + bias)) * gamma + shift along each row of C.
    bias, gamma, shift are device addresses (0 for none)."""
    ln = LayerNorm(bias or None, bias_dtype, gamma or None, shift or None, ln_dtype, eps)
    return lib.gemm_run_layernorm(h, _tr(transA), _tr(transB), M, N, K, float(alpha), A, lda, B,
                                  ldb, float(beta), C, ldc, Dtypes(*dtypes), ctypes.byref(ln),
                                  stream)


def gemm_layernorm_plan_query(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                              dtypes, bias=0, bias_dtype=GEMM_F32, gamma=0, shift=0,
                              ln_dtype=GEMM_F32, eps=1e-5, num_sms=152, smem_optin=232448):
    """(status, plan dict with "ln_fused") gemm_run_layernorm would use
    (host logic only)."""
    ln = LayerNorm(bias or None, bias_dtype, gamma or None, shift or None, ln_dtype, eps)
    plan = Plan()
    fused = ctypes.c_int32(-1)
    st = lib.gemm_layernorm_plan_query(_tr(transA), _tr(transB), M, N, K, float(alpha), A, lda, B,
                                       ldb, float(beta), C, ldc, Dtypes(*dtypes), ctypes.byref(ln),
                                       num_sms, smem_optin, ctypes.byref(plan),
                                       ctypes.byref(fused))
    if st != 0:
        return st, None
    d = plan.as_dict()
    d["ln_fused"] = fused.value
    return st, d


def gemm_run_noalloc(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                     dtypes, stream=0) -> int:
    """Raw C-ABI call of the entry point that allocates nothing (no handle):
    for callers that cannot call cudaMalloc.  Same arguments as gemm_run
    without the handle; returns the gemm_status_t code."""
    return lib.gemm_run_noalloc(_tr(transA), _tr(transB), M, N, K, float(alpha), A, lda, B, ldb,
                                float(beta), C, ldc, Dtypes(*dtypes), stream)


def gemm_check_args(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtypes) -> int:
    return lib.gemm_check_args(_tr(transA), _tr(transB), M, N, K, float(alpha), A, lda, B, ldb,
                               float(beta), C, ldc, Dtypes(*dtypes))


def gemm_plan_query(transA, transB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtypes,
                    num_sms=152, smem_optin=232448):
    """(status, plan dict) of the path gemm_run would take (host logic only)."""
    plan = Plan()
    st = lib.gemm_plan_query(_tr(transA), _tr(transB), M, N, K, float(alpha), A, lda, B, ldb,
                             float(beta), C, ldc, Dtypes(*dtypes), num_sms, smem_optin,
                             ctypes.byref(plan))
    return st, (plan.as_dict() if st == 0 else None)


def declared_symbols():
    """Function names declared in the headers under include/."""
    import re
    names = set()
    for h in HEADERS:
        text = open(h).read()
        names |= set(re.findall(r"^\s*(?:gemm_status_t|const char\*|int64_t)\s+"
                                r"((?:gemm|softmax|conv2d|glu|norm|grad|expert|ortho)_\w+)\s*\(",
                                text, flags=re.M))
    return sorted(names)


def softmax_rows(rows, cols, X, ldx, x_dtype, Y, ldy, y_dtype, stream=0) -> int:
    """Raw C-ABI call: Y = softmax(X) along each row.  X, Y are device
    addresses (ints); dtypes GEMM_F16/GEMM_BF16/GEMM_F32; stream a
    cudaStream_t value.  Returns the gemm_status_t code."""
    return lib.softmax_rows(rows, cols, X, ldx, x_dtype, Y, ldy, y_dtype, stream)


SOFTMAX_DEBUG_SKIP_FIRST_LOAD = 1


def conv2d_output_dims(H, W, R, S, pad=(0, 0), stride=(1, 1), dilation=(1, 1)):
    """(P, Q) of a forward convolution (raises on bad geometry)."""
    P, Q = ctypes.c_int64(), ctypes.c_int64()
    st = lib.conv2d_output_dims(H, W, R, S, pad[0], pad[1], stride[0], stride[1], dilation[0],
                                dilation[1], ctypes.byref(P), ctypes.byref(Q))
    if st != 0:
        raise GemmError(st, "conv2d_output_dims")
    return P.value, Q.value


def conv2d_fprop(h, N, H, W, C, K, R, S, pad, stride, dilation, alpha, X, Wt, beta, Y, dtypes,
                 bias=0, bias_dtype=GEMM_F32, act=ACT_NONE, stream=0) -> int:
    """Raw C-ABI call (include/conv_sm103.h): X (NHWC), Wt (KRSC), Y (NPQK)
    device addresses; pad/stride/dilation (h, w) pairs; dtypes (x, w, y).
    Returns the gemm_status_t code."""
    ep = Epilogue(bias or None, bias_dtype, act)
    return lib.conv2d_fprop(h, N, H, W, C, K, R, S, pad[0], pad[1], stride[0], stride[1],
                            dilation[0], dilation[1], float(alpha), X, Wt, float(beta), Y,
                            Dtypes(*dtypes), ctypes.byref(ep), stream)


def conv2d_plan_query(N, H, W, C, K, R, S, pad, stride, dilation, alpha, X, Wt, beta, Y, dtypes,
                      num_sms=152, smem_optin=232448):
    """(status, GEMM plan dict) conv2d_fprop would use (host logic only)."""
    plan = Plan()
    st = lib.conv2d_plan_query(N, H, W, C, K, R, S, pad[0], pad[1], stride[0], stride[1],
                               dilation[0], dilation[1], float(alpha), X, Wt, float(beta), Y,
                               Dtypes(*dtypes), num_sms, smem_optin, ctypes.byref(plan))
    return st, (plan.as_dict() if st == 0 else None)


def softmax_sync(stream=0) -> int:
    """Wait for the stream; GEMM_ERR_DEVICE_TIMEOUT (5) if a softmax kernel
    recorded a bounded wait that ran out (then cleared)."""
    return lib.softmax_sync(stream)


def softmax_debug_set(flags: int, wait_limit_ns: int = 0) -> int:
    """Test hook of the softmax failure path (see include/softmax_sm103.h)."""
    return lib.softmax_debug_set(flags, wait_limit_ns)


def softmax_plan_query(rows, cols, X, ldx, x_dtype, Y, ldy, y_dtype, num_sms=152,
                       ctas_per_sm=0):
    """(status, plan dict) of the work split softmax_rows would use (host logic)."""
    plan = SoftmaxPlan()
    st = lib.softmax_plan_query(rows, cols, X, ldx, x_dtype, Y, ldy, y_dtype, num_sms,
                                ctas_per_sm, ctypes.byref(plan))
    return st, (plan.as_dict() if st == 0 else None)


def softmax(X, Y=None, rows=None, cols=None, stream=None):
    """Row softmax of a 2-D torch tensor on the GPU (unit inner stride, row
    pitch = stride(0)) into Y (a new tensor of X's type and shape if None;
    Y may be X for in place).  Returns Y."""
    import torch
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be 2-D with unit inner stride")
    if Y is None:
        Y = torch.empty_like(X)
    if Y.dim() != 2 or Y.stride(1) != 1:
        raise ValueError("Y must be 2-D with unit inner stride")
    rows = X.shape[0] if rows is None else rows
    cols = X.shape[1] if cols is None else cols
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    st = softmax_rows(rows, cols, X.data_ptr(), X.stride(0), dtype_code(X.dtype), Y.data_ptr(),
                      Y.stride(0), dtype_code(Y.dtype), stream)
    if st != 0:
        raise GemmError(st, "softmax_rows")
    return Y


# ----------------------------------------------------- the gated linear layer

def glu_forward(h, M, F, K, X, ldx, W, ldw, H, ldh, dtypes, act=ACT_NONE, bias=0,
                bias_dtype=GEMM_F32, P=0, ldp=0, stream=0) -> int:
    """Raw C-ABI call (include/glu_sm103.h): H = act(X Wg^T + bg) * (X Wu^T + bu),
    W = [Wg; Wu] stored 2F x K; P (0 for none) receives X W^T + bias.  Device
    addresses; returns the gemm_status_t code."""
    o = GluForward(act, bias or None, bias_dtype, P or None, ldp)
    return lib.glu_forward(h, M, F, K, X, ldx, W, ldw, H, ldh, Dtypes(*dtypes), ctypes.byref(o),
                           stream)


def glu_plan_query(M, F, K, X, ldx, W, ldw, H, ldh, dtypes, act=ACT_NONE, bias=0,
                   bias_dtype=GEMM_F32, P=0, ldp=0, num_sms=152, smem_optin=232448):
    """(status, plan dict) glu_forward would use (host logic only)."""
    o = GluForward(act, bias or None, bias_dtype, P or None, ldp)
    plan = Plan()
    st = lib.glu_plan_query(M, F, K, X, ldx, W, ldw, H, ldh, Dtypes(*dtypes), ctypes.byref(o),
                            num_sms, smem_optin, ctypes.byref(plan))
    return st, (plan.as_dict() if st == 0 else None)


def glu_backward(h, M, F, K, dH, lddh, P, ldp, X, ldx, W, ldw, dtype, dP, lddp, act=ACT_NONE,
                 p_dtype=None, dX=0, lddx=0, dx_dtype=GEMM_F32, dW=0, lddw=0, dw_dtype=GEMM_F32,
                 beta_w=0.0, dbias=0, dbias_dtype=GEMM_F32, stream=0) -> int:
    """Raw C-ABI call of the gated linear layer's backward pass; p_dtype None
    means dtype.  Returns the gemm_status_t code."""
    o = GluBackward(act, dtype if p_dtype is None else p_dtype, dP or None, lddp, dX or None, lddx,
                    dx_dtype, dW or None, lddw, dw_dtype, beta_w, dbias or None, dbias_dtype)
    return lib.glu_backward(h, M, F, K, dH or None, lddh, P or None, ldp, X or None, ldx,
                            W or None, ldw, dtype, ctypes.byref(o), stream)


# ------------------------------------------------------- norms around a block

def norm_block_forward(M, N, X, ldx, Z, ldz, XO, ldxo, Y, ldy, x_dtype, z_dtype, block,
                       stream=0) -> int:
    """Raw C-ABI call (include/norm_sm103.h); `block` a NormBlock, addresses 0
    for what is absent.  Returns the gemm_status_t code."""
    return lib.norm_block_forward(M, N, X or None, ldx, Z or None, ldz, XO or None, ldxo, Y or None,
                                  ldy, x_dtype, z_dtype, ctypes.byref(block), stream)


def norm_block_backward_raw(M, N, XO, ldxo, Z, ldz, dY, lddy, dXO, lddxo, dX, lddx, dZ, lddz,
                            x_dtype, z_dtype, block, grads, workspace, workspace_bytes,
                            stream=0) -> int:
    """Raw C-ABI call of norm_block_backward; `grads` a NormBlockGrads."""
    return lib.norm_block_backward(M, N, XO or None, ldxo, Z or None, ldz, dY or None, lddy,
                                   dXO or None, lddxo, dX or None, lddx, dZ or None, lddz, x_dtype,
                                   z_dtype, ctypes.byref(block), ctypes.byref(grads),
                                   workspace or None, workspace_bytes, stream)


def norm_block_backward_workspace(M, N, gate_rows=1, num_sms=0) -> int:
    """Bytes of workspace norm_block_backward needs (host logic when num_sms > 0)."""
    return lib.norm_block_backward_workspace(M, N, gate_rows, num_sms)


# The planner and the raw C calls need no torch: the first call that takes tensors imports it.
torch = None
_CODE = {}
_DEVICES = {}


def _need_torch():
    global torch
    import torch as t
    _CODE.update({t.float16: GEMM_F16, t.bfloat16: GEMM_BF16, t.float32: GEMM_F32})
    torch = t


# Every launch of a small problem waits for these checks, so they look at each
# tensor once and with few calls; what is wrong is spelled out by _refuse.

def _refuse(t, name, shape, dtype, dev):
    if t.get_device() < 0:
        raise ValueError(f"{name} must be on the GPU")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    raise ValueError(f"{name} must be {' x '.join(map(str, shape))}, with unit inner stride")


def _device(t, name):
    """The current CUDA device, which the tensor has to be on."""
    if torch is None:
        _need_torch()
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        _refuse(t, name, t.shape, None, -1)
    return dev


def _mat(t, name, rows, cols, dtype, dev):
    """(address, row pitch) of a rows x cols matrix; (0, 0) for None."""
    if t is None:
        return 0, 0
    if t.shape != (rows, cols) or dtype is not None and t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, name, (rows, cols), dtype, dev)
    st = t.stride()
    if st[1] != 1 and cols > 1:
        _refuse(t, name, (rows, cols), dtype, dev)
    # torch may give any stride to a single row, or to rows of nothing
    return t.data_ptr(), st[0] if rows > 1 and cols > 0 else max(cols, 1)


def _vec(t, name, n, dtype, dev):
    """Address of a vector of n elements; 0 for None."""
    if t is None:
        return 0
    if t.shape != (n,) or dtype is not None and t.dtype is not dtype or t.get_device() != dev or \
            n > 1 and t.stride(0) != 1:
        _refuse(t, name, (n,), dtype, dev)
    return t.data_ptr()


def _stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev)


def _empty(shape, dtype, dev, stream):
    """A new tensor of the caching allocator for a call on `stream` (None: the
    current one), from that stream's own memory: what another stream freed may
    still be in use there."""
    where = _DEVICES.get(dev)
    if where is None:
        where = _DEVICES[dev] = torch.device("cuda", dev)
    if stream is None or stream == _stream(dev):
        return torch.empty(shape, dtype=dtype, device=where)
    s = torch.cuda.ExternalStream(stream, where) if stream else torch.cuda.default_stream(where)
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=where)


def _first_dtype(*tensors):
    for t in tensors:
        if t is not None:
            return t.dtype
    return None


def _norm_config(N, rows, dev, pre, pre_weight, pre_bias, post, post_weight, post_bias, gate,
                 gate_rows, scale, eps):
    vec = _first_dtype(pre_weight, pre_bias, post_weight, post_bias, gate)
    gp = ld = 0
    if gate is not None:
        if gate_rows < 1:
            raise ValueError("gate_rows must be at least 1")
        gp, ld = _mat(gate, "gate", -(-rows // gate_rows), N, vec, dev)
    return NormBlock(NORM_KINDS[pre], NORM_KINDS[post], _vec(pre_weight, "pre_weight", N, vec, dev),
                     _vec(pre_bias, "pre_bias", N, vec, dev),
                     _vec(post_weight, "post_weight", N, vec, dev),
                     _vec(post_bias, "post_bias", N, vec, dev), gp, ld, gate_rows,
                     GEMM_F32 if vec is None else _CODE[vec], scale, eps)


def norm_block(X, Z=None, XO=None, Y=None, *, pre="rms", pre_weight=None, pre_bias=None, post=None,
               post_weight=None, post_bias=None, gate=None, gate_rows=1, scale=1.0, eps=1e-5,
               stream=None):
    """Norms around a transformer block, on 2-D CUDA tensors: (XO, Y) with
    XO = X + scale * gate * Norm_post(Z) and Y = Norm_pre(XO).

    X (M x N) is the residual stream, Z the block's output; Z None gives
    (None, Norm_pre(X)).  pre and post are "rms", "layer" or None; pre None
    (with no pre_weight or pre_bias) skips Y.  The gate has one row of N for
    every gate_rows rows of X.  XO may be X (in place); XO and Y are new
    tensors where None.  Weights, biases and gate share a dtype."""
    dev = _device(X, "X")
    if X.dim() != 2:
        raise ValueError("X must be 2-D with unit inner stride")
    M, N = X.shape
    xt = X.dtype
    x, ldx = _mat(X, "X", M, N, xt, dev)
    want_y = Y is not None or pre not in (None, "none") or pre_weight is not None or pre_bias is not None
    if Z is not None:
        zt = Z.dtype
        if XO is None:
            XO = _empty((M, N), xt, dev, stream)
    elif XO is not None:
        raise ValueError("XO goes with Z")
    else:
        zt = xt if Y is None else Y.dtype
    if want_y and Y is None:
        Y = _empty((M, N), zt, dev, stream)
    z, ldz = _mat(Z, "Z", M, N, zt, dev)
    xo, ldxo = _mat(XO, "XO", M, N, xt, dev)
    y, ldy = _mat(Y, "Y", M, N, zt, dev)
    block = _norm_config(N, M, dev, pre, pre_weight, pre_bias, post, post_weight, post_bias, gate,
                         gate_rows, scale, eps)
    st = norm_block_forward(M, N, x, ldx, z, ldz, xo, ldxo, y, ldy, dtype_code(xt), dtype_code(zt),
                            block, _stream(dev) if stream is None else stream)
    if st != 0:
        raise GemmError(st, "norm_block_forward")
    return XO, Y


def norm_block_backward(XO, dY=None, dXO=None, Z=None, *, pre="rms", pre_weight=None, post=None,
                        post_weight=None, post_bias=None, gate=None, gate_rows=1, scale=1.0,
                        eps=1e-5, dX=None, dZ=None, dgate=None, dpre_weight=None, dpre_bias=None,
                        dpost_weight=None, dpost_bias=None, workspace=None, stream=None):
    """Backward pass of norm_block into the given tensors (None: not wanted).

    XO is norm_block's output (X where there was no Z), dY and dXO the
    gradients with respect to Y and XO (None: zero).  dX may be dXO and dZ may
    be Z.  The vector gradients share a dtype; dgate is contiguous, as the
    gate.  workspace: a uint8 tensor of norm_block_backward_workspace bytes
    (a new one of the caching allocator where None)."""
    dev = _device(XO, "XO")
    if XO.dim() != 2:
        raise ValueError("XO must be 2-D with unit inner stride")
    M, N = XO.shape
    xt = XO.dtype
    zt = _first_dtype(Z, dY, dZ) or xt
    mats = _mat(XO, "XO", M, N, xt, dev) + _mat(Z, "Z", M, N, zt, dev) + \
        _mat(dY, "dY", M, N, zt, dev) + _mat(dXO, "dXO", M, N, xt, dev) + \
        _mat(dX, "dX", M, N, xt, dev) + _mat(dZ, "dZ", M, N, zt, dev)
    block = _norm_config(N, M, dev, pre, pre_weight, None, post, post_weight, post_bias, gate,
                         gate_rows, scale, eps)
    gt = _first_dtype(dpre_weight, dpre_bias, dpost_weight, dpost_bias, dgate)
    dg = 0
    if dgate is not None:
        if gate is None:
            raise ValueError("dgate goes with gate")
        dg, _ = _mat(dgate, "dgate", gate.shape[0], N, gt, dev)
        if not dgate.is_contiguous():
            raise ValueError("dgate must be contiguous")
    grads = NormBlockGrads(_vec(dpre_weight, "dpre_weight", N, gt, dev),
                           _vec(dpre_bias, "dpre_bias", N, gt, dev),
                           _vec(dpost_weight, "dpost_weight", N, gt, dev),
                           _vec(dpost_bias, "dpost_bias", N, gt, dev), dg,
                           GEMM_F32 if gt is None else dtype_code(gt))
    ws = nbytes = 0
    if gt is not None:
        if workspace is None:
            need = lib.norm_block_backward_workspace(M, N, gate_rows if gate is not None else 1, 0)
            workspace = _empty(max(need, 16), torch.uint8, dev, stream)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous, on the current CUDA device")
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = norm_block_backward_raw(M, N, *mats, dtype_code(xt), dtype_code(zt), block, grads, ws,
                                 nbytes, _stream(dev) if stream is None else stream)
    if st != 0:
        raise GemmError(st, "norm_block_backward")


# ------------------------------------------------ gradient norm and clipping

def grad_clip_workspace(count, num_sms=0) -> int:
    """Bytes of workspace grad_clip needs (host logic when num_sms > 0)."""
    return lib.grad_clip_workspace(count, num_sms)


def grad_clip_raw(grads, outs, sizes, dtypes, max_norm, inv_scale, norm, workspace,
                  workspace_bytes, stream=0) -> int:
    """Raw C-ABI call (include/grad_sm103.h): lists of device addresses (outs
    None: in place), element counts and type codes.  Returns the status code."""
    a = array.array("Q", grads)
    o = None if outs is None else array.array("Q", outs)
    z = array.array("q", sizes)
    d = array.array("i", dtypes)
    return lib.grad_clip(len(grads), a.buffer_info()[0], None if o is None else o.buffer_info()[0],
                         z.buffer_info()[0], d.buffer_info()[0], max_norm, inv_scale, norm or None,
                         workspace or None, workspace_bytes, stream)


def grad_clip(grads, max_norm, outputs=None, inv_scale=1.0, norm=None, workspace=None, stream=None):
    """Clips a list of gradient tensors (contiguous CUDA tensors of any shape;
    FP16, BF16 or FP32) by their global norm, in place or into `outputs`:
    out = g * inv_scale * min(1, max_norm / norm), with
    norm = inv_scale * sqrt(sum of all g^2) returned as a 1-element FP32
    tensor.  A norm that is not finite clips nothing."""
    if torch is None:
        _need_torch()
    dev = _device(grads[0], "gradients") if len(grads) else torch.cuda.current_device()
    T = torch.Tensor                      # (mapped methods: a list may hold hundreds of tensors)
    if not set(map(T.get_device, grads)) <= {dev} or not all(map(T.is_contiguous, grads)):
        raise ValueError("gradients must be contiguous, on the current CUDA device")
    ptrs, sizes = list(map(T.data_ptr, grads)), list(map(T.numel, grads))
    dtypes = [g.dtype for g in grads]
    codes = [_CODE[t] for t in dtypes]
    outs = None
    if outputs is not None:
        if len(outputs) != len(grads):
            raise ValueError("as many outputs as gradients")
        if list(map(T.numel, outputs)) != sizes or [o.dtype for o in outputs] != dtypes or \
                not set(map(T.get_device, outputs)) <= {dev} or not all(map(T.is_contiguous, outputs)):
            raise ValueError("an output must be contiguous, of its gradient's dtype, size and device")
        outs = list(map(T.data_ptr, outputs))
    if norm is None:
        norm = _empty(1, torch.float32, dev, stream)
    elif norm.dtype != torch.float32 or norm.numel() != 1 or norm.get_device() != dev:
        raise ValueError("norm must be one FP32 element on the current CUDA device")
    if workspace is None:
        workspace = _empty(lib.grad_clip_workspace(len(ptrs), 0), torch.uint8, dev, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous, on the current CUDA device")
    st = grad_clip_raw(ptrs, outs, sizes, codes, max_norm, inv_scale, norm.data_ptr(),
                       workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                       _stream(dev) if stream is None else stream)
    if st != 0:
        raise GemmError(st, "grad_clip")
    return norm


# -------------------------------------------- tokens sorted by expert and back

def expert_sort_raw(T, k, E, ids, ldids, id_bytes, pos, offsets, order=0, stream=0) -> int:
    """Raw C-ABI call (include/expert_sm103.h); order 0: not wanted.  Returns the
    gemm_status_t code."""
    return lib.expert_sort(T, k, E, ids or None, ldids, id_bytes, pos or None, offsets or None,
                           order or None, stream)


def expert_rows_raw(name, T, k, D, rows, *args, weights=None, stream=0) -> int:
    """Raw C-ABI call of ``name`` (expert_gather, expert_combine or one's backward
    pass); args as in the header, between rows and w; `weights` an ExpertWeights."""
    return getattr(lib, name)(T, k, D, rows, *args, None if weights is None else ctypes.byref(weights),
                              stream)


def expert_sort(ids, experts, pos=None, offsets=None, order=None, stream=None):
    """Sorts the choices of T tokens by expert: (pos, offsets, order).

    ids (T x k, int32 or int64) holds the experts' numbers, 0 .. experts - 1; others
    (-1) choose none.  pos (T x k): the row of each choice, -1 for none; offsets
    (experts + 1): the experts' first rows; order (T * k): the choice t * k + j of
    each row, -1 behind the last.  int32 all, new tensors where None.  Rows are in
    the order of the experts, and of the choices within one."""
    dev = _device(ids, "ids")
    if ids.dim() != 2 or ids.dtype is not torch.int64 and ids.dtype is not torch.int32:
        raise ValueError("ids must be T x k of int32 or int64")
    T, k = ids.shape
    i, ldi = _mat(ids, "ids", T, k, None, dev)
    if pos is None:
        pos = _empty((T, k), torch.int32, dev, stream)
    if offsets is None:
        offsets = _empty((experts + 1,), torch.int32, dev, stream)
    if order is None:
        order = _empty((T * k,), torch.int32, dev, stream)
    st = lib.expert_sort(T, k, experts, i, ldi, ids.element_size(), _pos(pos, T, k, dev),
                         _vec(offsets, "offsets", experts + 1, torch.int32, dev),
                         _vec(order, "order", T * k, torch.int32, dev),
                         _stream(dev) if stream is None else stream)
    if st != 0:
        raise GemmError(st, "expert_sort")
    return pos, offsets, order


def _pos(pos, T, k, dev):
    if pos.shape != (T, k) or pos.dtype is not torch.int32 or pos.get_device() != dev or \
            not pos.is_contiguous():
        if pos.is_contiguous():
            _refuse(pos, "pos", (T, k), torch.int32, dev)
        raise ValueError("pos must be contiguous")
    return pos.data_ptr()


def _expert_weights(weight, dweight, T, k, dev):
    """The weights' argument; None where there are none."""
    if weight is None and dweight is None:
        return None
    w, ldw = _mat(weight, "weight", T, k, None, dev)
    dw, lddw = _mat(dweight, "dweight", T, k, None, dev)
    return ctypes.byref(ExpertWeights(
        w, ldw, GEMM_F32 if weight is None else dtype_code(weight.dtype), dw, lddw,
        GEMM_F32 if dweight is None else dtype_code(dweight.dtype)))


def _expert_shapes(tokens, pos, name):
    dev = _device(tokens, name)
    if tokens.dim() != 2 or pos.dim() != 2:
        raise ValueError(f"{name} and pos must be 2-D")
    return (dev, *tokens.shape, pos.shape[1])


def expert_gather(X, pos, weight=None, Xs=None, stream=None):
    """The tokens' rows to their experts: Xs[pos[t, j]] = weight[t, j] * X[t].

    X is T x D, pos (T x k) expert_sort's, weight T x k or None (1).  Xs has X's
    type and D columns (a new T * k x D tensor where None); rows that pos does not
    name are left as they are.  Returns Xs."""
    dev, T, D, k = _expert_shapes(X, pos, "X")
    if Xs is None:
        Xs = _empty((T * k, D), X.dtype, dev, stream)
    x, ldx = _mat(X, "X", T, D, None, dev)
    xs, ldxs = _mat(Xs, "Xs", Xs.shape[0], D, X.dtype, dev)
    st = lib.expert_gather(T, k, D, Xs.shape[0], x, ldx, _pos(pos, T, k, dev), xs, ldxs,
                           dtype_code(X.dtype), _expert_weights(weight, None, T, k, dev),
                           _stream(dev) if stream is None else stream)
    if st != 0:
        raise GemmError(st, "expert_gather")
    return Xs


def expert_combine(Ys, pos, weight=None, Y=None, stream=None):
    """The experts' rows back to the tokens: Y[t] = sum over j of
    weight[t, j] * Ys[pos[t, j]], in FP32 and rounded once.

    Ys has D columns, pos (T x k) is expert_sort's, weight T x k or None (1); Y is
    T x D of Ys's type (a new tensor where None).  Returns Y."""
    dev, rows, D, k = _expert_shapes(Ys, pos, "Ys")
    T = pos.shape[0]
    if Y is None:
        Y = _empty((T, D), Ys.dtype, dev, stream)
    ys, ldys = _mat(Ys, "Ys", rows, D, None, dev)
    y, ldy = _mat(Y, "Y", T, D, Ys.dtype, dev)
    st = lib.expert_combine(T, k, D, rows, ys, ldys, _pos(pos, T, k, dev), y, ldy,
                            dtype_code(Ys.dtype), _expert_weights(weight, None, T, k, dev),
                            _stream(dev) if stream is None else stream)
    if st != 0:
        raise GemmError(st, "expert_combine")
    return Y


def expert_gather_backward(dXs, pos, weight=None, X=None, dX=None, dweight=None, stream=None):
    """Backward pass of expert_gather into the given tensors (None: not wanted):
    dX[t] = sum over j of weight[t, j] * dXs[pos[t, j]] and
    dweight[t, j] = X[t] . dXs[pos[t, j]] (0 where pos is -1); X only with dweight."""
    dev, rows, D, k = _expert_shapes(dXs, pos, "dXs")
    T = pos.shape[0]
    if dweight is not None and X is None:
        raise ValueError("dweight needs X")
    if dX is None and dweight is None:
        raise ValueError("one of dX and dweight has to be given")
    g, ldg = _mat(dXs, "dXs", rows, D, None, dev)
    x, ldx = _mat(X, "X", T, D, dXs.dtype, dev)
    dx, lddx = _mat(dX, "dX", T, D, dXs.dtype, dev)
    st = lib.expert_gather_backward(T, k, D, rows, g, ldg, x, ldx, _pos(pos, T, k, dev), dx, lddx,
                                    dtype_code(dXs.dtype), _expert_weights(weight, dweight, T, k, dev),
                                    _stream(dev) if stream is None else stream)
    if st != 0:
        raise GemmError(st, "expert_gather_backward")


def expert_combine_backward(dY, pos, weight=None, Ys=None, dYs=None, dweight=None, stream=None):
    """Backward pass of expert_combine into the given tensors (None: not wanted):
    dYs[pos[t, j]] = weight[t, j] * dY[t] and dweight[t, j] = dY[t] . Ys[pos[t, j]]
    (0 where pos is -1); Ys only with dweight.  dYs may be Ys; rows that pos does not
    name are left as they are."""
    dev, T, D, k = _expert_shapes(dY, pos, "dY")
    if dweight is not None and Ys is None:
        raise ValueError("dweight needs Ys")
    if dYs is None and dweight is None:
        raise ValueError("one of dYs and dweight has to be given")
    rows = next((m.shape[0] for m in (dYs, Ys) if m is not None), 0)
    g, ldg = _mat(dY, "dY", T, D, None, dev)
    ys, ldys = _mat(Ys, "Ys", rows, D, dY.dtype, dev)
    dys, lddys = _mat(dYs, "dYs", rows, D, dY.dtype, dev)
    st = lib.expert_combine_backward(T, k, D, rows, g, ldg, ys, ldys, _pos(pos, T, k, dev), dys, lddys,
                                     dtype_code(dY.dtype), _expert_weights(weight, dweight, T, k, dev),
                                     _stream(dev) if stream is None else stream)
    if st != 0:
        raise GemmError(st, "expert_combine_backward")


# ------------------------------------------------------ the orthogonalised update

def ortho_update(h, batch, rows, cols, G, ldg, stride_g, g_dtype, O, ldo, stride_o, coefficients,
                 eps=1e-7, scale=1.0, stream=0) -> int:
    """Raw C-ABI call (include/ortho_sm103.h); coefficients: 3 floats per step.
    Returns the gemm_status_t code."""
    abc = array.array("f", coefficients)
    if len(abc) % 3:
        raise ValueError("coefficients: three for each step")
    o = OrthoUpdate(len(abc) // 3, abc.buffer_info()[0], eps, scale)
    return lib.ortho_update(h, batch, rows, cols, G or None, ldg, stride_g, g_dtype, O or None, ldo,
                            stride_o, ctypes.byref(o), stream)


def ortho_workspace(batch, rows, cols) -> int:
    """Bytes of the handle's workspace that ortho_update takes."""
    return lib.ortho_workspace(batch, rows, cols)


def dtype_code(t) -> int:
    if not _CODE:
        _need_torch()
    return _CODE[t]


class Gemm:
    """A library handle bound to the current CUDA device.

    ``g(A, B, C, transA, transB, alpha, beta, M=, N=, K=)`` marshals torch
    tensors (device, 2-D, unit inner stride, row pitch = stride(0)) into one
    gemm_run call on the current torch stream.  The logical sizes default to
    what the stored shapes imply."""

    def __init__(self):
        self.h = gemm_create()

    def close(self):
        if self.h:
            gemm_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __call__(self, A, B, C, transA="N", transB="N", alpha=1.0, beta=0.0,
                 M=None, N=None, K=None, stream=None, bias=None, act=None):
        import torch
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        for t in (A, B, C):
            if t is not None and (t.dim() != 2 or t.stride(1) != 1):
                raise ValueError("operands must be 2-D with unit inner stride")
        if M is None:
            M = C.shape[0]
        if N is None:
            N = C.shape[1]
        if K is None:
            K = A.shape[1] if transA in "Nn" else A.shape[0]
        dts = (dtype_code(A.dtype), dtype_code(B.dtype), dtype_code(C.dtype))
        if bias is None and act is None:
            st = gemm_run(self.h, transA, transB, M, N, K, alpha, A.data_ptr(), A.stride(0),
                          B.data_ptr(), B.stride(0), beta, C.data_ptr(), C.stride(0), dts, stream)
        else:
            st = gemm_run_ex(self.h, transA, transB, M, N, K, alpha, A.data_ptr(), A.stride(0),
                             B.data_ptr(), B.stride(0), beta, C.data_ptr(), C.stride(0), dts,
                             bias.data_ptr() if bias is not None else 0,
                             dtype_code(bias.dtype) if bias is not None else GEMM_F32,
                             ACTIVATIONS[act] if not isinstance(act, int) else act, stream)
        if st != 0:
            raise GemmError(st, "gemm_run")
        return C

    def layernorm(self, A, B, C, transA="N", transB="N", alpha=1.0, beta=1.0, bias=None,
                  gamma=None, shift=None, eps=1e-5, M=None, N=None, K=None, stream=None):
        """LayerNorm after the linear layer, in place on C (the residual when
        beta != 0): C <- (h - mean) / sqrt(var + eps) * gamma + shift per row,
        h = round_C(alpha*op(A)op(B) + beta*C + bias).  gamma and shift share
        one dtype."""
        import torch
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        for t in (A, B, C):
            if t is not None and (t.dim() != 2 or t.stride(1) != 1):
                raise ValueError("operands must be 2-D with unit inner stride")
        if gamma is not None and shift is not None and gamma.dtype != shift.dtype:
            raise ValueError("gamma and shift must share a dtype")
        M = C.shape[0] if M is None else M
        N = C.shape[1] if N is None else N
        if K is None:
            K = A.shape[1] if transA in "Nn" else A.shape[0]
        ln_t = gamma if gamma is not None else shift
        dts = (dtype_code(A.dtype), dtype_code(B.dtype), dtype_code(C.dtype))
        st = gemm_run_layernorm(
            self.h, transA, transB, M, N, K, alpha, A.data_ptr(), A.stride(0), B.data_ptr(),
            B.stride(0), beta, C.data_ptr(), C.stride(0), dts,
            bias.data_ptr() if bias is not None else 0,
            dtype_code(bias.dtype) if bias is not None else GEMM_F32,
            gamma.data_ptr() if gamma is not None else 0,
            shift.data_ptr() if shift is not None else 0,
            dtype_code(ln_t.dtype) if ln_t is not None else GEMM_F32, eps, stream)
        if st != 0:
            raise GemmError(st, "gemm_run_layernorm")
        return C

    def glu(self, X, W, H=None, act="silu", bias=None, P=None, stream=None):
        """The gated linear layer: H = act(X Wg^T + bg) * (X Wu^T + bu), with
        W = [Wg; Wu] (2F x K) and bias = [bg; bu] (2F) or None.  X is M x K, H
        M x F (a new tensor of X's type where None).  P (M x 2F, H's type)
        receives X W^T + bias for the backward pass."""
        dev = _device(X, "X")
        if X.dim() != 2 or W.dim() != 2 or W.shape[0] % 2:
            raise ValueError("X must be M x K and W 2F x K")
        M, K = X.shape
        F = W.shape[0] // 2
        xt = X.dtype
        if H is None:
            H = _empty((M, F), xt, dev, stream)
        x, ldx = _mat(X, "X", M, K, xt, dev)
        w, ldw = _mat(W, "W", 2 * F, K, xt, dev)
        hp, ldh = _mat(H, "H", M, F, None, dev)
        pp, ldp = _mat(P, "P", M, 2 * F, H.dtype, dev)
        c = _CODE[xt]
        st = glu_forward(self.h, M, F, K, x, ldx, w, ldw, hp, ldh, (c, c, _CODE[H.dtype]),
                         act if isinstance(act, int) else ACTIVATIONS[act],
                         _vec(bias, "bias", 2 * F, None, dev),
                         GEMM_F32 if bias is None else _CODE[bias.dtype], pp, ldp,
                         _stream(dev) if stream is None else stream)
        if st != 0:
            raise GemmError(st, "glu_forward")
        return H

    def glu_backward(self, dH, P, X, W, act="silu", dP=None, dX=None, dW=None, dbias=None,
                     beta_w=0.0, stream=None):
        """Backward pass of `glu` from dH (M x F) and the stored P (M x 2F):
        dP (a new tensor where None; may be P itself), and dX (M x K),
        dW (2F x K, beta_w * dW added) and dbias (2F) where given.  X may be
        None without dW, W without dX.  Returns dP."""
        dev = _device(dH, "dH")
        if dH.dim() != 2:
            raise ValueError("dH must be M x F")
        M, F = dH.shape
        t = dH.dtype
        if dP is None:
            dP = _empty((M, 2 * F), t, dev, stream)
        if dX is not None and W is None or dW is not None and X is None:
            raise ValueError("dX needs W and dW needs X")
        K = next((v.shape[-1] for v in (X, W, dX, dW) if v is not None), 0)
        h_, ldh = _mat(dH, "dH", M, F, t, dev)
        p, ldp = _mat(P, "P", M, 2 * F, None, dev)
        dp, lddp = _mat(dP, "dP", M, 2 * F, t, dev)
        x, ldx = _mat(X, "X", M, K, t, dev)
        w, ldw = _mat(W, "W", 2 * F, K, t, dev)
        dx, lddx = _mat(dX, "dX", M, K, None, dev)
        dw, lddw = _mat(dW, "dW", 2 * F, K, None, dev)
        st = glu_backward(self.h, M, F, K, h_, ldh, p, ldp, x, ldx or max(K, 1), w, ldw or max(K, 1),
                          _CODE[t], dp, lddp, act if isinstance(act, int) else ACTIVATIONS[act],
                          _CODE[P.dtype], dx, lddx, GEMM_F32 if dX is None else _CODE[dX.dtype], dw,
                          lddw, GEMM_F32 if dW is None else _CODE[dW.dtype], beta_w,
                          _vec(dbias, "dbias", 2 * F, None, dev),
                          GEMM_F32 if dbias is None else _CODE[dbias.dtype],
                          _stream(dev) if stream is None else stream)
        if st != 0:
            raise GemmError(st, "glu_backward")
        return dP

    def orthogonalize(self, G, O=None, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7,
                      scale=1.0, stream=None):
        """The update G brought near orthonormal rows or columns by Newton-Schulz
        steps (as the Muon optimiser does): X = G / (||G|| + eps), then `steps`
        times X = a X + (b A + c A^2) X with A = X X^T (on the shorter side);
        returns O = scale * X in BF16 (a new tensor where None).

        G is rows x cols, or a batch of such, of any type; coefficients are one
        (a, b, c) or one for each step.  O may be G."""
        dev = _device(G, "G")
        if G.dim() not in (2, 3):
            raise ValueError("G must be rows x cols, or batch x rows x cols")
        if O is None:
            O = _empty(tuple(G.shape), torch.bfloat16, dev, stream)
        if O.dim() != G.dim():
            raise ValueError("O must have G's shape")
        batch, sg, so, g, o = 1, 0, 0, G, O
        if G.dim() == 3:
            batch, sg, so = G.shape[0], G.stride(0), O.stride(0)
            if O.shape != G.shape:
                _refuse(O, "O", tuple(G.shape), torch.bfloat16, dev)
            if batch == 0:
                return O
            g, o = G[0], O[0]
        rows, cols = g.shape
        gp, ldg = _mat(g, "G", rows, cols, None, dev)
        op, ldo = _mat(o, "O", rows, cols, torch.bfloat16, dev)
        if len(coefficients) == 3 and not hasattr(coefficients[0], "__len__"):
            abc = tuple(coefficients) * steps
        elif len(coefficients) == steps and all(hasattr(c, "__len__") and len(c) == 3 for c in coefficients):
            abc = [v for step in coefficients for v in step]
        else:
            raise ValueError("coefficients: one (a, b, c), or one for each step")
        st = ortho_update(self.h, batch, rows, cols, gp, ldg, sg, dtype_code(G.dtype), op, ldo, so, abc, eps,
                          scale, _stream(dev) if stream is None else stream)
        if st != 0:
            raise GemmError(st, "ortho_update")
        return O

    def sync(self, stream=None):
        import torch
        if stream is None:
            stream = torch.cuda.current_stream().cuda_stream
        st = gemm_sync(self.h, stream)
        if st != 0:
            raise GemmError(st, "gemm_sync")
