"""Python binding of libdg (ctypes): argument marshalling only.

Every step of the GEMM runs in libdg's CUDA kernels.  This module loads the
in-tree ``libdg.so`` (built by ``precision_matmul_dg_gb300.build``), declares
the C signatures of ``include/dg.h`` and turns tensors into pointers and
leading dimensions.  PyTorch is used for device memory and streams only.
There is no fallback: if the library is missing, every call raises.
"""

import ctypes
import os

__all__ = [
    "DgError", "F16", "I8", "E2M1", "EPILOGUES", "lib", "lib_path", "gemm", "gemm_raw",
    "gemm_host", "gemm_host_raw", "gemm_ex", "gemm_ex_raw", "gemm_batched", "gemm_grouped",
    "gemm_strided_batched_raw", "prepare_grouped", "OPS", "MAX_EPILOGUE_OPS", "MXF4", "quantize_mxf4",
    "quantize_mxf4_raw", "gemm_mxf4", "gemm_mxf4_raw",
    "EpilogueOp", "EpilogueProgram", "make_program",
    "quantize_fp8", "gemm_fp8", "gemm_fp8_grouped", "gemm_fp8_grouped_wgrad", "moe_rows",
    "moe_sort", "moe_dispatch", "moe_dispatch_fp8", "moe_combine", "moe_combine_backward",
    "plan_tiles", "query_hw", "last_error", "check_status", "set_wait_timeout_ns",
    "selftest_wait_timeout", "launch_count", "shutdown", "HwDesc", "TilePlan", "EXPORTS",
]

F16, I8, E2M1, MXF4, BF16, F32 = 0, 1, 2, 3, 4, 5
DTYPES = {"f16": F16, "i8": I8, "e2m1": E2M1, "mxf4": MXF4}
EPILOGUES = {"none": 0, "bias": 1, "gelu": 2, "bias_gelu": 3}
OPS = {"bias": 1, "relu": 2, "gelu": 3, "scale": 4, "clamp": 5, "quant_i8": 6}
MAX_EPILOGUE_OPS = 8
STATUS = {0: "DG_OK", 1: "DG_ERR_INVALID_ARG", 2: "DG_ERR_UNSUPPORTED",
          3: "DG_ERR_NO_VALID_CANDIDATE", 4: "DG_ERR_CUDA", 5: "DG_ERR_TIMEOUT",
          6: "DG_ERR_INVALID_STATE"}
KERNELS = {0: "tc", 1: "gemv", 2: "tc_widened", 3: "skinny", 4: "gemv_mma", 5: "tc_streamk",
           -1: "none"}

# Every symbol include/dg.h declares.
EXPORTS = ["dg_query_hw", "dg_plan_tiles", "dg_gemm", "dg_gemm_planned", "dg_gemm_host",
           "dg_gemm_ex", "dg_gemm_strided_batched", "dg_gemm_grouped",
           "dg_quantize_mxf4", "dg_gemm_mxf4", "dg_gemm_mxf4_planned",
           "dg_quantize_fp8", "dg_gemm_fp8", "dg_gemm_fp8_grouped", "dg_gemm_fp8_grouped_wgrad",
           "dg_moe_rows", "dg_moe_sort", "dg_moe_dispatch", "dg_moe_dispatch_fp8",
           "dg_moe_dispatch_fp8_scratch", "dg_moe_dispatch_fp8_ex",
           "dg_moe_combine", "dg_moe_combine_backward",
           "dg_gemm_thin_noalloc", "dg_last_error",
           "dg_check_status", "dg_set_wait_timeout_ns", "dg_selftest_wait_timeout",
           "dg_launch_count", "dg_shutdown"]

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path():
    return os.path.join(_HERE, "libdg.so")


class DgError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__("%s: %s" % (self.name, message))


class HwDesc(ctypes.Structure):
    _fields_ = [("sm_count", ctypes.c_int), ("cc_major", ctypes.c_int), ("cc_minor", ctypes.c_int),
                ("smem_per_block_optin", ctypes.c_int), ("smem_per_sm", ctypes.c_int),
                ("regs_per_sm", ctypes.c_int), ("regs_per_thread_max", ctypes.c_int),
                ("max_threads_per_sm", ctypes.c_int), ("tmem_cols", ctypes.c_int),
                ("l2_bytes", ctypes.c_int64), ("hbm_gbps", ctypes.c_double),
                ("tc_f16_tflops", ctypes.c_double), ("clock_ghz", ctypes.c_double)]

    def as_dict(self):
        return {f[0]: getattr(self, f[0]) for f in self._fields_}


class TilePlan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("m_tile", ctypes.c_int), ("n_tile", ctypes.c_int),
                ("k_tile", ctypes.c_int), ("split_k", ctypes.c_int), ("stages", ctypes.c_int),
                ("cta_group", ctypes.c_int), ("swap_ab", ctypes.c_int),
                ("smem_bytes", ctypes.c_int), ("threads", ctypes.c_int),
                ("regs_per_thread", ctypes.c_int), ("grid", ctypes.c_int),
                ("occupancy", ctypes.c_double), ("est_us", ctypes.c_double),
                ("est_tflops", ctypes.c_double)]

    def as_dict(self):
        d = {f[0]: getattr(self, f[0]) for f in self._fields_}
        d["kernel_name"] = KERNELS.get(self.kernel, str(self.kernel))
        return d


_lib = None


class EpilogueOp(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("a", ctypes.c_float), ("b", ctypes.c_float)]


class EpilogueProgram(ctypes.Structure):
    _fields_ = [("n_ops", ctypes.c_int), ("ops", EpilogueOp * MAX_EPILOGUE_OPS)]


def make_program(ops):
    """EpilogueProgram from a list of ops: "relu", "gelu", "bias",
    ("scale", a), ("clamp", lo, hi), ("quant_i8", a) (last op: int8 D), or
    (type_code, a, b)."""
    ops = list(ops)
    if len(ops) > MAX_EPILOGUE_OPS:
        raise ValueError("at most %d epilogue ops" % MAX_EPILOGUE_OPS)
    prog = EpilogueProgram()
    prog.n_ops = len(ops)
    for k, op in enumerate(ops):
        if isinstance(op, str):
            op = (op,)
        code = OPS[op[0]] if isinstance(op[0], str) else int(op[0])
        args = [float(x) for x in op[1:]] + [0.0, 0.0]
        prog.ops[k] = EpilogueOp(code, args[0], args[1])
    return prog


def lib():
    """The loaded libdg.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError("libdg.so is not built (%s); run __graft_entry__.build()" % path)
    L = ctypes.CDLL(path)
    i64, vp, i32, f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.dg_query_hw.argtypes = [i32, ctypes.POINTER(HwDesc)]
    L.dg_plan_tiles.argtypes = [i64, i64, i64, i32, i32, i32, ctypes.POINTER(HwDesc),
                                ctypes.c_double, ctypes.POINTER(TilePlan), i32,
                                ctypes.POINTER(ctypes.c_int)]
    gemm_args = [i64, i64, i64, i32, i32, vp, i64, vp, i64, vp, vp, f32, f32, i32]
    L.dg_gemm.argtypes = gemm_args + [vp]
    L.dg_gemm_planned.argtypes = gemm_args + [ctypes.POINTER(TilePlan), vp]
    L.dg_gemm_thin_noalloc.argtypes = gemm_args + [vp]
    L.dg_gemm_host.argtypes = [i64, i64, i64, i32, i32, vp, i64, vp, i64, vp, vp, vp, f32, f32,
                               i32, vp]
    L.dg_gemm_strided_batched.argtypes = [i64, i64, i64, i64, i32, i32, vp, i64, i64, vp, i64,
                                          i64, vp, i64, vp, i64, f32, f32, i32, vp]
    L.dg_gemm_grouped.argtypes = [i64, ctypes.POINTER(ctypes.c_int64), i64, i64, i32, i32,
                                  ctypes.POINTER(vp), i64, ctypes.POINTER(vp), i64,
                                  ctypes.POINTER(vp), ctypes.POINTER(vp), f32, f32, i32, vp]
    L.dg_gemm_ex.argtypes = [i64, i64, i64, i32, i32, vp, i64, vp, i64, vp, i64, vp, i64, vp, f32,
                             f32, ctypes.POINTER(EpilogueProgram), vp]
    L.dg_quantize_mxf4.argtypes = [i64, i64, vp, i64, vp, i64, vp, i64, vp]
    L.dg_gemm_mxf4.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, f32,
                               f32, i32, vp]
    L.dg_gemm_mxf4_planned.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp,
                                       f32, f32, i32, ctypes.POINTER(TilePlan), vp]
    L.dg_quantize_fp8.argtypes = [i64, i64, i32, vp, i64, i32, vp, i64, vp, i64, vp, i64, vp, i64,
                                  vp]
    L.dg_gemm_fp8.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, vp, i32, i64,
                              vp, f32, f32, i32, vp]
    L.dg_gemm_fp8_grouped.argtypes = [i64, i64, i64, i64, vp, i64, vp, i64, vp, i64, i64, vp, i64,
                                      i64, vp, vp, i32, i64, vp, i64, f32, f32, i32, vp]
    L.dg_gemm_fp8_grouped_wgrad.argtypes = [i64, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                            vp, vp, i32, i64, i64, f32, f32, vp]
    L.dg_moe_rows.argtypes = [i64, i64, i64, i64]
    L.dg_moe_rows.restype = ctypes.c_int64
    L.dg_moe_sort.argtypes = [i64, i64, i64, vp, i64, i64, vp, vp, vp, vp]
    L.dg_moe_dispatch.argtypes = [i64, i64, i64, i32, vp, i64, i64, vp, vp, i64, vp]
    L.dg_moe_dispatch_fp8.argtypes = [i64, i64, i64, i32, vp, i64, i64, vp, vp, i64, vp, i64, vp]
    L.dg_moe_dispatch_fp8_scratch.argtypes = [i64, i64, i64, i64]
    L.dg_moe_dispatch_fp8_scratch.restype = ctypes.c_int64
    L.dg_moe_dispatch_fp8_ex.argtypes = [i64, i64, i64, i32, vp, i64, i64, vp, vp, i64, vp, i64, vp,
                                         i64, vp]
    L.dg_moe_combine.argtypes = [i64, i64, i64, i32, vp, i64, i64, vp, vp, vp, i64, vp]
    L.dg_moe_combine_backward.argtypes = [i64, i64, i64, i32, vp, i64, vp, i64, i64, vp, vp, vp,
                                          vp, i64, vp, vp]
    L.dg_last_error.restype = ctypes.c_char_p
    L.dg_last_error.argtypes = []
    L.dg_check_status.argtypes = [vp]
    L.dg_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    L.dg_selftest_wait_timeout.argtypes = [vp]
    L.dg_launch_count.restype = ctypes.c_uint64
    L.dg_launch_count.argtypes = []
    L.dg_shutdown.argtypes = []
    for name in ("dg_query_hw", "dg_plan_tiles", "dg_gemm", "dg_gemm_planned",
                 "dg_gemm_thin_noalloc", "dg_gemm_host", "dg_gemm_ex", "dg_gemm_strided_batched",
                 "dg_gemm_grouped", "dg_quantize_mxf4", "dg_gemm_mxf4", "dg_gemm_mxf4_planned",
                 "dg_quantize_fp8", "dg_gemm_fp8", "dg_gemm_fp8_grouped",
                 "dg_gemm_fp8_grouped_wgrad", "dg_moe_sort", "dg_moe_dispatch",
                 "dg_moe_dispatch_fp8", "dg_moe_dispatch_fp8_ex", "dg_moe_combine",
                 "dg_moe_combine_backward", "dg_check_status",
                 "dg_set_wait_timeout_ns", "dg_selftest_wait_timeout", "dg_shutdown"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def last_error():
    return lib().dg_last_error().decode()


def _check(status):
    if status != 0:
        raise DgError(status, last_error())


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream_handle(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(d):
    return DTYPES[d] if isinstance(d, str) else int(d)


def _epi_code(e):
    return EPILOGUES[e] if isinstance(e, str) else int(e)


def gemm_raw(M, N, K, dtype_a, dtype_b, A, lda, B, ldb, C, bias, alpha, beta, epilogue,
             stream=None, plan=None):
    """dg_gemm / dg_gemm_planned with the C argument order.  A, B, C, bias are
    tensors or raw device addresses; dtypes and epilogue are names or codes."""
    L = lib()
    args = (int(M), int(N), int(K), _dtype_code(dtype_a), _dtype_code(dtype_b), _ptr(A), int(lda),
            _ptr(B), int(ldb), _ptr(C), _ptr(bias), float(alpha), float(beta),
            _epi_code(epilogue))
    s = _stream_handle(stream)
    if plan is None:
        _check(L.dg_gemm(*args, s))
    else:
        _check(L.dg_gemm_planned(*args, ctypes.byref(_as_plan(plan)), s))


_TORCH_DTYPES = None


def _expect(t, kinds, what):
    import torch
    global _TORCH_DTYPES
    if _TORCH_DTYPES is None:
        _TORCH_DTYPES = {"f16": torch.float16, "i8": torch.int8, "e2m1": torch.uint8,
                         "i32": torch.int32}
    if t.dtype != _TORCH_DTYPES[kinds]:
        raise TypeError("%s must be %s, got %s" % (what, _TORCH_DTYPES[kinds], t.dtype))
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("%s must be 2-D with unit column stride" % what)


_TD = None  # (torch, B dtype -> code, code -> torch dtype), built on first use


def _td():
    global _TD
    if _TD is None:
        import torch
        _TD = (torch, {torch.float16: F16, torch.int8: I8, torch.uint8: E2M1},
               (torch.float16, torch.int8, torch.uint8))
    return _TD


def gemm(A, B, C, K=None, bias=None, alpha=1.0, beta=0.0, epilogue="none", dtype_b=None,
         stream=None, plan=None):
    """D = epilogue(alpha * A.B + beta * C), written into C.

    A: [M, lda] (fp16 or int8); B: [N, ldb] (fp16/int8) or [N, ldb/2] uint8
    packed E2M1 codes; C: [M, N] fp16 (int32 for int8); K defaults to
    A.shape[1]; bias: [N] fp16.  The leading dimensions are the row strides.
    (Written for a short host path: small GEMMs are bound by it.)
    """
    torch, b_code, code_dt = _TD or _td()
    da = I8 if A.dtype is torch.int8 else F16
    db = b_code[B.dtype] if dtype_b is None else _dtype_code(dtype_b)
    sa, sb, sc = A.stride(), B.stride(), C.stride()
    names = ("f16", "i8", "e2m1")
    if A.dtype is not code_dt[da] or len(sa) != 2 or sa[1] != 1:
        _expect(A, names[da], "A")
    if B.dtype is not code_dt[db] or len(sb) != 2 or sb[1] != 1:
        _expect(B, names[db], "B")
    if C.dtype is not (torch.int32 if da == I8 else torch.float16) or len(sc) != 2 or sc[1] != 1:
        _expect(C, "i32" if da == I8 else "f16", "C")
    M, N = C.shape
    if A.shape[0] != M or B.shape[0] != N:
        raise ValueError("shape mismatch: A %s, B %s, C %s" % (tuple(A.shape), tuple(B.shape),
                                                               tuple(C.shape)))
    if sc[0] != N:
        raise ValueError("C must be dense row-major (leading dimension N)")
    if K is None:
        K = A.shape[1]
    ldb = sb[0] * (2 if db == E2M1 else 1)
    if plan is not None:
        gemm_raw(M, N, K, da, db, A, sa[0], B, ldb, C, bias, alpha, beta, epilogue,
                 stream=stream, plan=plan)
        return C
    s = _stream_handle(stream)
    _check(lib().dg_gemm(M, N, K, da, db, A.data_ptr(), sa[0], B.data_ptr(), ldb, C.data_ptr(),
                         None if bias is None else bias.data_ptr(), alpha, beta,
                         EPILOGUES[epilogue] if isinstance(epilogue, str) else int(epilogue), s))
    return C


def quantize_mxf4_raw(rows, K, X, ldx, codes, ldq, scales, lds, stream=None):
    """dg_quantize_mxf4 with the C argument order (ldq in codes, lds in bytes)."""
    _check(lib().dg_quantize_mxf4(int(rows), int(K), _ptr(X), int(ldx), _ptr(codes), int(ldq),
                                  _ptr(scales), int(lds), _stream_handle(stream)))


def quantize_mxf4(X, K=None, stream=None):
    """MXFP4 block quantization of the fp16 rows X [rows, >= K] along K.

    Returns (codes, scales): codes uint8 [rows, ldq / 2] (two E2M1 codes per
    byte, ldq = K rounded up to 32), scales uint8 [rows, ceil(K / 32)] (E8M0).
    """
    import torch
    _expect(X, "f16", "X")
    rows = X.shape[0]
    K = X.shape[1] if K is None else int(K)
    ldq = (K + 31) // 32 * 32
    nblk = (K + 31) // 32
    codes = torch.zeros((rows, ldq // 2), dtype=torch.uint8, device=X.device)
    scales = torch.zeros((rows, nblk), dtype=torch.uint8, device=X.device)
    quantize_mxf4_raw(rows, K, X, X.stride(0), codes, ldq, scales, nblk, stream)
    return codes, scales


def _as_plan(plan):
    if isinstance(plan, dict):
        return TilePlan(**{k: v for k, v in plan.items() if k in dict(TilePlan._fields_)})
    return plan


def gemm_mxf4_raw(M, N, K, A, lda, scale_a, lds_a, B, ldb, scale_b, lds_b, C, bias, alpha, beta,
                  epilogue="none", stream=None, plan=None):
    """dg_gemm_mxf4 (dg_gemm_mxf4_planned with a plan) with the C argument
    order (lda, ldb in codes)."""
    epi = EPILOGUES[epilogue] if isinstance(epilogue, str) else int(epilogue)
    args = (int(M), int(N), int(K), _ptr(A), int(lda), _ptr(scale_a), int(lds_a), _ptr(B),
            int(ldb), _ptr(scale_b), int(lds_b), _ptr(C), _ptr(bias), float(alpha), float(beta),
            epi)
    if plan is None:
        _check(lib().dg_gemm_mxf4(*args, _stream_handle(stream)))
    else:
        _check(lib().dg_gemm_mxf4_planned(*args, ctypes.byref(_as_plan(plan)),
                                          _stream_handle(stream)))


def gemm_mxf4(A, scale_a, B, scale_b, C, K, bias=None, alpha=1.0, beta=0.0, epilogue="none",
              stream=None, plan=None):
    """D = epilogue(alpha * A.B + beta * C) for MXFP4 A and B, written into C.

    A: uint8 [M, lda / 2] packed codes with scale_a uint8 [M, >= ceil(K/32)];
    B: uint8 [N, ldb / 2] with scale_b [N, ...]; C: fp16 [M, N] dense.
    plan: a dg_plan_tiles candidate for (M, N, K, "mxf4", "mxf4") to run
    instead of the planner's first.
    """
    for t, what in ((A, "A"), (B, "B"), (scale_a, "scale_a"), (scale_b, "scale_b")):
        _expect(t, "e2m1", what)
    _expect(C, "f16", "C")
    M, N = C.shape
    if A.shape[0] != M or B.shape[0] != N or scale_a.shape[0] != M or scale_b.shape[0] != N:
        raise ValueError("shape mismatch")
    if C.stride(0) != N:
        raise ValueError("C must be dense row-major (leading dimension N)")
    gemm_mxf4_raw(M, N, K, A, 2 * A.stride(0), scale_a, scale_a.stride(0), B, 2 * B.stride(0),
                  scale_b, scale_b.stride(0), C, bias, alpha, beta, epilogue, stream, plan)
    return C


def gemm_ex_raw(M, N, K, dtype_a, dtype_b, A, lda, B, ldb, C, ldc, D, ldd, bias, alpha, beta,
                program=None, stream=None):
    """dg_gemm_ex with the C argument order.  program: None, an
    EpilogueProgram, or a list of ops for make_program."""
    if program is not None and not isinstance(program, EpilogueProgram):
        program = make_program(program)
    args = (int(M), int(N), int(K), _dtype_code(dtype_a), _dtype_code(dtype_b), _ptr(A), int(lda),
            _ptr(B), int(ldb), _ptr(C), int(ldc), _ptr(D), int(ldd), _ptr(bias), float(alpha),
            float(beta), ctypes.byref(program) if program is not None else None,
            _stream_handle(stream))
    _check(lib().dg_gemm_ex(*args))


def gemm_ex(A, B, D, C=None, K=None, bias=None, alpha=1.0, beta=0.0, program=(), dtype_b=None,
            stream=None):
    """D = program(alpha * A.B + beta * C) with C read and D written.

    A and B as in gemm(); C and D are [M, N] views with unit column stride
    and any row stride (leading dimension) >= N, e.g. column slices of wider
    buffers; C may be D itself.  program: list of ops, applied in order
    ("bias", "relu", "gelu", ("scale", a), ("clamp", lo, hi)); a program
    ending in ("quant_i8", a) writes an int8 D (C, when given, stays fp16).
    """
    import torch
    dtype_a = "i8" if A.dtype == torch.int8 else "f16"
    if dtype_b is None:
        dtype_b = {torch.float16: "f16", torch.int8: "i8", torch.uint8: "e2m1"}[B.dtype]
    _expect(A, dtype_a, "A")
    _expect(B, dtype_b, "B")
    out = "i32" if dtype_a == "i8" else "f16"
    ops = list(program or [])
    last = ops[-1] if ops else None
    quant = last is not None and (last[0] if isinstance(last, tuple) else last) in ("quant_i8", 6)
    _expect(D, "i8" if quant else out, "D")
    M, N = D.shape
    ldc = D.stride(0)
    if C is not None:
        _expect(C, out, "C")
        if tuple(C.shape) != (M, N):
            raise ValueError("C must be [M, N] like D")
        ldc = C.stride(0)
    if A.shape[0] != M or B.shape[0] != N:
        raise ValueError("shape mismatch: A %s, B %s, D %s" % (tuple(A.shape), tuple(B.shape),
                                                               tuple(D.shape)))
    if K is None:
        K = A.shape[1]
    ldb = B.stride(0) * (2 if dtype_b == "e2m1" else 1)
    gemm_ex_raw(M, N, K, dtype_a, dtype_b, A, A.stride(0), B, ldb, C, ldc, D, D.stride(0), bias,
                alpha, beta, program=make_program(ops), stream=stream)
    return D


def gemm_strided_batched_raw(batch, M, N, K, dtype_a, dtype_b, A, lda, stride_a, B, ldb, stride_b,
                             C, stride_c, bias, stride_bias, alpha, beta, epilogue, stream=None):
    """dg_gemm_strided_batched with the C argument order."""
    args = (int(batch), int(M), int(N), int(K), _dtype_code(dtype_a), _dtype_code(dtype_b),
            _ptr(A), int(lda), int(stride_a), _ptr(B), int(ldb), int(stride_b), _ptr(C),
            int(stride_c), _ptr(bias), int(stride_bias), float(alpha), float(beta),
            _epi_code(epilogue), _stream_handle(stream))
    _check(lib().dg_gemm_strided_batched(*args))


def gemm_batched(A, B, C, K=None, bias=None, alpha=1.0, beta=0.0, epilogue="none",
                 dtype_b=None, stream=None):
    """D_z = epilogue(alpha * A_z.B_z + beta * C_z) for every z, written into C.

    A: [batch, M, lda]; B: [batch, N, ldb] or [N, ldb] (shared by all
    problems; uint8 packed codes for E2M1); C: [batch, M, N], each [M, N]
    dense; bias: [batch, N] or [N] (shared).  The batch strides are the
    tensors' first-dimension strides.
    """
    import torch
    dtype_a = "i8" if A.dtype == torch.int8 else "f16"
    if dtype_b is None:
        dtype_b = {torch.float16: "f16", torch.int8: "i8", torch.uint8: "e2m1"}[B.dtype]
    if A.dim() != 3 or C.dim() != 3 or B.dim() not in (2, 3):
        raise ValueError("A and C must be 3-D, B 2-D or 3-D")
    batch, M, N = C.shape
    _expect(A[0], dtype_a, "A")
    B0 = B[0] if B.dim() == 3 else B
    _expect(B0, dtype_b, "B")
    _expect(C[0], "i32" if dtype_a == "i8" else "f16", "C")
    if A.shape[0] != batch or A.shape[1] != M or B0.shape[0] != N or \
            (B.dim() == 3 and B.shape[0] != batch):
        raise ValueError("shape mismatch: A %s, B %s, C %s" % (tuple(A.shape), tuple(B.shape),
                                                               tuple(C.shape)))
    if C.stride(1) != N:
        raise ValueError("each C[z] must be dense row-major (leading dimension N)")
    if K is None:
        K = A.shape[2]
    codes = 2 if dtype_b == "e2m1" else 1
    ldb = B0.stride(0) * codes
    stride_b = B.stride(0) * codes if B.dim() == 3 else 0
    stride_bias = 0
    if bias is not None and bias.dim() == 2:
        stride_bias = bias.stride(0)
    gemm_strided_batched_raw(batch, M, N, K, dtype_a, dtype_b, A, A.stride(1), A.stride(0), B,
                             ldb, stride_b, C, C.stride(0), bias, stride_bias, alpha, beta,
                             epilogue, stream=stream)
    return C


def prepare_grouped(As, Bs, Cs, K=None, bias=None, alpha=1.0, beta=0.0, epilogue="none"):
    """Checks a group of problems once and returns run(stream=None), which
    issues dg_gemm_grouped on them with the prepared pointer arrays (for a
    group that is run again and again, e.g. one mixture-of-experts layer).
    The tensors must stay alive and keep their storage.  Arguments as
    gemm_grouped."""
    import torch
    count = len(As)
    if not isinstance(Bs, (list, tuple)):
        Bs = [Bs] * count
    if bias is not None and not isinstance(bias, (list, tuple)):
        bias = [bias] * count
    if len(Bs) != count or len(Cs) != count or (bias is not None and len(bias) != count):
        raise ValueError("As, Bs, Cs (and bias) must have one entry per problem")
    if count == 0:
        return lambda stream=None: Cs
    A0, B0 = As[0], Bs[0]
    dtype_a = "i8" if A0.dtype == torch.int8 else "f16"
    dtype_b = {torch.float16: "f16", torch.int8: "i8", torch.uint8: "e2m1"}[B0.dtype]
    N = Cs[0].shape[1]
    if K is None:
        K = A0.shape[1]
    lda = A0.stride(0)
    ldb = B0.stride(0) * (2 if dtype_b == "e2m1" else 1)
    for g in range(count):
        _expect(As[g], dtype_a, "A[%d]" % g)
        _expect(Bs[g], dtype_b, "B[%d]" % g)
        _expect(Cs[g], "i32" if dtype_a == "i8" else "f16", "C[%d]" % g)
        if As[g].stride(0) != lda or Bs[g].stride(0) * (2 if dtype_b == "e2m1" else 1) != ldb:
            raise ValueError("every problem must share lda and ldb")
        if Cs[g].shape[1] != N or Cs[g].shape[0] != As[g].shape[0] or Bs[g].shape[0] != N or \
                (Cs[g].shape[0] and Cs[g].stride(0) != N):
            raise ValueError("problem %d: shapes or C layout do not match" % g)
    vp = ctypes.c_void_p
    Ms = (ctypes.c_int64 * count)(*[int(a.shape[0]) for a in As])
    pa = (vp * count)(*[a.data_ptr() for a in As])
    pb = (vp * count)(*[b.data_ptr() for b in Bs])
    pc = (vp * count)(*[c.data_ptr() for c in Cs])
    pbias = None if bias is None else (vp * count)(*[b.data_ptr() for b in bias])
    args = (count, Ms, int(N), int(K), _dtype_code(dtype_a), _dtype_code(dtype_b), pa, int(lda),
            pb, int(ldb), pc, pbias, float(alpha), float(beta), _epi_code(epilogue))
    fn = lib().dg_gemm_grouped

    def run(stream=None):
        _check(fn(*args, _stream_handle(stream)))
        return Cs
    return run


def gemm_grouped(As, Bs, Cs, K=None, bias=None, alpha=1.0, beta=0.0, epilogue="none",
                 stream=None):
    """D_g = epilogue(alpha * A_g.B_g + beta * C_g) for every g, written into Cs[g].

    As: list of [M_g, lda] tensors (one lda, M_g may differ, 0 skips); Bs: a
    list of [N, ldb] tensors or one tensor shared by all; Cs: list of [M_g, N]
    dense tensors; bias: None, one [N] tensor or a list.  All problems share
    N, K, the dtypes, scalars and epilogue.
    """
    return prepare_grouped(As, Bs, Cs, K, bias, alpha, beta, epilogue)(stream)
    A0, B0 = As[0], Bs[0]
    dtype_a = "i8" if A0.dtype == torch.int8 else "f16"
    dtype_b = {torch.float16: "f16", torch.int8: "i8", torch.uint8: "e2m1"}[B0.dtype]
    N = Cs[0].shape[1]
    if K is None:
        K = A0.shape[1]
    lda = A0.stride(0)
    ldb = B0.stride(0) * (2 if dtype_b == "e2m1" else 1)
    for g in range(count):
        _expect(As[g], dtype_a, "A[%d]" % g)
        _expect(Bs[g], dtype_b, "B[%d]" % g)
        _expect(Cs[g], "i32" if dtype_a == "i8" else "f16", "C[%d]" % g)
        if As[g].stride(0) != lda or Bs[g].stride(0) * (2 if dtype_b == "e2m1" else 1) != ldb:
            raise ValueError("every problem must share lda and ldb")
        if Cs[g].shape[1] != N or Cs[g].shape[0] != As[g].shape[0] or Bs[g].shape[0] != N or \
                (Cs[g].shape[0] and Cs[g].stride(0) != N):
            raise ValueError("problem %d: shapes or C layout do not match" % g)
    vp = ctypes.c_void_p
    Ms = (ctypes.c_int64 * count)(*[int(a.shape[0]) for a in As])
    pa = (vp * count)(*[a.data_ptr() for a in As])
    pb = (vp * count)(*[b.data_ptr() for b in Bs])
    pc = (vp * count)(*[c.data_ptr() for c in Cs])
    pbias = None if bias is None else (vp * count)(*[b.data_ptr() for b in bias])
    _check(lib().dg_gemm_grouped(count, Ms, int(N), int(K), _dtype_code(dtype_a),
                                 _dtype_code(dtype_b), pa, int(lda), pb, int(ldb), pc, pbias,
                                 float(alpha), float(beta), _epi_code(epilogue),
                                 _stream_handle(stream)))
    return Cs


def gemm_host_raw(M, N, K, dtype_a, dtype_b, A, lda, B, ldb, C, D, bias, alpha, beta, epilogue,
                  stream=None):
    """dg_gemm_host with the C argument order: A, B, C, D, bias are host
    tensors (ideally pinned) or raw host addresses."""
    args = (int(M), int(N), int(K), _dtype_code(dtype_a), _dtype_code(dtype_b), _ptr(A), int(lda),
            _ptr(B), int(ldb), _ptr(C), _ptr(D), _ptr(bias), float(alpha), float(beta),
            _epi_code(epilogue), _stream_handle(stream))
    _check(lib().dg_gemm_host(*args))


def gemm_host(A, B, D, C=None, K=None, bias=None, alpha=1.0, beta=0.0, epilogue="none",
              dtype_b=None, stream=None):
    """D = epilogue(alpha * A.B + beta * C) on host (CPU) tensors, copies
    included: the call is asynchronous on `stream`, so synchronise it before
    reading D.  Layouts as gemm(); C (read when beta != 0) and D are [M, N]."""
    import torch
    dtype_a = "i8" if A.dtype == torch.int8 else "f16"
    if dtype_b is None:
        dtype_b = {torch.float16: "f16", torch.int8: "i8", torch.uint8: "e2m1"}[B.dtype]
    for t, what in ((A, "A"), (B, "B"), (D, "D"), (C, "C"), (bias, "bias")):
        if t is not None and t.device.type != "cpu":
            raise ValueError("%s must be a host tensor" % what)
    _expect(A, dtype_a, "A")
    _expect(B, dtype_b, "B")
    out = "i32" if dtype_a == "i8" else "f16"
    _expect(D, out, "D")
    M, N = D.shape
    if C is not None:
        _expect(C, out, "C")
        if tuple(C.shape) != (M, N) or C.stride(0) != N:
            raise ValueError("C must be dense [M, N]")
    if A.shape[0] != M or B.shape[0] != N or D.stride(0) != N:
        raise ValueError("shape mismatch: A %s, B %s, D %s" % (tuple(A.shape), tuple(B.shape),
                                                               tuple(D.shape)))
    if K is None:
        K = A.shape[1]
    ldb = B.stride(0) * (2 if dtype_b == "e2m1" else 1)
    gemm_host_raw(M, N, K, dtype_a, dtype_b, A, A.stride(0), B, ldb, C, D, bias, alpha, beta,
                  epilogue, stream=stream)
    return D


# ------------------------------------------------- FP8 and expert routing

_FP = None  # (torch, {16-bit and 32-bit float dtype: code}), built on first use
_raw_stream = None
_gpus = 0  # that torch sees


def _fp():
    global _FP, _raw_stream, _gpus
    if _FP is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _gpus = torch.cuda.device_count()
        _FP = (torch, {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32})
    return _FP


def _same_gpu(torch, tensors):
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("tensors must be on the current GPU (cuda:%d), got one on %s" % (
                device, t.device))


def _stream_of(stream, *tensors):
    """The handle of `stream`, by default the current one (as
    torch.cuda.current_stream, whose Stream object costs more than a launch),
    for a call on these CUDA tensors (None: not given), which must be on the
    current GPU, where the library launches.  (Where there is one GPU, they are.)"""
    if _gpus != 1:
        _same_gpu(_FP[0], tensors)
    if stream is None and _raw_stream is not None:
        return _raw_stream(tensors[0].get_device())
    return _stream_handle(stream)


def _float_code(t, what, kinds=(F16, BF16)):
    code = (_FP or _fp())[1].get(t.dtype, -1)
    if code not in kinds:
        raise TypeError("%s must be float16%s, got %s" % (
            what, ", bfloat16 or float32" if F32 in kinds else " or bfloat16", t.dtype))
    return code


def _rows(t, dtype, what, shape=None, dim=2):
    """The strides of t, which must be on the GPU, of this type, of `dim`
    dimensions with unit last stride and (where given) of this shape."""
    s = t.stride()
    if t.dtype is dtype and t.is_cuda and len(s) == dim and s[-1] == 1 and (
            shape is None or t.shape == shape):
        return s
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if len(s) != dim or (s[-1] != 1 and t.shape[-1] > 1 and t.numel()):
        raise ValueError("%s must be %d-D with unit last stride" % (what, dim))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % what)
    return s


def _fp8_operand(torch, codes, scales, what, dim=2):
    s = _rows(codes, torch.float8_e4m3fn, what, None, dim)
    z = _rows(scales, torch.float32, "the scales of " + what, None, dim)
    return s, z


def quantize_fp8(X, form="rows", block_rows=1, out=None, stream=None):
    """E4M3 block quantization of X [rows, K] (float16 or bfloat16).

    form "rows": (codes [rows, K] float8_e4m3fn, scales [ceil(rows /
    block_rows), ceil(K / 128)] float32), blocks along K; "transposed": the
    same of X's transpose (codes_t [K, rows], blocks along the rows of X);
    "both": (codes, scales, codes_t, scales_t) from one read of X.
    block_rows: 1 (activations) or 128 (weights).  out: such a tuple to write
    into; codes rows start on 16-byte boundaries.
    """
    torch = (_FP or _fp())[0]
    code = _float_code(X, "X")
    sx = _rows(X, X.dtype, "X")
    rows, K = X.shape
    if form not in ("rows", "transposed", "both"):
        raise ValueError("form must be rows, transposed or both")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    shapes = [(rows, K)] * (form != "transposed") + [(K, rows)] * (form != "rows")
    if out is None:
        out = ()
        for r, c in shapes:
            room = torch.empty((r, (c + 15) // 16 * 16), dtype=torch.float8_e4m3fn,
                               device=X.device)
            out += (room[:, :c], torch.empty((-(-r // block_rows), -(-c // 128)),
                                             dtype=torch.float32, device=X.device))
    if len(out) != 2 * len(shapes):
        raise ValueError("form %r has %d outputs" % (form, 2 * len(shapes)))
    args = []
    for i, (r, c) in enumerate(shapes):
        sq = _rows(out[2 * i], torch.float8_e4m3fn, "out[%d]" % (2 * i), (r, c))
        ss = _rows(out[2 * i + 1], torch.float32, "out[%d]" % (2 * i + 1),
                   (-(-r // block_rows), -(-c // 128)))
        args += [out[2 * i].data_ptr(), sq[0], out[2 * i + 1].data_ptr(), ss[0]]
    none = [None, 0, None, 0]
    if form == "rows":
        args += none
    elif form == "transposed":
        args = none + args
    _check(lib().dg_quantize_fp8(rows, K, code, X.data_ptr(), sx[0], block_rows, *args,
                                 _stream_of(stream, X, *out)))
    return out


def gemm_fp8(A, scale_a, B, scale_b, D, bias=None, alpha=1.0, beta=0.0, epilogue="none",
             stream=None):
    """D = epilogue(alpha * A.B^T + beta * D) for FP8 operands, written into D.

    A: float8_e4m3fn [M, K] with scale_a float32 [M, ceil(K / 128)]; B: [N, K]
    with scale_b [N, ...] or [ceil(N / 128), ...] (128 x 128 blocks); D: [M, N]
    float16, bfloat16 or float32; bias: [N] of D's type.
    """
    torch, codes = _FP or _fp()
    sa, za = _fp8_operand(torch, A, scale_a, "A")
    sb, zb = _fp8_operand(torch, B, scale_b, "B")
    dt = _float_code(D, "D", (F16, BF16, F32))
    sd = _rows(D, D.dtype, "D")
    M, N = D.shape
    K = A.shape[1]
    nb = scale_b.shape[0]
    kb = (K + 127) // 128
    if A.shape[0] != M or B.shape[0] != N or B.shape[1] != K or scale_a.shape[0] != M or \
            scale_a.shape[1] < kb or scale_b.shape[1] < kb or nb not in (N, (N + 127) // 128):
        raise ValueError("shape mismatch: A %s with %s, B %s with %s, D %s" % tuple(
            tuple(t.shape) for t in (A, scale_a, B, scale_b, D)))
    if bias is not None:
        _rows(bias, D.dtype, "bias", (N,), 1)
    _check(lib().dg_gemm_fp8(
        M, N, K, A.data_ptr(), sa[0], scale_a.data_ptr(), za[0], B.data_ptr(), sb[0],
        scale_b.data_ptr(), zb[0], 1 if nb == N else 128, D.data_ptr(), dt, sd[0],
        None if bias is None else bias.data_ptr(), alpha, beta, _epi_code(epilogue),
        _stream_of(stream, A, scale_a, B, scale_b, D, bias)))
    return D


def gemm_fp8_grouped(A, scale_a, B, scale_b, offsets, D, bias=None, alpha=1.0, beta=0.0,
                     epilogue="none", stream=None):
    """D[i] = epilogue(alpha * A[i].B[e]^T + beta * D[i]) for the rows i of each
    expert e, offsets[e] <= i < offsets[e + 1] (int32 [count + 1] on the device).

    A: float8_e4m3fn [rows, K] with scale_a [rows, ceil(K / 128)]; B: [count, N,
    K] with scale_b [count, ceil(N / 128), ceil(K / 128)]; D: [rows, N]; bias:
    [count, N] of D's type.
    """
    torch, codes = _FP or _fp()
    sa, za = _fp8_operand(torch, A, scale_a, "A")
    sb, zb = _fp8_operand(torch, B, scale_b, "B", 3)
    dt = _float_code(D, "D", (F16, BF16, F32))
    sd = _rows(D, D.dtype, "D")
    rows, N = D.shape
    count, K = B.shape[0], A.shape[1]
    kb = (K + 127) // 128
    if A.shape[0] != rows or B.shape[1] != N or B.shape[2] != K or scale_a.shape[0] != rows or \
            scale_a.shape[1] < kb or scale_b.shape[0] != count or \
            scale_b.shape[1] != (N + 127) // 128 or scale_b.shape[2] < kb:
        raise ValueError("shape mismatch: A %s with %s, B %s with %s, D %s" % tuple(
            tuple(t.shape) for t in (A, scale_a, B, scale_b, D)))
    _rows(offsets, torch.int32, "offsets", (count + 1,), 1)
    stride_bias = 0
    if bias is not None:
        stride_bias = _rows(bias, D.dtype, "bias", (count, N))[0]
    _check(lib().dg_gemm_fp8_grouped(
        count, rows, N, K, A.data_ptr(), sa[0], scale_a.data_ptr(), za[0], B.data_ptr(), sb[1],
        sb[0], scale_b.data_ptr(), zb[1], zb[0], offsets.data_ptr(), D.data_ptr(), dt, sd[0],
        None if bias is None else bias.data_ptr(), stride_bias, alpha, beta, _epi_code(epilogue),
        _stream_of(stream, A, scale_a, B, scale_b, offsets, D, bias)))
    return D


def gemm_fp8_grouped_wgrad(A, scale_a, B, scale_b, offsets, D, alpha=1.0, beta=0.0, stream=None):
    """D[e] = alpha * A[:, e's rows].B[:, e's rows]^T + beta * D[e].

    A: float8_e4m3fn [M, rows] with scale_a [M, ceil(rows / 128)]; B: [N, rows]
    likewise (both the transposed form of quantize_fp8); offsets: int32 [count
    + 1] on the device, multiples of 128; D: [count, M, N].
    """
    torch, codes = _FP or _fp()
    sa, za = _fp8_operand(torch, A, scale_a, "A")
    sb, zb = _fp8_operand(torch, B, scale_b, "B")
    dt = _float_code(D, "D", (F16, BF16, F32))
    sd = _rows(D, D.dtype, "D", None, 3)
    count, M, N = D.shape
    rows = A.shape[1]
    kb = (rows + 127) // 128
    if A.shape[0] != M or B.shape[0] != N or B.shape[1] != rows or scale_a.shape[0] != M or \
            scale_b.shape[0] != N or scale_a.shape[1] < kb or scale_b.shape[1] < kb:
        raise ValueError("shape mismatch: A %s with %s, B %s with %s, D %s" % tuple(
            tuple(t.shape) for t in (A, scale_a, B, scale_b, D)))
    _rows(offsets, torch.int32, "offsets", (count + 1,), 1)
    _check(lib().dg_gemm_fp8_grouped_wgrad(
        count, M, N, rows, A.data_ptr(), sa[0], scale_a.data_ptr(), za[0], B.data_ptr(), sb[0],
        scale_b.data_ptr(), zb[0], offsets.data_ptr(), D.data_ptr(), dt, sd[1], sd[0], alpha, beta,
        _stream_of(stream, A, scale_a, B, scale_b, offsets, D)))
    return D


def moe_rows(tokens, top_k, count, align=1):
    """The rows that moe_sort needs room for (dg_moe_rows)."""
    n = lib().dg_moe_rows(int(tokens), int(top_k), int(count), int(align))
    if n < 0:
        raise ValueError("moe_rows: tokens %s, top_k %s, count %s, align %s" % (
            tokens, top_k, count, align))
    return n


def moe_sort(ids, count, align=1, out=None, stream=None):
    """Sorts the tokens' choices ids [tokens, top_k] (int32; outside [0, count):
    dropped) by expert.  Returns (offsets [count + 1], row_slot [rows], slot_row
    [tokens, top_k]), int32: each expert's rows, the slot t * top_k + j that a
    row holds (-1: none) and the row of each slot (-1: dropped).  Segments
    start at multiples of align.  out: such a tuple to write into.
    """
    torch = (_FP or _fp())[0]
    _rows(ids, torch.int32, "ids")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    tokens, top_k = ids.shape
    if out is None:
        def room(*shape):
            return torch.empty(shape, dtype=torch.int32, device=ids.device)
        out = (room(count + 1), room(moe_rows(tokens, top_k, count, align)), room(tokens, top_k))
    offsets, row_slot, slot_row = out
    for t, what in ((offsets, "offsets"), (row_slot, "row_slot")):
        _rows(t, torch.int32, what, None, 1)
    _rows(slot_row, torch.int32, "slot_row", ids.shape)
    if offsets.shape[0] != count + 1 or not slot_row.is_contiguous():
        raise ValueError("offsets must be [count + 1], slot_row contiguous like ids")
    _check(lib().dg_moe_sort(tokens, top_k, count, ids.data_ptr(), align, row_slot.shape[0],
                             offsets.data_ptr(), row_slot.data_ptr(), slot_row.data_ptr(),
                             _stream_of(stream, ids, offsets, row_slot, slot_row)))
    return out


def moe_dispatch(X, row_slot, top_k, D, stream=None):
    """D[r] = X[row_slot[r] // top_k], zeros where row_slot[r] is -1.  X: [tokens,
    width] float16 or bfloat16, D: [rows, width] of its type.  The gradient is
    moe_combine without weights."""
    torch = (_FP or _fp())[0]
    code = _float_code(X, "X")
    sx = _rows(X, X.dtype, "X")
    rows = row_slot.shape[0]
    tokens, width = X.shape
    _rows(row_slot, torch.int32, "row_slot", None, 1)
    sd = _rows(D, X.dtype, "D", (rows, width))
    _check(lib().dg_moe_dispatch(tokens, top_k, width, code, X.data_ptr(), sx[0], rows,
                                 row_slot.data_ptr(), D.data_ptr(), sd[0],
                                 _stream_of(stream, X, row_slot, D)))
    return D


_SCRATCH_FROM = 1 << 23  # rows * width below which dg_moe_dispatch_fp8_scratch asks for nothing


def _scratch(torch, nbytes, device, stream):
    """nbytes of device memory for one call on `stream`: from torch's allocator
    for that stream (while torch.cuda.graph captures it, from the graph's pool),
    so its next user comes after the call and a graph keeps what it captured."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_handle(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else \
            torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def moe_dispatch_fp8(X, row_slot, top_k, codes, scales, stream=None):
    """moe_dispatch and quantize_fp8 in one: codes float8_e4m3fn [rows, width],
    scales float32 [rows, ceil(width / 128)].  Large calls quantize the tokens
    once, in scratch from torch's allocator (dg_moe_dispatch_fp8_ex)."""
    torch = (_FP or _fp())[0]
    code = _float_code(X, "X")
    sx = _rows(X, X.dtype, "X")
    rows = row_slot.shape[0]
    tokens, width = X.shape
    _rows(row_slot, torch.int32, "row_slot", None, 1)
    sq = _rows(codes, torch.float8_e4m3fn, "codes", (rows, width))
    ss = _rows(scales, torch.float32, "scales", (rows, (width + 127) // 128))
    args = (tokens, top_k, width, code, X.data_ptr(), sx[0], rows, row_slot.data_ptr(),
            codes.data_ptr(), sq[0], scales.data_ptr(), ss[0])
    handle = _stream_of(stream, X, row_slot, codes, scales)
    if rows * width >= _SCRATCH_FROM:
        nbytes = lib().dg_moe_dispatch_fp8_scratch(tokens, top_k, width, rows)
        if nbytes > 0:
            scratch = _scratch(torch, nbytes, X.device, stream)
            _check(lib().dg_moe_dispatch_fp8_ex(*args, scratch.data_ptr(), nbytes, handle))
            return codes, scales
    _check(lib().dg_moe_dispatch_fp8(*args, handle))
    return codes, scales


def moe_combine(Y, slot_row, D, weights=None, stream=None):
    """D[t] = sum over j of weights[t, j] * Y[slot_row[t, j]] (dropped slots add
    nothing).  Y: [rows, width] float16 or bfloat16, D: [tokens, width] of its
    type, weights: float32 [tokens, top_k] or None for ones."""
    torch = (_FP or _fp())[0]
    code = _float_code(Y, "Y")
    sy = _rows(Y, Y.dtype, "Y")
    _rows(slot_row, torch.int32, "slot_row")
    tokens, top_k = slot_row.shape
    width = Y.shape[1]
    sd = _rows(D, Y.dtype, "D", (tokens, width))
    if weights is not None:
        _rows(weights, torch.float32, "weights", slot_row.shape)
    if not slot_row.is_contiguous() or not (weights is None or weights.is_contiguous()):
        raise ValueError("slot_row and weights must be contiguous")
    _check(lib().dg_moe_combine(tokens, top_k, width, code, Y.data_ptr(), sy[0], Y.shape[0],
                                slot_row.data_ptr(),
                                None if weights is None else weights.data_ptr(), D.data_ptr(),
                                sd[0], _stream_of(stream, Y, slot_row, D, weights)))
    return D


def moe_combine_backward(dD, Y, slot_row, row_slot, weights, dY, dweights=None, stream=None):
    """The gradient of moe_combine: dY[r] = weights[s] * dD[s // top_k] for the
    slot s of row r (zeros without one), dweights[s] = dD[s // top_k] . Y[r].
    weights may be None for ones; without dweights Y may be None.  Returns
    (dY, dweights)."""
    torch = (_FP or _fp())[0]
    code = _float_code(dD, "dD")
    s_dd = _rows(dD, dD.dtype, "dD")
    _rows(slot_row, torch.int32, "slot_row")
    _rows(row_slot, torch.int32, "row_slot", None, 1)
    tokens, top_k = slot_row.shape
    width, rows = dD.shape[1], row_slot.shape[0]
    if dD.shape[0] != tokens:
        raise ValueError("dD must be [tokens, width]")
    s_dy = _rows(dY, dD.dtype, "dY", (rows, width))
    s_y = (0,)
    if dweights is not None:
        if Y is None:
            raise ValueError("dweights needs Y")
        s_y = _rows(Y, dD.dtype, "Y", (rows, width))
    for t, what in ((weights, "weights"), (dweights, "dweights")):
        if t is not None:
            _rows(t, torch.float32, what, slot_row.shape)
            if not t.is_contiguous():
                raise ValueError("%s must be contiguous" % what)
    if not slot_row.is_contiguous():
        raise ValueError("slot_row must be contiguous")
    _check(lib().dg_moe_combine_backward(
        tokens, top_k, width, code, dD.data_ptr(), s_dd[0],
        None if dweights is None else Y.data_ptr(), s_y[0], rows, row_slot.data_ptr(),
        slot_row.data_ptr(), None if weights is None else weights.data_ptr(), dY.data_ptr(),
        s_dy[0], None if dweights is None else dweights.data_ptr(),
        _stream_of(stream, dD, None if dweights is None else Y, slot_row, row_slot, weights, dY,
                   dweights)))
    return dY, dweights


def query_hw(device=0):
    h = HwDesc()
    _check(lib().dg_query_hw(int(device), ctypes.byref(h)))
    return h


def plan_tiles(M, N, K, dtype_a="f16", dtype_b="f16", epilogue="none", hw=None,
               target_occupancy=0.0, max_out=64):
    """The planner's ranked candidates (list of dicts)."""
    if isinstance(hw, dict):
        h = HwDesc(**hw)
        hw_p = ctypes.byref(h)
    elif hw is not None:
        hw_p = ctypes.byref(hw)
    else:
        hw_p = None
    out = (TilePlan * max_out)()
    n = ctypes.c_int(0)
    _check(lib().dg_plan_tiles(int(M), int(N), int(K), _dtype_code(dtype_a), _dtype_code(dtype_b),
                               _epi_code(epilogue), hw_p, float(target_occupancy), out,
                               int(max_out), ctypes.byref(n)))
    return [out[i].as_dict() for i in range(n.value)]


def check_status(stream=None):
    _check(lib().dg_check_status(_stream_handle(stream)))


def set_wait_timeout_ns(ns):
    _check(lib().dg_set_wait_timeout_ns(int(ns)))


def selftest_wait_timeout(stream=None):
    _check(lib().dg_selftest_wait_timeout(_stream_handle(stream)))


def launch_count():
    return int(lib().dg_launch_count())


def shutdown():
    _check(lib().dg_shutdown())
