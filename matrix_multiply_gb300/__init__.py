"""Python binding of tcgemm, the GB300 (sm_103a) GEMM library.

C = alpha * op(A) @ op(B) + beta * C, row-major, NN/TN/NT/TT, leading
dimensions, f16/bf16 (tcgen05 tensor cores) or f32 (exact FFMA) inputs with
fp32 accumulation -- the operation of the tensorcore gemm.md page, section
"Surface".

This module only marshals arguments: every step of the computation runs in
the CUDA kernels of ``_lib/libtcgemm.so``.  The functions keep the C names
(``tc_gemm``, ``tc_gemm_async``, ``tc_gemm_batched``, ...) and take either raw
device addresses or torch tensors (PyTorch provides device memory and
streams only).  Where a tensor is given, its capacity is checked in
elements before the call (the tessl architecture.md "nn Boundary" rule: a
view of too few elements is refused, nothing is launched).  ``GroupedGemm``
and ``PreparedGemm`` run those checks once for a group or a single product
that is issued many times; each ``enqueue()`` is then one C call.

``Q4Weight`` holds a 4-bit weight with group scales: ``tc_quantize_q4`` fills
one, ``tc_gemm_q4_weight`` (or ``PreparedGemm``) multiplies by it, and
``tc_moe_q4`` (or ``PreparedMoe``) runs a mixture-of-experts layer over two.

``PreparedXent`` (``tc_linear_xent``) and ``PreparedRoute`` (``tc_moe_route``)
are what such a model trains on: the softmax cross entropy against a vocabulary,
and the choice of experts with its balance loss, each with its backward call.

There is no fallback: if the library is missing, importing this package
raises.  Build it with ``python -c "import __graft_entry__ as g; g.build()"``.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libtcgemm.so")

# ------------------------------------------------------------------ enums

TC_F16, TC_BF16, TC_F32, TC_I8, TC_I32, TC_I4, TC_I64 = 1, 2, 3, 4, 5, 6, 7
STATUS = {
    0: "TC_OK", 1: "TC_ERR_NULL", 2: "TC_ERR_DIM", 3: "TC_ERR_LD", 4: "TC_ERR_DTYPE",
    5: "TC_ERR_SCALAR", 6: "TC_ERR_OVERLAP", 7: "TC_ERR_OVERFLOW", 8: "TC_ERR_ALIGN_UNSUPPORTED",
    9: "TC_ERR_CUDA", 10: "TC_ERR_DEVICE_TIMEOUT", 11: "TC_ERR_STRIDE", 12: "TC_ERR_VARIANT",
    13: "TC_ERR_SCRATCH", 14: "TC_ERR_EPILOGUE", 15: "TC_ERR_LAYOUT",
}
for _code, _name in STATUS.items():
    globals()[_name] = _code


class tc_gemm_desc(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
        ("a_dtype", ctypes.c_int), ("b_dtype", ctypes.c_int), ("c_dtype", ctypes.c_int),
        ("accum_dtype", ctypes.c_int),
        ("transpose_a", ctypes.c_bool), ("transpose_b", ctypes.c_bool),
        ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
        ("lda", ctypes.c_int32), ("ldb", ctypes.c_int32), ("ldc", ctypes.c_int32),
    ]


TC_ACT_NONE, TC_ACT_GELU_TANH = 0, 1
_ACTIVATIONS = {None: TC_ACT_NONE, "none": TC_ACT_NONE, "gelu_tanh": TC_ACT_GELU_TANH}


class tc_epilogue(ctypes.Structure):
    """Fused epilogue: bias (device pointer to N values of C's dtype, or
    None) and activation (TC_ACT_*)."""
    _fields_ = [("bias", ctypes.c_void_p), ("activation", ctypes.c_int)]


class tc_gemm_batched_desc(ctypes.Structure):
    _fields_ = [("base", tc_gemm_desc), ("batch", ctypes.c_int32),
                ("stride_a", ctypes.c_int64), ("stride_b", ctypes.c_int64),
                ("stride_c", ctypes.c_int64)]


class tc_q4_weight(ctypes.Structure):
    """A 4-bit weight with group scales (see include/tcgemm.h)."""
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("group", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int), ("ldw", ctypes.c_int32), ("ld_scale", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p)]


TC_MOE_MAX_TOKENS, TC_MOE_MAX_EXPERTS, TC_MOE_MAX_TOPK = 32, 512, 16


class tc_moe_desc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("x_dtype", ctypes.c_int), ("router_dtype", ctypes.c_int), ("y_dtype", ctypes.c_int),
                ("renormalize", ctypes.c_bool),
                ("ldx", ctypes.c_int32), ("ld_router", ctypes.c_int32), ("ldy", ctypes.c_int32)]


TC_REDUCE_NONE, TC_REDUCE_SUM, TC_REDUCE_MEAN = 0, 1, 2
_REDUCTIONS = {"none": TC_REDUCE_NONE, "sum": TC_REDUCE_SUM, "mean": TC_REDUCE_MEAN}


class tc_xent_desc(ctypes.Structure):
    """A softmax cross entropy against a vocabulary (see include/tcgemm.h)."""
    _fields_ = [("tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int), ("target_dtype", ctypes.c_int),
                ("reduction", ctypes.c_int), ("scale", ctypes.c_float), ("z_weight", ctypes.c_float),
                ("ldx", ctypes.c_int32), ("ldw", ctypes.c_int32), ("lddx", ctypes.c_int32), ("lddw", ctypes.c_int32)]


class tc_route_desc(ctypes.Structure):
    """A routing of tokens to experts (see include/tcgemm.h)."""
    _fields_ = [("tokens", ctypes.c_int32), ("experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("logits_dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int), ("renormalize", ctypes.c_bool),
                ("ld_logits", ctypes.c_int32), ("ld_dlogits", ctypes.c_int32)]


class TcError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({_lib.tc_status_string(status).decode()})")


# ------------------------------------------------------------------ loading

def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"tcgemm CUDA library not built ({LIB_PATH} missing); run "
            "python -c \"import __graft_entry__ as g; g.build()\"")
    lib = ctypes.CDLL(LIB_PATH)
    vp, st = ctypes.c_void_p, ctypes.c_int
    D = ctypes.POINTER(tc_gemm_desc)
    BD = ctypes.POINTER(tc_gemm_batched_desc)
    E = ctypes.POINTER(tc_epilogue)
    Q = ctypes.POINTER(tc_q4_weight)
    MD = ctypes.POINTER(tc_moe_desc)
    XD = ctypes.POINTER(tc_xent_desc)
    RD = ctypes.POINTER(tc_route_desc)
    i32 = ctypes.c_int32
    sig = {
        "tc_ctx_create": (st, [ctypes.POINTER(vp), ctypes.c_int]),
        "tc_ctx_destroy": (None, [vp]),
        "tc_stream_create": (st, [vp, ctypes.POINTER(vp)]),
        "tc_stream_wrap": (st, [vp, vp, ctypes.POINTER(vp)]),
        "tc_stream_sync": (st, [vp]),
        "tc_stream_handle": (vp, [vp]),
        "tc_stream_destroy": (None, [vp]),
        "tc_gemm": (st, [vp, D, vp, vp, vp]),
        "tc_gemm_async": (st, [vp, D, vp, vp, vp, vp]),
        "tc_gemm_batched": (st, [vp, BD, vp, vp, vp]),
        "tc_gemm_batched_async": (st, [vp, BD, vp, vp, vp, vp]),
        "tc_gemm_grouped_async": (st, [vp, ctypes.c_int, D, ctypes.POINTER(vp), ctypes.POINTER(vp),
                                       ctypes.POINTER(vp), vp]),
        "tc_gemm_epilogue": (st, [vp, D, E, vp, vp, vp]),
        "tc_gemm_epilogue_async": (st, [vp, D, E, vp, vp, vp, vp]),
        "tc_gemm_epilogue_validate": (st, [D, E, vp, vp, vp]),
        "tc_gemm_f32_relaxed": (st, [vp, D, E, vp, vp, vp]),
        "tc_gemm_i8_dequant": (st, [vp, D, vp, vp, vp, vp]),
        "tc_gemm_i8_dequant_async": (st, [vp, D, vp, vp, vp, vp, vp]),
        "tc_gemm_q8_weight": (st, [vp, D, vp, vp, vp, vp]),
        "tc_gemm_q8_weight_async": (st, [vp, D, vp, vp, vp, vp, vp]),
        "tc_gemm_q8_weight_validate": (st, [D, vp, vp, vp, vp]),
        "tc_gemm_f32_relaxed_async": (st, [vp, D, E, vp, vp, vp, vp]),
        "tc_quantize_q4": (st, [vp, ctypes.c_int, i32, vp, Q]),
        "tc_quantize_q4_async": (st, [vp, ctypes.c_int, i32, vp, Q, vp]),
        "tc_dequantize_q4": (st, [vp, Q, ctypes.c_int, i32, vp]),
        "tc_dequantize_q4_async": (st, [vp, Q, ctypes.c_int, i32, vp, vp]),
        "tc_q4_validate": (st, [Q, ctypes.c_int, i32, vp]),
        "tc_gemm_q4_weight": (st, [vp, D, Q, vp, vp]),
        "tc_gemm_q4_weight_async": (st, [vp, D, Q, vp, vp, vp]),
        "tc_gemm_q4_weight_validate": (st, [D, Q, vp, vp]),
        "tc_moe_q4": (st, [vp, MD, vp, vp, Q, Q, vp, vp, vp]),
        "tc_moe_q4_async": (st, [vp, MD, vp, vp, Q, Q, vp, vp, vp, vp]),
        "tc_moe_q4_validate": (st, [MD, vp, vp, Q, Q, vp, vp, vp]),
        "tc_linear_xent": (st, [vp, XD, vp, vp, vp, vp, vp]),
        "tc_linear_xent_async": (st, [vp, XD, vp, vp, vp, vp, vp, vp]),
        "tc_linear_xent_backward": (st, [vp, XD, vp, vp, vp, vp, vp, vp, vp]),
        "tc_linear_xent_backward_async": (st, [vp, XD, vp, vp, vp, vp, vp, vp, vp, vp]),
        "tc_linear_xent_validate": (st, [XD, vp, vp, vp, vp, vp]),
        "tc_linear_xent_backward_validate": (st, [XD, vp, vp, vp, vp, vp, vp, vp]),
        "tc_moe_route": (st, [vp, RD, vp, vp, vp, vp, vp, vp]),
        "tc_moe_route_async": (st, [vp, RD, vp, vp, vp, vp, vp, vp, vp]),
        "tc_moe_route_backward": (st, [vp, RD, vp, vp, vp, vp, vp, vp, vp]),
        "tc_moe_route_backward_async": (st, [vp, RD, vp, vp, vp, vp, vp, vp, vp, vp]),
        "tc_moe_route_validate": (st, [RD, vp, vp, vp, vp, vp, vp]),
        "tc_moe_route_backward_validate": (st, [RD, vp, vp, vp, vp, vp, vp, vp]),
        "tc_gemm_host": (st, [vp, D, vp, vp, vp]),
        "tc_gemm_splitk_noalloc": (st, [D, vp, vp, vp, ctypes.c_int, vp]),
        "tc_gemm_validate": (st, [D, vp, vp, vp]),
        "tc_gemm_batched_validate": (st, [BD, vp, vp, vp]),
        "tc_gemm_plan": (st, [D, vp, vp, vp, ctypes.c_int, ctypes.c_char_p, ctypes.c_size_t]),
        "tc_last_kernel": (ctypes.c_char_p, [vp]),
        "tc_launch_count": (ctypes.c_uint64, [vp]),
        "tc_status_string": (ctypes.c_char_p, [st]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()
EXPORTED = (
    "tc_ctx_create", "tc_ctx_destroy", "tc_stream_create", "tc_stream_wrap", "tc_stream_sync",
    "tc_stream_handle", "tc_stream_destroy", "tc_gemm", "tc_gemm_async", "tc_gemm_batched",
    "tc_gemm_batched_async", "tc_gemm_grouped_async", "tc_gemm_host", "tc_gemm_splitk_noalloc",
    "tc_gemm_validate",
    "tc_gemm_batched_validate", "tc_gemm_plan", "tc_last_kernel", "tc_launch_count",
    "tc_status_string", "tc_gemm_epilogue", "tc_gemm_epilogue_async", "tc_gemm_epilogue_validate",
    "tc_gemm_f32_relaxed", "tc_gemm_f32_relaxed_async", "tc_gemm_i8_dequant", "tc_gemm_i8_dequant_async",
    "tc_gemm_q8_weight", "tc_gemm_q8_weight_async", "tc_gemm_q8_weight_validate",
    "tc_quantize_q4", "tc_quantize_q4_async", "tc_dequantize_q4", "tc_dequantize_q4_async", "tc_q4_validate",
    "tc_gemm_q4_weight", "tc_gemm_q4_weight_async", "tc_gemm_q4_weight_validate",
    "tc_moe_q4", "tc_moe_q4_async", "tc_moe_q4_validate",
    "tc_linear_xent", "tc_linear_xent_async", "tc_linear_xent_backward", "tc_linear_xent_backward_async",
    "tc_linear_xent_validate", "tc_linear_xent_backward_validate",
    "tc_moe_route", "tc_moe_route_async", "tc_moe_route_backward", "tc_moe_route_backward_async",
    "tc_moe_route_validate", "tc_moe_route_backward_validate",
)


def library():
    """The loaded ctypes library (for tests that call the ABI directly)."""
    return _lib


def _check(status: int, what: str):
    if status != 0:
        raise TcError(status, what)


# ------------------------------------------------------------------ helpers

_DT_NAMES = {"f16": TC_F16, "bf16": TC_BF16, "f32": TC_F32, "i8": TC_I8, "i4": TC_I4, "i32": TC_I32, "i64": TC_I64}


def _torch_dtype_code(t) -> int:
    import torch
    return {torch.float16: TC_F16, torch.bfloat16: TC_BF16, torch.float32: TC_F32}[t.dtype]


def _addr(x) -> int:
    """A device address from a torch tensor or an int."""
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return x.data_ptr()


def make_desc(M, N, K, a_dtype, c_dtype=None, *, transpose_a=False, transpose_b=False,
              alpha=1.0, beta=0.0, lda=0, ldb=0, ldc=0, b_dtype=None) -> tc_gemm_desc:
    """A descriptor; B has A's type unless ``b_dtype`` is given (the
    int8-weight and 4-bit-weight products: a_dtype "f16"/"bf16", b_dtype
    "i8" or "i4")."""
    a = _DT_NAMES.get(a_dtype, a_dtype)
    b = _DT_NAMES.get(b_dtype, b_dtype) if b_dtype is not None else a
    c = _DT_NAMES.get(c_dtype, c_dtype) if c_dtype is not None else a
    accum = TC_I32 if a == TC_I8 else TC_F32       # int8 x int8 accumulates in int32
    return tc_gemm_desc(M, N, K, a, b, c, accum, bool(transpose_a), bool(transpose_b),
                        float(alpha), float(beta), lda, ldb, ldc)


def _require(t, n_elems: int, what: str):
    """Capacity check in elements (tessl architecture.md, 'nn Boundary')."""
    if t is None or isinstance(t, int):
        return
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    avail = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
    if n_elems > avail:
        raise ValueError(f"{what} holds {avail} elements, the descriptor needs {n_elems}")


def _extent(rows, cols, ld):
    return (rows - 1) * ld + cols


def _check_capacity(d: tc_gemm_desc, A, B, C, batch=1, sa=0, sb=0, sc=0):
    lda = d.lda or (d.M if d.transpose_a else d.K)
    ldb = d.ldb or (d.K if d.transpose_b else d.N)
    ldc = d.ldc or d.N
    ar, ac = (d.K, d.M) if d.transpose_a else (d.M, d.K)
    br, bc = (d.N, d.K) if d.transpose_b else (d.K, d.N)
    if min(d.M, d.N, d.K, batch) < 1 or lda < ac or ldb < bc or ldc < d.N:
        return   # the library reports the precise error
    _require(A, (batch - 1) * sa + _extent(ar, ac, lda), "A")
    _require(B, (batch - 1) * sb + _extent(br, bc, ldb), "B")
    _require(C, (batch - 1) * sc + _extent(d.M, d.N, ldc), "C")


# ------------------------------------------------------------------ objects

class Context:
    """A tc_ctx on one CUDA device."""

    def __init__(self, device: int = 0):
        p = ctypes.c_void_p()
        _check(_lib.tc_ctx_create(ctypes.byref(p), device), "tc_ctx_create")
        self.ptr = p.value
        self.device = device

    def close(self):
        if self.ptr:
            _lib.tc_ctx_destroy(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def last_kernel(self) -> str:
        return _lib.tc_last_kernel(self.ptr).decode()

    @property
    def launch_count(self) -> int:
        return int(_lib.tc_launch_count(self.ptr))


class Stream:
    """A tc_stream: owned (created by the library) or wrapping a torch stream."""

    def __init__(self, ctx: Context, torch_stream=None):
        p = ctypes.c_void_p()
        if torch_stream is None:
            _check(_lib.tc_stream_create(ctx.ptr, ctypes.byref(p)), "tc_stream_create")
        else:
            _check(_lib.tc_stream_wrap(ctx.ptr, ctypes.c_void_p(torch_stream.cuda_stream),
                                       ctypes.byref(p)), "tc_stream_wrap")
        self.ptr = p.value
        self.ctx = ctx

    @property
    def handle(self) -> int:
        return _lib.tc_stream_handle(self.ptr) or 0

    def sync(self):
        _check(_lib.tc_stream_sync(self.ptr), "tc_stream_sync")

    def close(self):
        if self.ptr:
            _lib.tc_stream_destroy(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _check_pitch(what: str, t, rows: int, row_len: int, per: int = 1):
    """Rows that lie apart, at a pitch (``per`` units an element of t) that the
    C structures hold.  Rows that share memory, as expand gives them, have none:
    a stride of 0 would mean the default pitch there, past the end of t."""
    if rows > 1 and not row_len <= t.stride(0) <= (2 ** 31 - 1) // per:
        raise ValueError(f"{what} has a row stride of {t.stride(0)}, its rows are {row_len} long")


class Q4Weight:
    """A 4-bit weight W[N, K] with group scales in caller-owned CUDA tensors:
    codes uint8 [N, >= K/2], scales f16/bf16 [ceil(K/group), >= N], zeros
    uint8 laid out as the scales or None (include/tcgemm.h states the
    format).  Strides and capacities are checked here; ``desc`` is the C
    structure.  The tensors stay referenced as long as this object.
    ``Q4Weight.empty`` allocates the tensors for tc_quantize_q4 to fill."""

    def __init__(self, N: int, K: int, group: int, codes, scales, zeros=None):
        import torch
        groups = -(-K // group) if group > 0 else 0
        for name, t, rows, need in (("codes", codes, N, -(-K // 32) * 16), ("scales", scales, groups, N),
                                    ("zeros", zeros, groups, N)):
            if t is None and name == "zeros":
                continue
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.dim() != 2 or t.stride(1) != 1:
                raise ValueError(f"{name} must be 2-D with unit column stride")
            if t.shape[0] < rows or t.shape[1] < need:
                raise ValueError(f"{name} is {tuple(t.shape)}, the weight needs at least ({rows}, {need})")
            _check_pitch(name, t, rows, need, 2 if name == "codes" else 1)
        for name, t in (("codes", codes), ("zeros", zeros)):
            if t is not None and t.dtype != torch.uint8:
                raise ValueError(f"{name} must be uint8")
        if scales.dtype not in (torch.float16, torch.bfloat16):
            raise ValueError("scales must be float16 or bfloat16")
        if zeros is not None and groups > 1 and zeros.stride(0) != scales.stride(0):
            raise ValueError("zeros must be laid out as the scales")
        self.N, self.K, self.group = N, K, group
        self.codes, self.scales, self.zeros = codes, scales, zeros
        # (a single row's stride is torch's choice: 0 lets the library take the minimum)
        self.desc = tc_q4_weight(N, K, group, _torch_dtype_code(scales), codes.stride(0) * 2 if N > 1 else 0,
                                 scales.stride(0) if groups > 1 else 0, codes.data_ptr(), scales.data_ptr(),
                                 zeros.data_ptr() if zeros is not None else None)
        self.ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, N: int, K: int, group: int = 128, *, scale_dtype=None, zeros: bool = False, device="cuda"):
        """Uninitialised tensors of an [N, K] weight, for tc_quantize_q4."""
        import torch
        if N < 1 or K < 1 or group < 1:
            raise ValueError("N, K and group must be at least 1")
        groups, ns = -(-K // group), -(-N // 16) * 16
        return cls(N, K, group, torch.empty(N, -(-K // 32) * 16, dtype=torch.uint8, device=device),
                   torch.empty(groups, ns, dtype=scale_dtype or torch.float16, device=device),
                   torch.empty(groups, ns, dtype=torch.uint8, device=device) if zeros else None)


# ------------------------------------------------------------------ C names

def tc_gemm(ctx: Context, d: tc_gemm_desc, A, B, C):
    _check_capacity(d, A, B, C)
    _check(_lib.tc_gemm(ctx.ptr, ctypes.byref(d), _addr(A), _addr(B), _addr(C)), "tc_gemm")


def tc_gemm_async(ctx: Context, d: tc_gemm_desc, A, B, C, stream: Stream):
    _check_capacity(d, A, B, C)
    _check(_lib.tc_gemm_async(ctx.ptr, ctypes.byref(d), _addr(A), _addr(B), _addr(C), stream.ptr),
           "tc_gemm_async")


def tc_gemm_batched(ctx: Context, bd: tc_gemm_batched_desc, A, B, C):
    _check_capacity(bd.base, A, B, C, bd.batch, bd.stride_a, bd.stride_b, bd.stride_c)
    _check(_lib.tc_gemm_batched(ctx.ptr, ctypes.byref(bd), _addr(A), _addr(B), _addr(C)),
           "tc_gemm_batched")


def tc_gemm_batched_async(ctx: Context, bd: tc_gemm_batched_desc, A, B, C, stream: Stream):
    _check_capacity(bd.base, A, B, C, bd.batch, bd.stride_a, bd.stride_b, bd.stride_c)
    _check(_lib.tc_gemm_batched_async(ctx.ptr, ctypes.byref(bd), _addr(A), _addr(B), _addr(C),
                                      stream.ptr), "tc_gemm_batched_async")


class GroupedGemm:
    """The arguments of tc_gemm_grouped_async marshalled once: descriptors
    and operand addresses in C arrays, capacities checked here.  enqueue()
    then costs one C call, so that a group issued many times with the same
    operands does not pay the per-problem Python work each time.  The
    tensors stay referenced (alive) as long as this object."""

    def __init__(self, descs, As, Bs, Cs):
        n = len(descs)
        if not (len(As) == len(Bs) == len(Cs) == n):
            raise ValueError("descs, As, Bs and Cs must have the same length")
        for d, a, b, c in zip(descs, As, Bs, Cs):
            _check_capacity(d, a, b, c)
        self.n = n
        self._keep = (list(As), list(Bs), list(Cs))
        self._descs = (tc_gemm_desc * n)(*descs)
        self._A = (ctypes.c_void_p * n)(*[_addr(x) for x in As])
        self._B = (ctypes.c_void_p * n)(*[_addr(x) for x in Bs])
        self._C = (ctypes.c_void_p * n)(*[_addr(x) for x in Cs])

    def enqueue(self, ctx: Context, stream: Stream):
        _check(_lib.tc_gemm_grouped_async(ctx.ptr, self.n, self._descs, self._A, self._B, self._C, stream.ptr),
               "tc_gemm_grouped_async")


def tc_gemm_grouped_async(ctx: Context, descs, As, Bs, Cs, stream: Stream):
    GroupedGemm(descs, As, Bs, Cs).enqueue(ctx, stream)


class PreparedGemm:
    """One asynchronous product with its arguments checked and marshalled
    once: tc_gemm_async; with ``bias``/``activation`` tc_gemm_epilogue_async;
    with ``relaxed`` tc_gemm_f32_relaxed_async; with ``col_scale``
    tc_gemm_i8_dequant_async; with ``q8_scale`` tc_gemm_q8_weight_async;
    with a Q4Weight for B tc_gemm_q4_weight_async.
    enqueue() is then one C call -- the library still plans the product and
    launches its kernels every time -- for a caller that issues the same
    product on the same buffers many times (the Python checks otherwise
    cost about as much host time per call as the library itself).  The
    tensors stay referenced as long as this object."""

    def __init__(self, ctx: Context, d: tc_gemm_desc, A, B, C, stream: Stream, *, bias=None, activation=None,
                 relaxed: bool = False, col_scale=None, q8_scale=None):
        vp = ctypes.c_void_p
        self._e = None
        if isinstance(B, Q4Weight):
            if relaxed or any(x is not None for x in (bias, activation, col_scale, q8_scale)):
                raise ValueError("a 4-bit weight takes no epilogue, scales or relaxed mode")
            _check_q4_capacity(d, A, C)
            self._fn, self._name = _lib.tc_gemm_q4_weight_async, "tc_gemm_q4_weight_async"
            self._args = (vp(ctx.ptr), ctypes.byref(d), B.ref, vp(_addr(A)), vp(_addr(C)), vp(stream.ptr))
            self._keep = (ctx, d, A, B, C, stream)
            return
        _check_capacity(d, A, B, C)
        head = (vp(ctx.ptr), ctypes.byref(d))
        abc = (vp(_addr(A)), vp(_addr(B)), vp(_addr(C)), vp(stream.ptr))
        if q8_scale is not None:
            _require(q8_scale, d.N, "scale")
            self._fn, self._name = _lib.tc_gemm_q8_weight_async, "tc_gemm_q8_weight_async"
            self._args = head + (vp(_addr(q8_scale)),) + abc
        elif col_scale is not None:
            _require(col_scale, d.N, "col_scale")
            self._fn, self._name = _lib.tc_gemm_i8_dequant_async, "tc_gemm_i8_dequant_async"
            self._args = head + (vp(_addr(col_scale)),) + abc
        elif relaxed or bias is not None or activation is not None:
            _check_bias(d, bias)
            self._e = make_epilogue(bias, activation)
            self._name = "tc_gemm_f32_relaxed_async" if relaxed else "tc_gemm_epilogue_async"
            self._fn = getattr(_lib, self._name)
            self._args = head + (ctypes.byref(self._e),) + abc
        else:
            self._fn, self._name = _lib.tc_gemm_async, "tc_gemm_async"
            self._args = head + abc
        self._keep = (ctx, d, A, B, C, stream, bias, col_scale, q8_scale)

    def enqueue(self):
        _check(self._fn(*self._args), self._name)


def make_epilogue(bias=None, activation=None) -> tc_epilogue:
    """bias: a CUDA tensor of N values in C's dtype (or an address, or
    None); activation: None/"none" or "gelu_tanh" (or a TC_ACT_* code)."""
    act = _ACTIVATIONS.get(activation, activation)
    return tc_epilogue(_addr(bias) or None, int(act))


def _check_bias(d: tc_gemm_desc, bias):
    if bias is None or isinstance(bias, int):
        return
    _require(bias, d.N, "bias")
    if d.c_dtype in (TC_F16, TC_BF16, TC_F32) and _torch_dtype_code(bias) != d.c_dtype:
        raise ValueError("bias must have C's dtype")


def tc_gemm_epilogue(ctx: Context, d: tc_gemm_desc, A, B, C, bias=None, activation=None):
    """C = activation(alpha*op(A)@op(B) + beta*C + bias), synchronously."""
    _check_capacity(d, A, B, C)
    _check_bias(d, bias)
    e = make_epilogue(bias, activation)
    _check(_lib.tc_gemm_epilogue(ctx.ptr, ctypes.byref(d), ctypes.byref(e), _addr(A), _addr(B), _addr(C)),
           "tc_gemm_epilogue")


def tc_gemm_epilogue_async(ctx: Context, d: tc_gemm_desc, A, B, C, stream: Stream, bias=None, activation=None):
    _check_capacity(d, A, B, C)
    _check_bias(d, bias)
    e = make_epilogue(bias, activation)
    _check(_lib.tc_gemm_epilogue_async(ctx.ptr, ctypes.byref(d), ctypes.byref(e), _addr(A), _addr(B), _addr(C),
                                       stream.ptr), "tc_gemm_epilogue_async")


def tc_gemm_epilogue_validate(d: tc_gemm_desc, bias=None, activation=None, A=1 << 20, B=2 << 40,
                              C=3 << 40) -> int:
    """Host-only validation status of a fused-epilogue call."""
    e = make_epilogue(bias, activation)
    return int(_lib.tc_gemm_epilogue_validate(ctypes.byref(d), ctypes.byref(e), _addr(A), _addr(B), _addr(C)))


def tc_gemm_f32_relaxed(ctx: Context, d: tc_gemm_desc, A, B, C, bias=None, activation=None):
    """fp32 GEMM on the bf16 tensor cores through a two-part bf16 split of
    each operand (see include/tcgemm.h), synchronously; optional fused
    epilogue."""
    _check_capacity(d, A, B, C)
    _check_bias(d, bias)
    e = make_epilogue(bias, activation)
    _check(_lib.tc_gemm_f32_relaxed(ctx.ptr, ctypes.byref(d), ctypes.byref(e), _addr(A), _addr(B), _addr(C)),
           "tc_gemm_f32_relaxed")


def tc_gemm_f32_relaxed_async(ctx: Context, d: tc_gemm_desc, A, B, C, stream: Stream, bias=None, activation=None):
    _check_capacity(d, A, B, C)
    _check_bias(d, bias)
    e = make_epilogue(bias, activation)
    _check(_lib.tc_gemm_f32_relaxed_async(ctx.ptr, ctypes.byref(d), ctypes.byref(e), _addr(A), _addr(B), _addr(C),
                                          stream.ptr), "tc_gemm_f32_relaxed_async")


def tc_gemm_i8_dequant(ctx: Context, d: tc_gemm_desc, A, B, C, col_scale):
    """int8 x int8 accumulated exactly, then C = alpha * acc * col_scale[n] +
    beta * C (C fp32; col_scale a CUDA tensor of N floats), synchronously."""
    _check_capacity(d, A, B, C)
    _require(col_scale, d.N, "col_scale")
    _check(_lib.tc_gemm_i8_dequant(ctx.ptr, ctypes.byref(d), _addr(col_scale), _addr(A), _addr(B), _addr(C)),
           "tc_gemm_i8_dequant")


def tc_gemm_i8_dequant_async(ctx: Context, d: tc_gemm_desc, A, B, C, col_scale, stream: Stream):
    _check_capacity(d, A, B, C)
    _require(col_scale, d.N, "col_scale")
    _check(_lib.tc_gemm_i8_dequant_async(ctx.ptr, ctypes.byref(d), _addr(col_scale), _addr(A), _addr(B), _addr(C),
                                         stream.ptr), "tc_gemm_i8_dequant_async")


def tc_gemm_q8_weight(ctx: Context, d: tc_gemm_desc, X, W, C, scale):
    """Out = alpha * (X @ W^T) * scale[n] + beta * Out, X [M,K] f16/bf16,
    W [N,K] int8, scale N floats (CUDA tensors), synchronously."""
    _check_capacity(d, X, W, C)
    _require(scale, d.N, "scale")
    _check(_lib.tc_gemm_q8_weight(ctx.ptr, ctypes.byref(d), _addr(scale), _addr(X), _addr(W), _addr(C)),
           "tc_gemm_q8_weight")


def tc_gemm_q8_weight_async(ctx: Context, d: tc_gemm_desc, X, W, C, scale, stream: Stream):
    _check_capacity(d, X, W, C)
    _require(scale, d.N, "scale")
    _check(_lib.tc_gemm_q8_weight_async(ctx.ptr, ctypes.byref(d), _addr(scale), _addr(X), _addr(W), _addr(C),
                                        stream.ptr), "tc_gemm_q8_weight_async")


def tc_gemm_q8_weight_validate(d: tc_gemm_desc, scale=4 << 40, X=1 << 20, W=2 << 40, C=3 << 40) -> int:
    """Host-only validation status of an int8-weight product."""
    return int(_lib.tc_gemm_q8_weight_validate(ctypes.byref(d), _addr(scale), _addr(X), _addr(W), _addr(C)))


def _matrix_2d(t, N: int, K: int, what: str) -> tuple[int, int]:
    """(dtype code, leading dimension) of a CUDA tensor holding [N, K]."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.dim() != 2 or tuple(t.shape) != (N, K) or (K > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be [{N}, {K}] with unit column stride")
    _check_pitch(what, t, N, K)
    return _torch_dtype_code(t), t.stride(0) if N > 1 else 0


def tc_quantize_q4(ctx: Context, W, q: Q4Weight):
    """W [N, K] (f16/bf16/f32 CUDA tensor) into q's codes, scales and zeros,
    synchronously."""
    dt, ld = _matrix_2d(W, q.N, q.K, "W")
    _check(_lib.tc_quantize_q4(ctx.ptr, dt, ld, _addr(W), q.ref), "tc_quantize_q4")


def tc_quantize_q4_async(ctx: Context, W, q: Q4Weight, stream: Stream):
    dt, ld = _matrix_2d(W, q.N, q.K, "W")
    _check(_lib.tc_quantize_q4_async(ctx.ptr, dt, ld, _addr(W), q.ref, stream.ptr), "tc_quantize_q4_async")


def tc_dequantize_q4(ctx: Context, q: Q4Weight, V):
    """V [N, K] (f16/bf16/f32 CUDA tensor) = the values q stands for,
    synchronously."""
    dt, ld = _matrix_2d(V, q.N, q.K, "V")
    _check(_lib.tc_dequantize_q4(ctx.ptr, q.ref, dt, ld, _addr(V)), "tc_dequantize_q4")


def tc_dequantize_q4_async(ctx: Context, q: Q4Weight, V, stream: Stream):
    dt, ld = _matrix_2d(V, q.N, q.K, "V")
    _check(_lib.tc_dequantize_q4_async(ctx.ptr, q.ref, dt, ld, _addr(V), stream.ptr), "tc_dequantize_q4_async")


def tc_q4_validate(q: tc_q4_weight, dtype: int = TC_F16, ld: int = 0, W=1 << 20) -> int:
    """Host-only validation status of a 4-bit weight and a matrix beside it."""
    return int(_lib.tc_q4_validate(ctypes.byref(q) if q is not None else None, dtype, ld, _addr(W)))


def _check_q4_capacity(d: tc_gemm_desc, X, C):
    if min(d.M, d.N, d.K) < 1:
        return   # the library reports the precise error
    _require(X, _extent(d.M, d.K, d.lda or d.K), "X")
    _require(C, _extent(d.M, d.N, d.ldc or d.N), "C")
    # _require counts elements: of a narrower type they would be too few bytes
    import torch
    types = {TC_F16: torch.float16, TC_BF16: torch.bfloat16, TC_F32: torch.float32}
    for name, t, code in (("X", X, d.a_dtype), ("C", C, d.c_dtype)):
        if t is not None and not isinstance(t, int) and t.dtype != types.get(code, t.dtype):
            raise ValueError(f"{name} must have the descriptor's dtype")


def tc_gemm_q4_weight(ctx: Context, d: tc_gemm_desc, X, q: Q4Weight, C):
    """C = alpha * X @ W^T + beta * C, X [M,K] f16/bf16, W the 4-bit weight q
    (d: b_dtype "i4", transpose_b), synchronously."""
    _check_q4_capacity(d, X, C)
    _check(_lib.tc_gemm_q4_weight(ctx.ptr, ctypes.byref(d), q.ref, _addr(X), _addr(C)), "tc_gemm_q4_weight")


def tc_gemm_q4_weight_async(ctx: Context, d: tc_gemm_desc, X, q: Q4Weight, C, stream: Stream):
    _check_q4_capacity(d, X, C)
    _check(_lib.tc_gemm_q4_weight_async(ctx.ptr, ctypes.byref(d), q.ref, _addr(X), _addr(C), stream.ptr),
           "tc_gemm_q4_weight_async")


def tc_gemm_q4_weight_validate(d: tc_gemm_desc, q: tc_q4_weight, X=1 << 20, C=3 << 40) -> int:
    """Host-only validation status of a 4-bit-weight product."""
    return int(_lib.tc_gemm_q4_weight_validate(ctypes.byref(d), ctypes.byref(q), _addr(X), _addr(C)))


def make_moe_desc(tokens, hidden, inter, experts, top_k, x_dtype, y_dtype=None, *, router_dtype="f32",
                  renormalize=True, ldx=0, ld_router=0, ldy=0) -> tc_moe_desc:
    x = _DT_NAMES.get(x_dtype, x_dtype)
    y = _DT_NAMES.get(y_dtype, y_dtype) if y_dtype is not None else x
    return tc_moe_desc(tokens, hidden, inter, experts, top_k, x, _DT_NAMES.get(router_dtype, router_dtype), y,
                       bool(renormalize), ldx, ld_router, ldy)


class PreparedMoe:
    """A mixture-of-experts layer (tc_moe_q4) with its arguments checked and
    marshalled once, as PreparedGemm does for a product: X [tokens, hidden],
    router [experts, hidden], gate_up and down Q4Weights, Y [tokens, hidden],
    and optionally ids (int32) and weights (float32), both [tokens, top_k]
    and contiguous.  enqueue() is one C call; run() the synchronous form."""

    def __init__(self, ctx: Context, d: tc_moe_desc, X, router, gate_up: Q4Weight, down: Q4Weight, Y,
                 stream: Stream | None = None, *, ids=None, weights=None):
        import torch
        vp = ctypes.c_void_p
        if min(d.tokens, d.hidden, d.experts, d.top_k) >= 1:
            for name, t, rows, ld, code in (("X", X, d.tokens, d.ldx, d.x_dtype),
                                            ("router", router, d.experts, d.ld_router, d.router_dtype),
                                            ("Y", Y, d.tokens, d.ldy, d.y_dtype)):
                _require(t, _extent(rows, d.hidden, ld or d.hidden), name)
                if not isinstance(t, int) and _torch_dtype_code(t) != code:
                    raise ValueError(f"{name} must have the descriptor's dtype")
            for name, t, dt in (("ids", ids, torch.int32), ("weights", weights, torch.float32)):
                _require(t, d.tokens * d.top_k, name)
                if t is not None and not isinstance(t, int) and (t.dtype != dt or not t.is_contiguous()):
                    raise ValueError(f"{name} must be contiguous {dt}")
        self._args = (vp(ctx.ptr), ctypes.byref(d), vp(_addr(X)), vp(_addr(router)), gate_up.ref, down.ref,
                      vp(_addr(Y)), vp(_addr(ids) or None), vp(_addr(weights) or None))
        self._async = self._args + (vp(stream.ptr),) if stream is not None else None
        self._keep = (ctx, d, X, router, gate_up, down, Y, stream, ids, weights)

    def enqueue(self):
        if self._async is None:
            raise ValueError("enqueue() needs the stream the layer was prepared with")
        _check(_lib.tc_moe_q4_async(*self._async), "tc_moe_q4_async")

    def run(self):
        _check(_lib.tc_moe_q4(*self._args), "tc_moe_q4")


def tc_moe_q4(ctx: Context, d: tc_moe_desc, X, router, gate_up: Q4Weight, down: Q4Weight, Y, ids=None, weights=None):
    """A mixture-of-experts layer over 4-bit weights (include/tcgemm.h),
    synchronously."""
    PreparedMoe(ctx, d, X, router, gate_up, down, Y, ids=ids, weights=weights).run()


def tc_moe_q4_async(ctx: Context, d: tc_moe_desc, X, router, gate_up: Q4Weight, down: Q4Weight, Y, stream: Stream,
                    ids=None, weights=None):
    PreparedMoe(ctx, d, X, router, gate_up, down, Y, stream, ids=ids, weights=weights).enqueue()


def tc_moe_q4_validate(d: tc_moe_desc, gate_up: tc_q4_weight, down: tc_q4_weight, X=1 << 20, router=1 << 30,
                       Y=3 << 40, ids=None, weights=None) -> int:
    """Host-only validation status of a mixture-of-experts layer."""
    return int(_lib.tc_moe_q4_validate(ctypes.byref(d), _addr(X), _addr(router), ctypes.byref(gate_up),
                                       ctypes.byref(down), _addr(Y), _addr(ids) or None, _addr(weights) or None))


def make_xent_desc(tokens, hidden, vocab, dtype, grad_dtype=None, *, reduction="mean", scale=1.0, z_weight=0.0,
                   target_dtype="i64", ldx=0, ldw=0, lddx=0, lddw=0) -> tc_xent_desc:
    """reduction: "none", "sum" or "mean" (or a TC_REDUCE_* code)."""
    dt = _DT_NAMES.get(dtype, dtype)
    return tc_xent_desc(tokens, hidden, vocab, dt, _DT_NAMES.get(grad_dtype, grad_dtype) if grad_dtype is not None else dt,
                        _DT_NAMES.get(target_dtype, target_dtype), _REDUCTIONS.get(reduction, reduction), float(scale),
                        float(z_weight), ldx, ldw, lddx, lddw)


def _check_operand(name: str, t, n_elems: int, code: int):
    """Capacity in elements, and the type they are counted in."""
    import torch
    _require(t, n_elems, name)
    types = {TC_F16: torch.float16, TC_BF16: torch.bfloat16, TC_F32: torch.float32, TC_I32: torch.int32,
             TC_I64: torch.int64}
    if t is not None and not isinstance(t, int) and t.dtype != types.get(code, t.dtype):
        raise ValueError(f"{name} is {t.dtype}, the call needs {types[code]}")


def _check_vector(name: str, t, n_elems: int, code: int):
    _check_operand(name, t, n_elems, code)
    if t is not None and not isinstance(t, int) and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_rows(name: str, t, rows: int, cols: int, ld: int, code: int):
    """A matrix at the descriptor's leading dimension: a 2-D tensor of that stride,
    or a contiguous one of any shape where the rows follow one another."""
    _check_operand(name, t, _extent(rows, cols, ld or cols), code)
    if t is None or isinstance(t, int) or ((ld or cols) == cols and t.is_contiguous()):
        return
    if t.dim() != 2 or (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) != (ld or cols)):
        raise ValueError(f"{name} has strides {tuple(t.stride())}, the descriptor rows of {cols} at {ld or cols}")


def _check_device(ctx: Context, **tensors):
    """The context's kernels run on its device."""
    for name, t in tensors.items():
        if t is not None and not isinstance(t, int) and t.is_cuda and t.device.index != ctx.device:
            raise ValueError(f"{name} is on {t.device}, the context on device {ctx.device}")


def _prepared_call(name: str, args, stream, wait: bool):
    """A prepared half of a training loss: synchronously, or on its stream."""
    if args is None:
        raise ValueError(f"{name} was not prepared: its outputs are missing")
    if wait:
        return _check(getattr(_lib, name)(*args), name)
    if stream is None:
        raise ValueError("enqueueing needs the stream the call was prepared with")
    _check(getattr(_lib, name + "_async")(*args, stream), name + "_async")


class PreparedXent:
    """A softmax cross entropy against a vocabulary (tc_linear_xent) with its
    arguments checked and marshalled once: X [tokens, hidden], W [vocab,
    hidden], targets [tokens], lse [tokens].  With ``loss`` (tokens floats, or
    one where the descriptor reduces), enqueue() writes it and lse; with
    ``grad`` (as loss) and ``dX`` and/or ``dW``, enqueue_backward() writes
    those from lse.  One C call each; the tensors stay referenced as long as
    this object."""

    def __init__(self, ctx: Context, d: tc_xent_desc, X, W, targets, lse, stream: Stream | None = None, *, loss=None,
                 grad=None, dX=None, dW=None):
        vp = ctypes.c_void_p
        if loss is None and grad is None:
            raise ValueError("give loss, or grad with dX or dW")
        if (grad is None) != (dX is None and dW is None):
            raise ValueError("grad comes with dX or dW")
        if min(d.tokens, d.hidden, d.vocab) >= 1:
            n = d.tokens if d.reduction == TC_REDUCE_NONE else 1
            _check_rows("X", X, d.tokens, d.hidden, d.ldx, d.dtype)
            _check_rows("W", W, d.vocab, d.hidden, d.ldw, d.dtype)
            _check_rows("dX", dX, d.tokens, d.hidden, d.lddx, d.grad_dtype)
            _check_rows("dW", dW, d.vocab, d.hidden, d.lddw, d.grad_dtype)
            _check_vector("targets", targets, d.tokens, d.target_dtype)
            for name, t, count in (("lse", lse, d.tokens), ("loss", loss, n), ("grad", grad, n)):
                _check_vector(name, t, count, TC_F32)
        _check_device(ctx, X=X, W=W, targets=targets, lse=lse, loss=loss, grad=grad, dX=dX, dW=dW)
        head = (vp(ctx.ptr), ctypes.byref(d), vp(_addr(X)), vp(_addr(W)), vp(_addr(targets)))
        self._forward = head + (vp(_addr(loss)), vp(_addr(lse))) if loss is not None else None
        self._backward = head + (vp(_addr(lse)), vp(_addr(grad)), vp(_addr(dX) or None), vp(_addr(dW) or None)) \
            if grad is not None else None
        self._stream = vp(stream.ptr) if stream is not None else None
        self._keep = (ctx, d, X, W, targets, lse, stream, loss, grad, dX, dW)

    def enqueue(self):
        _prepared_call("tc_linear_xent", self._forward, self._stream, False)

    def run(self):
        _prepared_call("tc_linear_xent", self._forward, self._stream, True)

    def enqueue_backward(self):
        _prepared_call("tc_linear_xent_backward", self._backward, self._stream, False)

    def run_backward(self):
        _prepared_call("tc_linear_xent_backward", self._backward, self._stream, True)


def tc_linear_xent(ctx: Context, d: tc_xent_desc, X, W, targets, loss, lse):
    """Softmax cross entropy of X's rows against W's (include/tcgemm.h),
    synchronously."""
    PreparedXent(ctx, d, X, W, targets, lse, loss=loss).run()


def tc_linear_xent_async(ctx: Context, d: tc_xent_desc, X, W, targets, loss, lse, stream: Stream):
    PreparedXent(ctx, d, X, W, targets, lse, stream, loss=loss).enqueue()


def tc_linear_xent_backward(ctx: Context, d: tc_xent_desc, X, W, targets, lse, grad, dX=None, dW=None):
    """Its gradients (either may be None) from the lse it wrote, synchronously."""
    PreparedXent(ctx, d, X, W, targets, lse, grad=grad, dX=dX, dW=dW).run_backward()


def tc_linear_xent_backward_async(ctx: Context, d: tc_xent_desc, X, W, targets, lse, grad, dX, dW, stream: Stream):
    PreparedXent(ctx, d, X, W, targets, lse, stream, grad=grad, dX=dX, dW=dW).enqueue_backward()


def tc_linear_xent_validate(d: tc_xent_desc, X=1 << 20, W=1 << 40, targets=2 << 40, loss=3 << 40, lse=4 << 40) -> int:
    """Host-only validation status of a softmax cross entropy."""
    return int(_lib.tc_linear_xent_validate(ctypes.byref(d) if d is not None else None, _addr(X), _addr(W),
                                            _addr(targets), _addr(loss), _addr(lse)))


def tc_linear_xent_backward_validate(d: tc_xent_desc, X=1 << 20, W=1 << 40, targets=2 << 40, lse=4 << 40,
                                     grad=5 << 40, dX=6 << 40, dW=7 << 40) -> int:
    return int(_lib.tc_linear_xent_backward_validate(ctypes.byref(d) if d is not None else None, _addr(X), _addr(W),
                                                     _addr(targets), _addr(lse), _addr(grad), _addr(dX) or None,
                                                     _addr(dW) or None))


def make_route_desc(tokens, experts, top_k, logits_dtype="f32", grad_dtype=None, *, renormalize=True, ld_logits=0,
                    ld_dlogits=0) -> tc_route_desc:
    dt = _DT_NAMES.get(logits_dtype, logits_dtype)
    return tc_route_desc(tokens, experts, top_k, dt,
                         _DT_NAMES.get(grad_dtype, grad_dtype) if grad_dtype is not None else dt, bool(renormalize),
                         ld_logits, ld_dlogits)


class PreparedRoute:
    """A routing of tokens to experts (tc_moe_route) with its arguments checked
    and marshalled once: logits [tokens, experts], ids int32 [tokens, top_k],
    counts int32 [experts + 1], and valid (uint8 or bool [tokens]) or None.
    With ``weights`` (float32, as ids) and ``losses`` (two floats), enqueue()
    writes ids, weights, counts and losses; with ``dlogits``, and
    ``grad_weights`` and/or ``grad_losses``, enqueue_backward() writes the
    logits' gradient.  One C call each; the tensors stay referenced as long as
    this object."""

    def __init__(self, ctx: Context, d: tc_route_desc, logits, ids, counts, stream: Stream | None = None, *, valid=None,
                 weights=None, losses=None, grad_weights=None, grad_losses=None, dlogits=None):
        import torch
        vp = ctypes.c_void_p
        if (weights is None) != (losses is None):
            raise ValueError("weights come with losses")
        if weights is None and dlogits is None:
            raise ValueError("give weights and losses, or dlogits")
        if dlogits is None and (grad_weights is not None or grad_losses is not None):
            raise ValueError("gradients come with dlogits")
        if min(d.tokens, d.experts, d.top_k) >= 1:
            n = d.tokens * d.top_k
            _check_rows("logits", logits, d.tokens, d.experts, d.ld_logits, d.logits_dtype)
            _check_rows("dlogits", dlogits, d.tokens, d.experts, d.ld_dlogits, d.grad_dtype)
            for name, t, count, code in (("ids", ids, n, TC_I32), ("counts", counts, d.experts + 1, TC_I32),
                                         ("weights", weights, n, TC_F32), ("losses", losses, 2, TC_F32),
                                         ("grad_weights", grad_weights, n, TC_F32),
                                         ("grad_losses", grad_losses, 2, TC_F32)):
                _check_vector(name, t, count, code)
            if valid is not None and not isinstance(valid, int):
                if valid.dtype not in (torch.uint8, torch.bool):
                    raise ValueError("valid must be uint8 or bool")
                _check_vector("valid", valid, d.tokens, TC_I8)
        _check_device(ctx, logits=logits, ids=ids, counts=counts, valid=valid, weights=weights, losses=losses,
                      grad_weights=grad_weights, grad_losses=grad_losses, dlogits=dlogits)
        head = (vp(ctx.ptr), ctypes.byref(d), vp(_addr(logits)), vp(_addr(valid) or None), vp(_addr(ids)))
        self._forward = head + (vp(_addr(weights)), vp(_addr(counts)), vp(_addr(losses))) if weights is not None else None
        self._backward = head + (vp(_addr(counts)), vp(_addr(grad_weights) or None), vp(_addr(grad_losses) or None),
                                 vp(_addr(dlogits))) if dlogits is not None else None
        self._stream = vp(stream.ptr) if stream is not None else None
        self._keep = (ctx, d, logits, ids, counts, stream, valid, weights, losses, grad_weights, grad_losses, dlogits)

    def enqueue(self):
        _prepared_call("tc_moe_route", self._forward, self._stream, False)

    def run(self):
        _prepared_call("tc_moe_route", self._forward, self._stream, True)

    def enqueue_backward(self):
        _prepared_call("tc_moe_route_backward", self._backward, self._stream, False)

    def run_backward(self):
        _prepared_call("tc_moe_route_backward", self._backward, self._stream, True)


def tc_moe_route(ctx: Context, d: tc_route_desc, logits, ids, weights, counts, losses, valid=None):
    """Choice of experts, its weights, counts and losses (include/tcgemm.h),
    synchronously."""
    PreparedRoute(ctx, d, logits, ids, counts, valid=valid, weights=weights, losses=losses).run()


def tc_moe_route_async(ctx: Context, d: tc_route_desc, logits, ids, weights, counts, losses, stream: Stream, valid=None):
    PreparedRoute(ctx, d, logits, ids, counts, stream, valid=valid, weights=weights, losses=losses).enqueue()


def tc_moe_route_backward(ctx: Context, d: tc_route_desc, logits, ids, counts, dlogits, grad_weights=None,
                          grad_losses=None, valid=None):
    """The logits' gradient, synchronously."""
    PreparedRoute(ctx, d, logits, ids, counts, valid=valid, grad_weights=grad_weights, grad_losses=grad_losses,
                  dlogits=dlogits).run_backward()


def tc_moe_route_backward_async(ctx: Context, d: tc_route_desc, logits, ids, counts, dlogits, stream: Stream,
                                grad_weights=None, grad_losses=None, valid=None):
    PreparedRoute(ctx, d, logits, ids, counts, stream, valid=valid, grad_weights=grad_weights, grad_losses=grad_losses,
                  dlogits=dlogits).enqueue_backward()


def tc_moe_route_validate(d: tc_route_desc, logits=1 << 40, valid=None, ids=2 << 40, weights=3 << 40, counts=4 << 40,
                          losses=5 << 40) -> int:
    """Host-only validation status of a routing."""
    return int(_lib.tc_moe_route_validate(ctypes.byref(d) if d is not None else None, _addr(logits), _addr(valid) or None,
                                          _addr(ids), _addr(weights), _addr(counts), _addr(losses)))


def tc_moe_route_backward_validate(d: tc_route_desc, logits=1 << 40, valid=None, ids=2 << 40, counts=4 << 40,
                                   grad_weights=6 << 40, grad_losses=7 << 40, dlogits=8 << 40) -> int:
    return int(_lib.tc_moe_route_backward_validate(ctypes.byref(d) if d is not None else None, _addr(logits),
                                                   _addr(valid) or None, _addr(ids), _addr(counts),
                                                   _addr(grad_weights) or None, _addr(grad_losses) or None, _addr(dlogits)))


def tc_gemm_host(ctx: Context, d: tc_gemm_desc, A_host, B_host, C_host):
    """Host operands (CPU tensors, ideally pinned): copy in, run, copy out."""
    for t in (A_host, B_host, C_host):
        if not isinstance(t, int) and t.is_cuda:
            raise ValueError("tc_gemm_host takes host tensors")
    _check(_lib.tc_gemm_host(ctx.ptr, ctypes.byref(d), _addr(A_host), _addr(B_host), _addr(C_host)),
           "tc_gemm_host")


def tc_gemm_splitk_noalloc(d: tc_gemm_desc, A, B, C, split: int = 0, torch_stream=None):
    """Split-K GEMM whose scratch is the library's static device buffer:
    nothing is allocated (for callers that must not allocate device memory;
    see include/tcgemm.h).  Asynchronous on ``torch_stream`` (default: the
    legacy default stream); calls that overlap on the GPU race."""
    _check_capacity(d, A, B, C)
    handle = torch_stream.cuda_stream if torch_stream is not None else 0
    _check(_lib.tc_gemm_splitk_noalloc(ctypes.byref(d), _addr(A), _addr(B), _addr(C), int(split),
                                       ctypes.c_void_p(handle)), "tc_gemm_splitk_noalloc")


def tc_gemm_validate(d: tc_gemm_desc, A=1 << 20, B=2 << 40, C=3 << 40) -> int:
    """Host-only validation status (no device needed)."""
    return int(_lib.tc_gemm_validate(ctypes.byref(d) if d is not None else None,
                                     _addr(A), _addr(B), _addr(C)))


def tc_gemm_batched_validate(bd: tc_gemm_batched_desc, A=1 << 20, B=2 << 40, C=3 << 40) -> int:
    return int(_lib.tc_gemm_batched_validate(ctypes.byref(bd), _addr(A), _addr(B), _addr(C)))


def tc_gemm_plan(d: tc_gemm_desc, A=1 << 20, B=2 << 40, C=3 << 40, num_sms: int = 152) -> str:
    """The variant the dispatcher picks (host-only)."""
    buf = ctypes.create_string_buffer(256)
    _check(_lib.tc_gemm_plan(ctypes.byref(d), _addr(A), _addr(B), _addr(C), num_sms, buf, 256),
           "tc_gemm_plan")
    return buf.value.decode()


def tc_last_kernel(ctx: Context) -> str:
    return ctx.last_kernel


def tc_launch_count(ctx: Context) -> int:
    return ctx.launch_count


def tc_status_string(status: int) -> str:
    return _lib.tc_status_string(status).decode()


# ------------------------------------------------------------------ tensor API

@dataclass
class _Shapes:
    M: int
    N: int
    K: int


def gemm(ctx: Context, A, B, C, *, transpose_a=False, transpose_b=False, alpha=1.0, beta=0.0,
         stream: Stream | None = None):
    """C = alpha*op(A)@op(B) + beta*C on torch CUDA tensors (2-D, row-major,
    unit column stride; row strides become leading dimensions)."""
    for name, t in (("A", A), ("B", B), ("C", C)):
        if t.dim() != 2 or t.stride(1) != 1:
            raise ValueError(f"{name} must be 2-D with unit column stride")
    M = A.shape[1] if transpose_a else A.shape[0]
    K = A.shape[0] if transpose_a else A.shape[1]
    N = B.shape[0] if transpose_b else B.shape[1]
    d = tc_gemm_desc(M, N, K, _torch_dtype_code(A), _torch_dtype_code(B), _torch_dtype_code(C), TC_F32,
                     bool(transpose_a), bool(transpose_b), float(alpha), float(beta),
                     A.stride(0), B.stride(0), C.stride(0))
    if stream is None:
        tc_gemm(ctx, d, A, B, C)
    else:
        tc_gemm_async(ctx, d, A, B, C, stream)
    return C
