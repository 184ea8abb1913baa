"""Thin ctypes binding of libtgemm (include/tgemm.h): argument marshalling only.

Every step of the product runs in the library's HIP kernels; PyTorch, when used, only
supplies device memory (``data_ptr()``) and streams (``cuda_stream``).  There is no CPU
fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import collections
import ctypes
import os

F16, BF16 = 0, 1
B_NK, B_KN = 0, 1
A_MK, A_KM = 0, 1
(KERNEL_GENERIC, KERNEL_TILED, KERNEL_SKINNY, KERNEL_DMA, KERNEL_PINGPONG, KERNEL_QUAD,
 KERNEL_SPLITK, KERNEL_DIRECT, KERNEL_QUAD_SPLITK, KERNEL_QUAD_STREAMK,
 KERNEL_MASKED) = range(11)
# the kernels that take operands of any 2-byte alignment
ANY_ALIGNMENT_KERNELS = (KERNEL_GENERIC, KERNEL_MASKED)
SPLIT_KERNELS = (KERNEL_SPLITK, KERNEL_QUAD_SPLITK)   # split K over workgroups (workspace)
WORKSPACE_KERNELS = SPLIT_KERNELS + (KERNEL_QUAD_STREAMK,)   # need a lent workspace
STREAMK_WORKSPACE_BYTES = 128 << 20                   # a QUAD_STREAMK configuration's

F32 = 2                     # logits of moe_route and moe_route_backward only
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1

SCRATCH_BYTES = 16 << 20    # the fixed per-GPU scratch of gemm_ex_noalloc
CLOCK_STAMP_SLOTS = 4096    # compute-unit slots of one clock stamp (2 int64 each)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtgemm.so")

EXPORTS = ("attn_fwd_f16", "gemm_f16", "gemm_bf16", "gemm_ex", "gemm_ex_ws", "gemm_ex_noalloc",
           "gemm_strided",
           "gemm_fused", "gemm_fused_backward", "gemm_grouped", "gemm_grouped_backward",
           "gemm_backward_workspace_size", "moe_route", "moe_route_backward", "moe_plan",
           "moe_plan_workspace_size", "moe_combine", "moe_combine_backward",
           "tgemm_query_config", "tgemm_query_config_ex", "tgemm_query_config_ws",
           "tgemm_workspace_size", "tgemm_list_configs", "tgemm_list_configs_ex",
           "tgemm_status_string", "tgemm_version", "tgemm_clock_stamp",
           "tgemm_wall_clock_hz")


__all__ = ["F16", "BF16", "B_NK", "B_KN", "A_MK", "A_KM", "KERNEL_GENERIC", "KERNEL_TILED",
           "KERNEL_SKINNY", "KERNEL_DMA", "KERNEL_PINGPONG", "KERNEL_QUAD", "KERNEL_SPLITK",
           "KERNEL_QUAD_SPLITK", "KERNEL_QUAD_STREAMK", "KERNEL_MASKED", "SPLIT_KERNELS",
           "WORKSPACE_KERNELS", "ALIGN_OPERANDS",
           "ANY_ALIGNMENT_KERNELS",
           "STREAMK_WORKSPACE_BYTES",
           "KERNEL_DIRECT",
           "LIB_PATH", "EXPORTS", "TGemmError", "Config", "load", "status_string", "gemm_f16",
           "gemm_bf16", "gemm_ex", "gemm_ex_ws", "gemm_ex_noalloc", "gemm_strided",
           "query_config", "SCRATCH_BYTES", "CLOCK_STAMP_SLOTS",
           "query_config_packed", "query_config_ws", "workspace_size", "list_configs",
           "attn_fwd_f16", "version", "gemm", "clock_stamp", "wall_clock_hz",
           "F32", "ACT_NONE", "ACT_RELU", "ACT_GELU", "ACT_GELU_TANH", "ACT_SILU",
           "SCORE_SOFTMAX", "SCORE_SIGMOID", "GROUP_MAX", "GROUP_TOP2", "Epilogue", "Plan",
           "gemm_fused", "gemm_fused_backward", "gemm_grouped", "gemm_grouped_backward",
           "backward_workspace_size", "moe_route", "moe_route_backward", "moe_plan",
           "plan_workspace_size", "moe_combine", "moe_combine_backward"]


class TGemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class Config(ctypes.Structure):
    """tgemm_config."""
    _fields_ = [("kernel", ctypes.c_int32), ("block_m", ctypes.c_int32),
                ("block_n", ctypes.c_int32), ("block_k", ctypes.c_int32),
                ("waves_m", ctypes.c_int32), ("waves_n", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("group_m", ctypes.c_int32),
                ("split_k", ctypes.c_int32), ("mfma", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {name: int(getattr(self, name)) for name, _ in self._fields_}

    @classmethod
    def from_dict(cls, d: dict) -> "Config":
        return cls(**{name: int(d[name]) for name, _ in cls._fields_})

    def __repr__(self):
        return f"Config({self.as_dict()})"


class Epilogue(ctypes.Structure):
    """tgemm_epilogue."""
    _fields_ = [("activation", ctypes.c_int32), ("gated", ctypes.c_int32),
                ("bias", ctypes.c_void_p), ("bias_stride", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("preact", ctypes.c_void_p), ("ldp", ctypes.c_int64)]


_lib = None


def load(path: str = LIB_PATH):
    """Load libtgemm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(
            f"{path} is missing: build it first (python -m tiled_dense_gemm_major_amd.build)")
    lib = ctypes.CDLL(path)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    cfgp = ctypes.POINTER(Config)
    lib.gemm_f16.argtypes = [i64, i64, i64, vp, vp, vp, i32, vp]
    lib.gemm_bf16.argtypes = [i64, i64, i64, vp, vp, vp, i32, vp]
    lib.gemm_ex.argtypes = [i32, i64, i64, i64, vp, vp, vp, i32, cfgp, vp]
    lib.gemm_ex_ws.argtypes = [i32, i64, i64, i64, vp, vp, vp, i32, cfgp, vp, i64, vp]
    lib.gemm_ex_noalloc.argtypes = [i32, i64, i64, i64, vp, vp, vp, i32, cfgp, vp]
    lib.attn_fwd_f16.argtypes = [i64, i64, i64, i64, vp, vp, vp, vp, i32, vp]
    lib.gemm_strided.argtypes = [i32, i64, i64, i64, vp, i64, i32, vp, i64, i32, vp, i64,
                                 cfgp, vp]
    f32, epip, i64p = ctypes.c_float, ctypes.POINTER(Epilogue), ctypes.POINTER(ctypes.c_int64)
    lib.gemm_fused.argtypes = [i32, i64, i64, i64, vp, i64, vp, i64, i32, vp, i64, epip, vp]
    lib.gemm_fused_backward.argtypes = [i32, i64, i64, i64, vp, i64, vp, i64, vp, i64, i32, i32,
                                        i32, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, i64,
                                        vp]
    lib.gemm_grouped.argtypes = [i32, i64, i64, i64, i64, vp, vp, i64, vp, i64, i64, vp, i64,
                                 i64, i32, vp, i64, epip, vp]
    lib.gemm_grouped_backward.argtypes = [i32, i64, i64, i64, i64, vp, vp, i64, vp, i64, vp,
                                          i64, i64, vp, i64, i64, i32, i32, i32, vp, i64, vp,
                                          i64, vp, i64, vp, i64, i64, vp, vp, i64, vp]
    lib.gemm_backward_workspace_size.argtypes = [i64, i64, i64, i64, i32, i64p]
    lib.moe_route.argtypes = [i32, i64, i64, i64, vp, i64, vp, i32, i64, i64, i32, i32, f32, vp,
                              vp, vp]
    lib.moe_route_backward.argtypes = [i32, i64, i64, i64, vp, i64, vp, vp, i32, i32, f32, vp,
                                       i64, vp]
    lib.moe_plan.argtypes = [i64, i64, vp, vp, vp, vp, vp, i64, vp]
    lib.moe_plan_workspace_size.argtypes = [i64, i64, i64p]
    lib.moe_combine.argtypes = [i32, i64, i64, i64, vp, i64, i64, vp, vp, vp, i64, vp, i64, vp]
    lib.moe_combine_backward.argtypes = [i32, i64, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp,
                                         i64, vp, vp]
    lib.tgemm_query_config.argtypes = [i32, i64, i64, i64, i32, cfgp]
    lib.tgemm_query_config_ex.argtypes = [i32, i64, i64, i64, i32, i32, i32, cfgp]
    lib.tgemm_query_config_ws.argtypes = [i32, i64, i64, i64, i32, i32, cfgp,
                                          ctypes.POINTER(ctypes.c_int64)]
    lib.tgemm_workspace_size.argtypes = [i64, i64, cfgp, ctypes.POINTER(ctypes.c_int64)]
    lib.tgemm_list_configs.argtypes = [i32, i32, cfgp, i32]
    lib.tgemm_list_configs_ex.argtypes = [i32, i32, i32, cfgp, i32]
    lib.tgemm_clock_stamp.argtypes = [vp, vp]
    lib.tgemm_wall_clock_hz.argtypes = [ctypes.POINTER(ctypes.c_int64)]
    lib.tgemm_status_string.argtypes = [i32]
    lib.tgemm_status_string.restype = ctypes.c_char_p
    for name in EXPORTS:
        if name != "tgemm_status_string":
            getattr(lib, name).restype = i32
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().tgemm_status_string(status).decode()


def _addr(x) -> int:
    """A device address from a torch tensor, an int, or None (NULL)."""
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        try:
            import torch
            if torch.cuda.is_available():
                return int(torch.cuda.current_stream().cuda_stream)
        except ImportError:
            pass
        return 0
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _check(rc: int, what: str):
    if rc != 0:
        raise TGemmError(rc, what)


def gemm_f16(m, n, k, A, B, C, b_layout=B_NK, stream=None):
    """C = A x B^T (B_NK) or A x B (B_KN), fp16.  A, B, C: device tensors or addresses."""
    _check(load().gemm_f16(m, n, k, _addr(A), _addr(B), _addr(C), b_layout, _stream(stream)),
           "gemm_f16")


def gemm_bf16(m, n, k, A, B, C, b_layout=B_NK, stream=None):
    """C = A x B^T (B_NK) or A x B (B_KN), bf16.  A, B, C: device tensors or addresses."""
    _check(load().gemm_bf16(m, n, k, _addr(A), _addr(B), _addr(C), b_layout, _stream(stream)),
           "gemm_bf16")


def gemm_ex(dtype, m, n, k, A, B, C, b_layout=B_NK, config: Config | None = None,
            stream=None):
    """The product with an explicit dtype and, optionally, an explicit configuration."""
    cfg = ctypes.byref(config) if config is not None else None
    _check(load().gemm_ex(dtype, m, n, k, _addr(A), _addr(B), _addr(C), b_layout, cfg,
                          _stream(stream)), "gemm_ex")


def gemm_ex_ws(dtype, m, n, k, A, B, C, workspace, workspace_bytes, b_layout=B_NK,
               config: Config | None = None, stream=None):
    """gemm_ex with a caller-lent device workspace (split-K configurations need one)."""
    cfg = ctypes.byref(config) if config is not None else None
    _check(load().gemm_ex_ws(dtype, m, n, k, _addr(A), _addr(B), _addr(C), b_layout, cfg,
                             _addr(workspace) if workspace is not None else None,
                             int(workspace_bytes), _stream(stream)), "gemm_ex_ws")


def gemm_ex_noalloc(dtype, m, n, k, A, B, C, b_layout=B_NK, config: Config | None = None,
                    stream=None):
    """gemm_ex_ws with the library's fixed scratch as the workspace: allocates nothing."""
    cfg = ctypes.byref(config) if config is not None else None
    _check(load().gemm_ex_noalloc(dtype, m, n, k, _addr(A), _addr(B), _addr(C), b_layout, cfg,
                                  _stream(stream)), "gemm_ex_noalloc")


ALIGN_OPERANDS = 2   # `aligned` value: A and B meet the fast rules, C or N does not


def _align_arg(aligned) -> int:
    return ALIGN_OPERANDS if (not isinstance(aligned, bool) and aligned == ALIGN_OPERANDS) \
        else int(bool(aligned))


def query_config_ws(dtype, m, n, k, b_layout=B_NK, aligned=True):
    """(configuration, workspace bytes) the table picks when a workspace can be lent;
    aligned: True (every fast-kernel rule), False (none) or ALIGN_OPERANDS."""
    out = Config()
    nbytes = ctypes.c_int64(0)
    _check(load().tgemm_query_config_ws(dtype, m, n, k, b_layout, _align_arg(aligned),
                                        ctypes.byref(out), ctypes.byref(nbytes)),
           "tgemm_query_config_ws")
    return out, int(nbytes.value)


def workspace_size(m, n, config: Config) -> int:
    nbytes = ctypes.c_int64(0)
    _check(load().tgemm_workspace_size(m, n, ctypes.byref(config), ctypes.byref(nbytes)),
           "tgemm_workspace_size")
    return int(nbytes.value)


def gemm_strided(dtype, m, n, k, A, lda, a_layout, B, ldb, b_layout, C, ldc,
                 config: Config | None = None, stream=None):
    """The general product: A [M,K] (A_MK) or [K,M] (A_KM), B [N,K] (B_NK) or [K,N] (B_KN),
    C [M,N], each with a leading dimension in elements."""
    cfg = ctypes.byref(config) if config is not None else None
    _check(load().gemm_strided(dtype, m, n, k, _addr(A), lda, a_layout, _addr(B), ldb,
                               b_layout, _addr(C), ldc, cfg, _stream(stream)), "gemm_strided")


def query_config(dtype, m, n, k, b_layout=B_NK, aligned=True, a_layout=A_MK) -> Config:
    """The choice for an alignment class: aligned True (every fast-kernel rule), False
    (none: the masked kernel) or ALIGN_OPERANDS (A and B meet the rules, C or N does not)."""
    out = Config()
    _check(load().tgemm_query_config_ex(dtype, m, n, k, a_layout, b_layout,
                                        _align_arg(aligned), ctypes.byref(out)),
           "tgemm_query_config_ex")
    return out


def query_config_packed(dtype, m, n, k, b_layout=B_NK) -> Config:
    """What gemm_f16 / gemm_bf16 pick for packed operands at 16-byte-aligned addresses
    (tgemm_query_config: the sizes decide whether the fast kernels apply)."""
    out = Config()
    _check(load().tgemm_query_config(dtype, m, n, k, b_layout, ctypes.byref(out)),
           "tgemm_query_config")
    return out


def list_configs(dtype, b_layout=B_NK, a_layout=A_MK) -> list:
    lib = load()
    count = lib.tgemm_list_configs_ex(dtype, a_layout, b_layout, None, 0)
    if count < 0:
        raise TGemmError(count, "tgemm_list_configs_ex")
    arr = (Config * count)()
    lib.tgemm_list_configs_ex(dtype, a_layout, b_layout, arr, count)
    return [arr[i] for i in range(count)]


def attn_fwd_f16(batch, seq, heads, dim, Q, K, V, O, causal=True, stream=None):
    """Attention forward, fp16 tensors [batch, seq, heads, dim]: O = softmax(Q K^T /
    sqrt(dim)) V per (batch, head), causal or not.  Q, K, V, O: device tensors or
    addresses."""
    _check(load().attn_fwd_f16(batch, seq, heads, dim, _addr(Q), _addr(K), _addr(V), _addr(O),
                               int(bool(causal)), _stream(stream)), "attn_fwd_f16")


def clock_stamp(out, stream=None):
    """Enqueue per-compute-unit (engine-clock counter, wall clock) stamps into ``out`` (a
    zeroed device tensor of CLOCK_STAMP_SLOTS x 2 int64, 16-byte aligned, or an
    address)."""
    if hasattr(out, "numel") and out.numel() < 2 * CLOCK_STAMP_SLOTS:
        raise ValueError(f"clock_stamp needs {2 * CLOCK_STAMP_SLOTS} int64, got {out.numel()}")
    _check(load().tgemm_clock_stamp(_addr(out), _stream(stream)), "tgemm_clock_stamp")


def wall_clock_hz() -> int:
    hz = ctypes.c_int64(0)
    _check(load().tgemm_wall_clock_hz(ctypes.byref(hz)), "tgemm_wall_clock_hz")
    return int(hz.value)


def version() -> int:
    return int(load().tgemm_version())


def gemm(A, B, C=None, b_layout=B_NK, config: Config | None = None, stream=None):
    """Torch convenience: A [M,K], B [N,K] (B_NK) or [K,N] (B_KN), same 16-bit dtype on
    one device; C [M,N] allocated by torch when not given.  Returns C."""
    import torch
    if A.dtype not in (torch.float16, torch.bfloat16) or B.dtype != A.dtype:
        raise TypeError("A and B must share dtype float16 or bfloat16")
    if not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous (packed row-major)")
    M, K = A.shape
    if b_layout == B_NK:
        N, Kb = B.shape
    else:
        Kb, N = B.shape
    if Kb != K:
        raise ValueError(f"K mismatch: {K} vs {Kb}")
    if C is None:
        C = torch.empty((M, N), dtype=A.dtype, device=A.device)
    elif C.shape != (M, N) or C.dtype != A.dtype or not C.is_contiguous():
        raise ValueError("C must be a contiguous [M,N] tensor of the input dtype")
    dtype = F16 if A.dtype == torch.float16 else BF16
    gemm_ex(dtype, M, N, K, A, B, C, b_layout, config, stream)
    return C


# ---- products with an epilogue, routing and experts' products: torch tensors ---------------
#
# Matrices are 2-D tensors whose last dimension is contiguous; the row stride is free.  All
# tensors of a call lie on one GPU, which need not be the current one; the work goes to the
# given stream, or to the current stream of that GPU.  Outputs may be passed in; those that
# are not, and workspaces, are allocated by torch in the pool of the stream that the work
# goes to, so that their memory is not given out again before the work is done.  Tensors
# passed to a call on another stream than their own are the caller's to keep, as for any
# other use on a second stream.  Nothing here is differentiable by itself: the gradients are
# calls of their own.

def _matrix(t, what, like=None, shape=None):
    """(address, rows, columns, row stride) of a 2-D tensor, after its checks."""
    size, step = t.shape, t.stride()
    if len(size) != 2:
        raise ValueError(f"{what} must have 2 dimensions, not {len(size)}")
    rows, cols = size
    if step[1] != 1 and cols > 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    if like is not None and (t.dtype != like.dtype or t.get_device() != like.get_device()):
        raise TypeError(f"{what} must have the dtype and device of the operands "
                        f"({like.dtype}, {like.device}), not {t.dtype}, {t.device}")
    if shape is not None and size != shape:
        raise ValueError(f"{what} must have shape {shape}, not {(rows, cols)}")
    return t.data_ptr(), rows, cols, (step[0] if rows > 1 else max(cols, 1))


def _vector(t, what, like, dtype, count):
    """The address of a contiguous tensor of `count` values of `dtype` on like's GPU."""
    if t.dtype != dtype or t.get_device() != like.get_device():
        raise TypeError(f"{what} must be {dtype} on {like.device}, not {t.dtype} on {t.device}")
    if t.numel() != count or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous with {count} elements, not {tuple(t.shape)}")
    return t.data_ptr()


_torch_names = None


def _torch():
    """The torch module and what the calls below look up in it, once."""
    global _torch_names
    if _torch_names is None:
        import torch
        halves = {torch.float16: F16, torch.bfloat16: BF16}
        # the address of a GPU's current stream, without making a Stream object of it
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch_names = (torch, halves, {**halves, torch.float32: F32}, raw)
    return _torch_names


def _operand_dtype(t, what):
    halves = _torch()[1]
    if t.dtype not in halves:
        raise TypeError(f"{what} must be float16 or bfloat16, not {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a GPU, not on {t.device}")
    return halves[t.dtype]


def _new(like, shape, stream, dtype=None):
    """An uninitialised tensor on like's GPU, in the pool of the given stream (None: the
    current one)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    cuda = _torch()[0].cuda
    if isinstance(stream, int):
        stream = cuda.ExternalStream(stream, device=like.device)
    with cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _launch(name, t, stream, *args):
    """The entry point `name` on t's GPU (kernels launch on the current one) and the given or
    that GPU's current stream."""
    torch, _, _, raw_stream = _torch()
    index = t.get_device()
    if stream is None:
        stream = raw_stream(index)
    elif not isinstance(stream, int):
        stream = int(stream.cuda_stream)
    fn = getattr(load(), name)
    if index == torch.cuda.current_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc != 0:
        raise TGemmError(rc, name)


def _b_sizes(B, b_layout, k):
    """(n, k) of B's last two dimensions, with k checked against A's columns."""
    n, kb = (B.shape[-2], B.shape[-1]) if b_layout == B_NK else (B.shape[-1], B.shape[-2])
    if k is not None and kb != k:
        raise ValueError(f"K mismatch: A has {k} columns, B has {kb}")
    return n, kb


def _epilogue(A, rows, n, width, activation, gated, bias, residual, preact, groups=None):
    """The Epilogue of a call, or None where it adds nothing."""
    if not activation and not gated and bias is None and residual is None and preact is None:
        return None
    e = Epilogue(activation=activation, gated=int(bool(gated)))
    if bias is not None:
        e.bias = _vector(bias, "bias", A, A.dtype, n * (groups or 1))
        e.bias_stride = n
    if residual is not None:
        e.residual, _, _, e.ldr = _matrix(residual, "residual", A, (rows, width))
    if preact is not None:
        e.preact, _, _, e.ldp = _matrix(preact, "preact", A, (rows, n))
    return ctypes.byref(e)


def _width(n, gated):
    if gated and n % 2:
        raise ValueError(f"a gated product needs an even N, not {n}")
    return n // 2 if gated else n


def gemm_fused(A, B, C=None, b_layout=B_NK, bias=None, activation=ACT_NONE, gated=False,
               residual=None, preact=None, stream=None):
    """C = act(z) + residual with z = A x B^T (B_NK) or A x B (B_KN) + bias; gated,
    C = act(z[:, :N/2]) * z[:, N/2:] + residual.  bias [N], residual like C (it may be C),
    preact [M,N] takes z.  Returns C."""
    dtype = _operand_dtype(A, "A")
    a, m, k, lda = _matrix(A, "A")
    b, _, _, ldb = _matrix(B, "B", A)
    n, _ = _b_sizes(B, b_layout, k)
    width = _width(n, gated)
    if C is None:
        C = _new(A, (m, width), stream)
    c, _, _, ldc = _matrix(C, "C", A, (m, width))
    e = _epilogue(A, m, n, width, activation, gated, bias, residual, preact)
    _launch("gemm_fused", A, stream, dtype, m, n, k, a, lda, b, ldb, b_layout, c, ldc, e)
    return C


def backward_workspace_size(rows, n, k=0, groups=1, dbias=True) -> int:
    """Workspace bytes that a backward call can use: needed with dbias, and with k > 0 those
    that let a dB of few tiles over many rows be summed in parts."""
    nbytes = ctypes.c_int64(0)
    _check(load().gemm_backward_workspace_size(groups, rows, n, k, int(bool(dbias)),
                                               ctypes.byref(nbytes)),
           "gemm_backward_workspace_size")
    return int(nbytes.value)


def _gradient(t, like, shape, stream, dtype=None):
    """An output that is wanted (a tensor, or True to allocate it) or not (None, False)."""
    if t is None or t is False:
        return None
    return _new(like, shape, stream, dtype) if t is True else t


def _gradient_buffers(A, rows, n, k, groups, activation, gated, preact, dZ, dA, dB, dbias,
                      workspace, stream):
    """(preact address and stride, dZ address and stride, workspace address and bytes)."""
    z = zs = d = ds = w = wb = 0
    if activation or gated:
        if preact is None:
            raise ValueError("preact is needed with an activation or a gate")
        z, _, _, zs = _matrix(preact, "preact", A, (rows, n))
        if dA is not None or dB is not None:
            if dZ is None:
                dZ = _new(A, (rows, n), stream)
            d, _, _, ds = _matrix(dZ, "dZ", A, (rows, n))
    if workspace is None:
        wb = backward_workspace_size(rows, n, 0 if dB is None else k, groups, dbias is not None)
        if wb:
            workspace = _new(A, (wb,), stream, _torch()[0].uint8)
            w = workspace.data_ptr()
    else:
        if workspace.get_device() != A.get_device() or not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous and on the operands' GPU")
        w, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    # the tensors allocated here are kept until the call has been enqueued
    return z, zs, d, ds, w, wb, (dZ, workspace)


def gemm_fused_backward(dC, A, B, preact=None, b_layout=B_NK, activation=ACT_NONE, gated=False,
                        dZ=None, dA=True, dB=True, dbias=False, workspace=None, stream=None):
    """(dA, dB, dbias) of gemm_fused for dC.  dA, dB, dbias: True (allocated), a tensor to
    fill, or None / False (not wanted; returned as None).  preact [M,N] is what the forward
    call kept (unused without an activation and a gate); dZ [M,N] takes the gradient of z
    (allocated if None; may be preact).  dbias is fp32 [N]."""
    dtype = _operand_dtype(A, "A")
    torch = _torch()[0]
    a, m, k, lda = _matrix(A, "A")
    b, b_rows, b_cols, ldb = _matrix(B, "B", A)
    n, _ = _b_sizes(B, b_layout, k)
    dc, _, _, lddc = _matrix(dC, "dC", A, (m, _width(n, gated)))
    dA, dB = _gradient(dA, A, (m, k), stream), _gradient(dB, A, (b_rows, b_cols), stream)
    dbias = _gradient(dbias, A, (n,), stream, torch.float32)
    da, _, _, ldda = (0, 0, 0, 0) if dA is None else _matrix(dA, "dA", A, (m, k))
    db, _, _, lddb = (0, 0, 0, 0) if dB is None else _matrix(dB, "dB", A, (b_rows, b_cols))
    dbv = 0 if dbias is None else _vector(dbias, "dbias", A, torch.float32, n)
    z, ldz, d, lddz, w, wb, keep = _gradient_buffers(
        A, m, n, k, 1, activation, gated, preact, dZ, dA, dB, dbias, workspace, stream)
    _launch("gemm_fused_backward", A, stream, dtype, m, n, k, dc, lddc, a, lda, b, ldb, b_layout,
            activation, int(bool(gated)), z, ldz, d, lddz, da, ldda, db, lddb, dbv, w, wb)
    return dA, dB, dbias


def _stack(B, what, like, shape=None):
    """(address, row stride, group stride) of a 3-D tensor [groups, rows, columns]."""
    if B.dim() != 3:
        raise ValueError(f"{what} must have 3 dimensions, not {B.dim()}")
    if shape is not None and tuple(B.shape) != shape:
        raise ValueError(f"{what} must have shape {shape}, not {tuple(B.shape)}")
    if B.dtype != like.dtype or B.get_device() != like.get_device():
        raise TypeError(f"{what} must have the dtype and device of the operands "
                        f"({like.dtype}, {like.device}), not {B.dtype}, {B.device}")
    groups, rows, cols = B.shape
    if cols > 1 and B.stride(2) != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return (B.data_ptr(), B.stride(1) if rows > 1 else max(cols, 1),
            B.stride(0) if groups > 1 else 0)


def _groups(A, B, offsets, row_index, row_div):
    """(rows, offsets address, row index address) of a grouped call."""
    torch = _torch()[0]
    off = _vector(offsets, "offsets", A, torch.int32, B.shape[0] + 1)
    if row_index is None:
        return A.shape[0], off, 0
    return row_index.numel(), off, _vector(row_index, "row_index", A, torch.int32,
                                           row_index.numel())


def gemm_grouped(A, B, offsets, C=None, row_index=None, row_div=1, b_layout=B_NK, bias=None,
                 activation=ACT_NONE, gated=False, residual=None, preact=None, stream=None):
    """One product per group of rows, with the epilogue of gemm_fused: rows
    offsets[g] .. offsets[g+1]-1 of C take B[g] (and bias[g]).  B is [groups, N, K] (B_NK) or
    [groups, K, N] (B_KN); with row_index, row s of C reads row row_index[s] // row_div of A.
    Rows of C and preact outside every group keep what they held.  Returns C."""
    dtype = _operand_dtype(A, "A")
    a, a_rows, k, lda = _matrix(A, "A")
    b, ldb, stride_b = _stack(B, "B", A)
    n, _ = _b_sizes(B, b_layout, k)
    width, groups = _width(n, gated), B.shape[0]
    rows, off, idx = _groups(A, B, offsets, row_index, row_div)
    if C is None:
        C = _new(A, (rows, width), stream)
    c, _, _, ldc = _matrix(C, "C", A, (rows, width))
    e = _epilogue(A, rows, n, width, activation, gated, bias, residual, preact, groups)
    _launch("gemm_grouped", A, stream, dtype, groups, rows, n, k, off, idx, row_div, a, a_rows,
            lda, b, ldb, stride_b, b_layout, c, ldc, e)
    return C


def gemm_grouped_backward(dC, A, B, offsets, preact=None, row_index=None, row_div=1,
                          b_layout=B_NK, activation=ACT_NONE, gated=False, dZ=None, dA=True,
                          dB=True, dbias=False, workspace=None, stream=None):
    """(dA, dB, dbias) of gemm_grouped for dC: dA one row per row of C, dB like B, dbias fp32
    [groups, N].  Outputs and the other arguments as in gemm_fused_backward."""
    dtype = _operand_dtype(A, "A")
    torch = _torch()[0]
    a, a_rows, k, lda = _matrix(A, "A")
    b, ldb, stride_b = _stack(B, "B", A)
    n, _ = _b_sizes(B, b_layout, k)
    groups, b_shape = B.shape[0], tuple(B.shape)
    rows, off, idx = _groups(A, B, offsets, row_index, row_div)
    dc, _, _, lddc = _matrix(dC, "dC", A, (rows, _width(n, gated)))
    dA, dB = _gradient(dA, A, (rows, k), stream), _gradient(dB, A, b_shape, stream)
    dbias = _gradient(dbias, A, (groups, n), stream, torch.float32)
    da, _, _, ldda = (0, 0, 0, 0) if dA is None else _matrix(dA, "dA", A, (rows, k))
    db, lddb, stride_db = (0, 0, 0) if dB is None else _stack(dB, "dB", A, b_shape)
    dbv = 0 if dbias is None else _vector(dbias, "dbias", A, torch.float32, groups * n)
    z, ldz, d, lddz, w, wb, keep = _gradient_buffers(
        A, rows, n, k, groups, activation, gated, preact, dZ, dA, dB, dbias, workspace, stream)
    _launch("gemm_grouped_backward", A, stream, dtype, groups, rows, n, k, off, idx, row_div, dc,
            lddc, a, a_rows, lda, b, ldb, stride_b, b_layout, activation, int(bool(gated)), z,
            ldz, d, lddz, da, ldda, db, lddb, stride_db, dbv, w, wb)
    return dA, dB, dbias


def _logits(x, what="logits"):
    names = _torch()[2]
    if x.dtype not in names:
        raise TypeError(f"{what} must be float16, bfloat16 or float32, not {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{what} must be on a GPU, not on {x.device}")
    return (names[x.dtype], *_matrix(x, what))


def moe_route(logits, k, scoring=SCORE_SOFTMAX, bias=None, groups=1, topk_groups=None,
              group_score=GROUP_MAX, renormalize=True, scale=1.0, ids=None, weights=None,
              stream=None):
    """(ids, weights) [tokens, k] of the k experts of each token, from logits
    [tokens, experts]: int32 and fp32, in descending order of the selection values.  bias is
    fp32 [experts] and only selects; groups and topk_groups limit the choice to the best
    groups of experts.  Masked logits (-inf, NaN) are never chosen: id -1, weight 0."""
    torch = _torch()[0]
    dtype, x, tokens, experts, ldx = _logits(logits)
    if ids is None:
        ids = _new(logits, (tokens, k), stream, torch.int32)
    if weights is None:
        weights = _new(logits, (tokens, k), stream, torch.float32)
    i = _vector(ids, "ids", logits, torch.int32, tokens * k)
    w = _vector(weights, "weights", logits, torch.float32, tokens * k)
    bv = 0 if bias is None else _vector(bias, "bias", logits, torch.float32, experts)
    _launch("moe_route", logits, stream, dtype, tokens, experts, k, x, ldx, bv, scoring, groups,
            groups if topk_groups is None else topk_groups, group_score,
            int(bool(renormalize)), scale, i, w)
    return ids, weights


def moe_route_backward(logits, ids, dweights, scoring=SCORE_SOFTMAX, renormalize=True,
                       scale=1.0, dlogits=None, stream=None):
    """The logits' gradient [tokens, experts] from the weights' gradient [tokens, k] fp32, for
    the choices that moe_route made."""
    torch = _torch()[0]
    dtype, x, tokens, experts, ldx = _logits(logits)
    k = ids.shape[-1]
    i = _vector(ids, "ids", logits, torch.int32, tokens * k)
    dw = _vector(dweights, "dweights", logits, torch.float32, tokens * k)
    if dlogits is None:
        dlogits = _new(logits, (tokens, experts), stream)
    dx, _, _, lddx = _matrix(dlogits, "dlogits", logits, (tokens, experts))
    _launch("moe_route_backward", logits, stream, dtype, tokens, experts, k, x, ldx, i, dw,
            scoring, int(bool(renormalize)), scale, dx, lddx)
    return dlogits


Plan = collections.namedtuple("Plan", "offsets order slots")


def plan_workspace_size(choices, experts) -> int:
    """Workspace bytes of moe_plan (0 up to 4096 choices)."""
    nbytes = ctypes.c_int64(0)
    _check(load().moe_plan_workspace_size(choices, experts, ctypes.byref(nbytes)),
           "moe_plan_workspace_size")
    return int(nbytes.value)


def moe_plan(ids, experts, offsets=None, order=None, slots=None, workspace=None, stream=None):
    """The choices ids (int32, [tokens, k]) sorted by expert, as Plan(offsets [experts + 1],
    order [tokens * k], slots like ids): the offsets of gemm_grouped, its row_index (with
    row_div = k) and the slots of moe_combine."""
    torch = _torch()[0]
    if not ids.is_cuda:
        raise ValueError(f"ids must be on a GPU, not on {ids.device}")
    count = ids.numel()
    i = _vector(ids, "ids", ids, torch.int32, count)
    if offsets is None:
        offsets = _new(ids, (experts + 1,), stream)
    if order is None:
        order = _new(ids, (count,), stream)
    if slots is None:
        slots = _new(ids, ids.shape, stream)
    if workspace is None and count > 4096:
        workspace = _new(ids, (plan_workspace_size(count, experts) // 4,), stream)
    w = wb = 0
    if workspace is not None:
        if workspace.get_device() != ids.get_device() or not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous and on the ids' GPU")
        w, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    off = _vector(offsets, "offsets", ids, torch.int32, experts + 1)
    o = _vector(order, "order", ids, torch.int32, count)
    s = _vector(slots, "slots", ids, torch.int32, count)
    _launch("moe_plan", ids, stream, count, experts, i, off, o, s, w, wb)
    return Plan(offsets, order, slots)


def moe_combine(O, slots, weights=None, residual=None, Y=None, stream=None):
    """Y[t] = residual[t] + sum_j weights[t,j] O[slots[t,j]], slots int32 [tokens, k] (one
    outside O adds nothing), weights fp32 [tokens, k] or None (all one).  residual may be Y.
    Returns Y."""
    torch = _torch()[0]
    dtype = _operand_dtype(O, "O")
    o, rows, width, ldo = _matrix(O, "O")
    if slots.dim() != 2:
        raise ValueError("slots must be [tokens, k]")
    tokens, k = slots.shape
    s = _vector(slots, "slots", O, torch.int32, tokens * k)
    w = 0 if weights is None else _vector(weights, "weights", O, torch.float32, tokens * k)
    if Y is None:
        Y = _new(O, (tokens, width), stream)
    y, _, _, ldy = _matrix(Y, "Y", O, (tokens, width))
    r, _, _, ldr = (0, 0, 0, 0) if residual is None else _matrix(residual, "residual", O,
                                                                (tokens, width))
    _launch("moe_combine", O, stream, dtype, tokens, k, width, o, rows, ldo, s, w, r, ldr, y, ldy)
    return Y


def moe_combine_backward(dY, O, slots, weights=None, dO=True, dweights=True, stream=None):
    """(dO, dweights) of moe_combine: dO[slots[t,j]] = weights[t,j] dY[t] (rows that no slot
    names keep what they held; each row is to be named at most once), dweights[t,j] = <dY[t], O[slots[t,j]]> in fp32.  Either:
    True (allocated), a tensor to fill, or None / False (not wanted)."""
    torch = _torch()[0]
    dtype = _operand_dtype(O, "O")
    o, rows, width, ldo = _matrix(O, "O")
    if slots.dim() != 2:
        raise ValueError("slots must be [tokens, k]")
    tokens, k = slots.shape
    dy, _, _, lddy = _matrix(dY, "dY", O, (tokens, width))
    s = _vector(slots, "slots", O, torch.int32, tokens * k)
    w = 0 if weights is None else _vector(weights, "weights", O, torch.float32, tokens * k)
    dO = _gradient(dO, O, (rows, width), stream)
    dweights = _gradient(dweights, O, (tokens, k), stream, torch.float32)
    do, _, _, lddo = (0, 0, 0, 0) if dO is None else _matrix(dO, "dO", O, (rows, width))
    dw = 0 if dweights is None else _vector(dweights, "dweights", O, torch.float32, tokens * k)
    _launch("moe_combine_backward", O, stream, dtype, tokens, k, width, dy, lddy, o, rows, ldo, s,
            w, do, lddo, dw)
    return dO, dweights
