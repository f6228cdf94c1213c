"""Python binding of the gfx950 skinny-GEMM C ABI (include/skinny_gemm.h).

Argument marshalling only: every step of y = x . W^T runs in the HIP kernels
of ``libskinny_gemm.so``.  PyTorch supplies device memory (``data_ptr()``)
and streams (``torch.cuda.current_stream().cuda_stream``).  There is no
fallback: if the shared library is missing or fails to load, every entry
point raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

__all__ = [
    "BF16", "FP8_BS128", "VARIANT_AUTO", "VARIANT_VECTOR", "VARIANT_MFMA", "MAX_M",
    "SkinnyError", "Linear", "Plan", "lib", "lib_path",
    "workspace_bytes", "stack_workspace_bytes", "skinny_gemm_bf16", "skinny_gemm_fp8_bs128",
    "decode_linear_stack", "decode_linear_stack_noalloc", "STATIC_SCRATCH_BYTES", "linear_run", "linear_run_timed", "launch_count", "band_rows", "plan_query",
    "status_string", "abi_version", "argmax_bf16", "argmax_workspace_bytes", "lm_head_argmax",
    "lm_head_workspace_bytes", "Mlp", "make_mlp", "mlp_workspace_bytes", "mlp_swiglu",
    "Experts", "make_experts", "moe_workspace_bytes", "moe_linear", "moe_linear_timed",
    "moe_plan_query", "moe_mlp_workspace_bytes", "moe_mlp_swiglu", "moe_mlp_swiglu_timed",
    "moe_mlp_set_spin_limit", "moe_mlp_gave_up", "moe_mlp_plan_query", "MOE_MLP_COUNTER_BYTES",
    "MOE_X_PER_ROUTE", "MOE_SWIGLU", "MAX_TOPK", "KERNEL_NAMES",
    "KV_BF16", "KV_FP8", "KvCache", "KvBatch", "make_kv_cache", "make_batch", "kv_append",
    "kv_attention", "kv_attention_workspace_bytes", "LOGITS_BF16", "LOGITS_F32", "Verify",
    "verify_draft", "verify_workspace_bytes", "verify_set_spin_limit",
    "VALUES_BF16", "VALUES_F32", "NORM_RMS", "NORM_LAYER", "Norm", "block_norm", "Lora", "make_lora",
    "lora_workspace_bytes", "lora_linear", "ROUTE_SOFTMAX", "ROUTE_SIGMOID", "Route", "moe_route",
]

BF16 = 0
FP8_BS128 = 1
VARIANT_AUTO = 0
VARIANT_VECTOR = 1
VARIANT_MFMA = 2
MAX_M = 16
MAX_LINEARS_PER_LAUNCH = 32    # descriptors in a launch's arguments; more go in a table
MAX_TOPK = 16
MOE_X_PER_ROUTE = 1
MOE_SWIGLU = 2
ABI_VERSION = 2
# enum skinny_kernel (skinny_plan.kernel): the main kernel's form, by the name
# of its HIP function (and instance).
KERNEL_NAMES = {1: "skinny_rows", 2: "skinny_rows (lean)", 3: "skinny_rows_flat",
                4: "skinny_tiles", 5: "skinny_tiles (8-wave)", 6: "skinny_tiles (K-split)",
                7: "skinny_moe_mlp1"}
STATIC_SCRATCH_BYTES = 64 << 20
LOGITS_BF16 = 0
LOGITS_F32 = 1
KV_BF16 = 0
KV_FP8 = 1
VALUES_BF16 = 0
VALUES_F32 = 1
NORM_RMS = 0
NORM_LAYER = 1
ROUTE_SOFTMAX = 0
ROUTE_SIGMOID = 1
MAX_LORA_SLICES = 4
MOE_MLP_COUNTER_BYTES = 256   # moe_mlp_swiglu's workspace: counter and flag, then gate_up outputs

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libskinny_gemm.so"

STATUS_NAMES = {0: "SKINNY_OK", 1: "SKINNY_ERR_INVALID_ARG", 2: "SKINNY_ERR_UNSUPPORTED",
                3: "SKINNY_ERR_WORKSPACE", 4: "SKINNY_ERR_HIP"}


class SkinnyError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


class Linear(ctypes.Structure):
    """struct skinny_linear"""
    _fields_ = [("dtype", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("reserved", ctypes.c_int), ("w", ctypes.c_void_p), ("w_scale", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p)]


class Mlp(ctypes.Structure):
    """struct skinny_mlp"""
    _fields_ = [("dtype", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int),
                ("reserved", ctypes.c_int), ("w_gate_up", ctypes.c_void_p),
                ("s_gate_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
                ("s_down", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p)]


class Experts(ctypes.Structure):
    """struct skinny_experts"""
    _fields_ = [("dtype", ctypes.c_int), ("E", ctypes.c_int), ("N", ctypes.c_int),
                ("K", ctypes.c_int), ("w", ctypes.c_void_p), ("w_scale", ctypes.c_void_p)]


class KvCache(ctypes.Structure):
    """struct skinny_kv_cache"""
    _fields_ = [("dtype", ctypes.c_int), ("pages", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("reserved", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]
    gpu = None                 # of the tensors that make_kv_cache was given


class KvBatch(ctypes.Structure):
    """struct skinny_kv_batch"""
    _fields_ = [("seqs", ctypes.c_int), ("tokens", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("reserved", ctypes.c_int), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p)]
    gpu = None                 # of the tensors that make_batch was given


class Verify(ctypes.Structure):
    """struct skinny_verify"""
    _fields_ = [("dtype", ctypes.c_int), ("vocab", ctypes.c_int), ("rows", ctypes.c_int),
                ("seqs", ctypes.c_int), ("q_start", ctypes.c_void_p), ("logits", ctypes.c_void_p),
                ("draft_logits", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
                ("temperature", ctypes.c_void_p), ("accept_u", ctypes.c_void_p),
                ("sample_u", ctypes.c_void_p), ("out_tokens", ctypes.c_void_p),
                ("accepted", ctypes.c_void_p)]


class Norm(ctypes.Structure):
    """struct skinny_norm"""
    _fields_ = [(n, ctypes.c_int) for n in ("kind", "rows", "width", "routes", "residual_dtype",
                                            "weight_dtype", "gate_rows", "reserved")] + \
               [(n, ctypes.c_float) for n in ("eps", "residual_scale", "block_scale",
                                              "weight_offset")] + \
               [(n, ctypes.c_void_p) for n in ("block", "route_weights", "post_weight", "post_bias",
                                               "gate", "residual", "residual_out", "weight", "bias",
                                               "out")]


class Lora(ctypes.Structure):
    """struct skinny_lora"""
    _fields_ = [("adapters", ctypes.c_int), ("rank", ctypes.c_int), ("K", ctypes.c_int),
                ("slices", ctypes.c_int), ("n", ctypes.c_int * MAX_LORA_SLICES),
                ("a", ctypes.c_void_p * MAX_LORA_SLICES), ("b", ctypes.c_void_p * MAX_LORA_SLICES),
                ("ranks", ctypes.c_void_p), ("scale", ctypes.c_void_p)]
    gpu = None                 # of the tensors that make_lora was given
    width = None               # of y, as make_lora summed it


class Route(ctypes.Structure):
    """struct skinny_route"""
    _fields_ = [(n, ctypes.c_int) for n in ("dtype", "scoring", "rows", "experts", "topk", "groups",
                                            "top_groups", "renormalize")] + \
               [("scale", ctypes.c_float), ("reserved", ctypes.c_int)] + \
               [(n, ctypes.c_void_p) for n in ("logits", "bias", "ids", "weights")]


class Plan(ctypes.Structure):
    """struct skinny_plan"""
    _fields_ = [("variant", ctypes.c_int), ("waves", ctypes.c_int), ("kernel", ctypes.c_int),
                ("reserved", ctypes.c_int * 5)]


_lib = None


def lib_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def _bind(path: str):
    """Load a built library and declare the C signatures of include/skinny_gemm.h."""
    L = ctypes.CDLL(path)
    sz, vp, i = ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
    lp = ctypes.POINTER(Linear)
    L.skinny_workspace_bytes.restype = sz
    L.skinny_workspace_bytes.argtypes = [i, i, i, i]
    L.skinny_stack_workspace_bytes.restype = sz
    L.skinny_stack_workspace_bytes.argtypes = [lp, i, i]
    L.skinny_gemm_bf16.restype = i
    L.skinny_gemm_bf16.argtypes = [vp, vp, vp, i, i, i, vp, sz, vp]
    L.skinny_gemm_fp8_bs128.restype = i
    L.skinny_gemm_fp8_bs128.argtypes = [vp, vp, vp, vp, i, i, i, vp, sz, vp]
    L.decode_linear_stack.restype = i
    L.decode_linear_stack.argtypes = [lp, i, i, vp, sz, vp]
    L.decode_linear_stack_noalloc.restype = i
    L.decode_linear_stack_noalloc.argtypes = [lp, i, i, vp]
    L.skinny_linear_run.restype = i
    L.skinny_linear_run.argtypes = [lp, i, i, ctypes.POINTER(Plan), vp, sz, vp]
    L.skinny_launch_count.restype = i
    L.skinny_launch_count.argtypes = [lp, i]
    L.skinny_linear_run_timed.restype = i
    L.skinny_linear_run_timed.argtypes = [lp, i, i, ctypes.POINTER(Plan),
                                          ctypes.POINTER(ctypes.c_void_p), i, vp, sz, vp]
    L.skinny_band_rows.restype = i
    L.skinny_band_rows.argtypes = [i, i, i]
    L.skinny_plan_query.restype = i
    L.skinny_plan_query.argtypes = [lp, i, i, ctypes.POINTER(Plan)]
    L.skinny_argmax_workspace_bytes.restype = sz
    L.skinny_argmax_workspace_bytes.argtypes = [i, i]
    L.skinny_argmax_bf16.restype = i
    L.skinny_argmax_bf16.argtypes = [vp, i, i, vp, vp, sz, vp]
    L.skinny_lm_head_workspace_bytes.restype = sz
    L.skinny_lm_head_workspace_bytes.argtypes = [lp, i]
    L.skinny_lm_head_argmax.restype = i
    L.skinny_lm_head_argmax.argtypes = [lp, i, vp, vp, sz, vp]
    mp = ctypes.POINTER(Mlp)
    L.skinny_mlp_workspace_bytes.restype = sz
    L.skinny_mlp_workspace_bytes.argtypes = [mp, i]
    L.skinny_mlp_swiglu.restype = i
    L.skinny_mlp_swiglu.argtypes = [mp, i, vp, sz, vp]
    ep = ctypes.POINTER(Experts)
    L.skinny_moe_workspace_bytes.restype = sz
    L.skinny_moe_workspace_bytes.argtypes = [ep, i, i, i]
    L.skinny_moe_linear.restype = i
    L.skinny_moe_linear.argtypes = [ep, vp, vp, i, i, i, vp, vp, sz, vp]
    L.skinny_moe_linear_timed.restype = i
    L.skinny_moe_linear_timed.argtypes = [ep, vp, vp, i, i, i, vp, ctypes.POINTER(vp), vp, sz, vp]
    L.skinny_moe_plan_query.restype = i
    L.skinny_moe_plan_query.argtypes = [ep, i, i, i, ctypes.POINTER(Plan)]
    L.skinny_moe_mlp_workspace_bytes.restype = sz
    L.skinny_moe_mlp_workspace_bytes.argtypes = [ep, ep, i, i]
    L.skinny_moe_mlp_swiglu.restype = i
    L.skinny_moe_mlp_swiglu.argtypes = [ep, ep, vp, vp, i, i, vp, vp, sz, vp]
    L.skinny_moe_mlp_swiglu_timed.restype = i
    L.skinny_moe_mlp_swiglu_timed.argtypes = [ep, ep, vp, vp, i, i, vp, ctypes.POINTER(vp), vp,
                                              sz, vp]
    L.skinny_moe_mlp_plan_query.restype = i
    L.skinny_moe_mlp_plan_query.argtypes = [ep, ep, i, i, ctypes.POINTER(Plan)]
    L.skinny_moe_mlp_set_spin_limit.restype = None
    L.skinny_moe_mlp_set_spin_limit.argtypes = [ctypes.c_longlong]
    cp, bp = ctypes.POINTER(KvCache), ctypes.POINTER(KvBatch)
    L.skinny_kv_append.restype = i
    L.skinny_kv_append.argtypes = [cp, bp, vp, i, vp, i, i, vp, vp]
    L.skinny_kv_attention_workspace_bytes.restype = sz
    L.skinny_kv_attention_workspace_bytes.argtypes = [cp, bp, i]
    L.skinny_kv_attention.restype = i
    L.skinny_kv_attention.argtypes = [cp, bp, vp, i, ctypes.c_float, vp, vp, sz, vp]
    L.skinny_verify_workspace_bytes.restype = sz
    L.skinny_verify_workspace_bytes.argtypes = [i, i, i]
    L.skinny_verify_draft.restype = i
    L.skinny_verify_draft.argtypes = [ctypes.POINTER(Verify), vp, sz, vp]
    L.skinny_verify_set_spin_limit.restype = None
    L.skinny_verify_set_spin_limit.argtypes = [ctypes.c_longlong]
    L.skinny_block_norm.restype = i
    L.skinny_block_norm.argtypes = [ctypes.POINTER(Norm), vp]
    L.skinny_lora_workspace_bytes.restype = sz
    L.skinny_lora_workspace_bytes.argtypes = [ctypes.POINTER(Lora), i]
    L.skinny_lora_linear.restype = i
    L.skinny_lora_linear.argtypes = [ctypes.POINTER(Lora), vp, vp, i, vp, vp, vp, sz, vp]
    L.skinny_moe_route.restype = i
    L.skinny_moe_route.argtypes = [ctypes.POINTER(Route), vp]
    # The same entry points for structures packed as bytes.
    L.norm_of_bytes, L.route_of_bytes = L["skinny_block_norm"], L["skinny_moe_route"]
    for f in (L.norm_of_bytes, L.route_of_bytes):
        f.restype = i
        f.argtypes = [ctypes.c_char_p, vp]
    L.skinny_status_string.restype = ctypes.c_char_p
    L.skinny_status_string.argtypes = [i]
    L.skinny_abi_version.restype = i
    L.skinny_abi_version.argtypes = []
    if L.skinny_abi_version() != ABI_VERSION:
        raise ImportError(f"{path}: ABI version {L.skinny_abi_version()} != {ABI_VERSION}")
    return L


def lib():
    """The loaded C library.  Raises if it is not built: there is no fallback."""
    global _lib
    if _lib is None:
        path = lib_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is not built; run __graft_entry__.build() or "
                              "python -m gemv_skinny_gemm_amd._build")
        _lib = _bind(path)
    return _lib


def _ptr(t) -> int | None:
    """Device address of a torch tensor, or an int address as given (None = NULL).
    The library reads and writes dense row-major device memory, so a tensor must
    be contiguous and on the GPU."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous (row-major)")
    if t.device.type != "cuda":
        raise ValueError(f"tensors passed to the library must be on the GPU, not {t.device}")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != 0:
        raise SkinnyError(status, where)


def status_string(status: int) -> str:
    return lib().skinny_status_string(int(status)).decode()


def abi_version() -> int:
    return lib().skinny_abi_version()


def workspace_bytes(dtype: int, M: int, N: int, K: int) -> int:
    return lib().skinny_workspace_bytes(dtype, M, N, K)


def _linear_array(linears):
    arr = (Linear * len(linears))()
    for i, L in enumerate(linears):
        arr[i] = L
    return arr


def stack_workspace_bytes(linears, M: int) -> int:
    arr = _linear_array(linears)
    return lib().skinny_stack_workspace_bytes(arr, len(linears), M)


def _shape2(t):
    if isinstance(t, int):
        raise TypeError("pass tensors, or call the raw C entry points through lib()")
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    return int(t.shape[0]), int(t.shape[1])


def _dtype_name(t) -> str:
    return str(t.dtype).replace("torch.", "")


def _need(t, shape, dtypes, what):
    """Refuse a tensor whose shape or dtype does not match what the C entry
    point will read or write: the library sees only pointers, so a short or
    mistyped buffer would be read or written past its end."""
    if isinstance(t, int) or t is None:
        return
    if tuple(int(v) for v in t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if _dtype_name(t) not in dtypes:
        raise ValueError(f"{what}: dtype {_dtype_name(t)}, expected one of {sorted(dtypes)}")


_BF16 = {"bfloat16"}
_FP8 = {"uint8", "float8_e4m3fn"}
_F32 = {"float32"}
_I32 = {"int32"}


def _scale_shape(N: int, K: int):
    return ((N + 127) // 128, (K + 127) // 128)


def _ws(workspace):
    if workspace is None:
        return None, 0
    if isinstance(workspace, tuple):
        return workspace
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def skinny_gemm_bf16(x, w, y, workspace, stream=None):
    """y[M][N] = x[M][K] . w[N][K]^T (bf16 tensors on the GPU; y written in place)."""
    M, K = _shape2(x)
    N, _ = _shape2(w)
    _need(x, (M, K), _BF16, "x")
    _need(w, (N, K), _BF16, "w")
    _need(y, (M, N), _BF16, "y")
    wp, wb = _ws(workspace)
    _check(lib().skinny_gemm_bf16(_ptr(x), _ptr(w), _ptr(y), M, N, K, wp, wb, _stream(stream)),
           "skinny_gemm_bf16")
    return y


def skinny_gemm_fp8_bs128(x, w_fp8, w_scale, y, workspace, stream=None):
    """y = x . (e4m3(w_fp8) * block scale)^T; w_fp8 [N][K] uint8 / float8_e4m3fn,
    w_scale [ceil(N/128)][ceil(K/128)] float32."""
    M, K = _shape2(x)
    N, _ = _shape2(w_fp8)
    _need(x, (M, K), _BF16, "x")
    _need(w_fp8, (N, K), _FP8, "w_fp8")
    _need(w_scale, _scale_shape(N, K), _F32, "w_scale")
    _need(y, (M, N), _BF16, "y")
    wp, wb = _ws(workspace)
    _check(lib().skinny_gemm_fp8_bs128(_ptr(x), _ptr(w_fp8), _ptr(w_scale), _ptr(y), M, N, K,
                                        wp, wb, _stream(stream)), "skinny_gemm_fp8_bs128")
    return y


def make_linear(x, w, y, w_scale=None, dtype=None) -> Linear:
    """A skinny_linear from GPU tensors x [M][K], w [N][K], y [M][N] (w_scale for FP8).

    Shapes and dtypes are checked here; the Linear remembers M (as ``rows``)
    so that a call with another M is refused before it reaches the library."""
    N, K = _shape2(w)
    if dtype is None:
        dtype = FP8_BS128 if w_scale is not None else BF16
    M = None
    if not isinstance(x, int):
        M, _ = _shape2(x)
        _need(x, (M, K), _BF16, "x")
        _need(y, (M, N), _BF16, "y")
    _need(w, (N, K), _BF16 if dtype == BF16 else _FP8, "w")
    if dtype == FP8_BS128:
        _need(w_scale, _scale_shape(N, K), _F32, "w_scale")
    lin = Linear(dtype, N, K, 0, _ptr(w), _ptr(w_scale), _ptr(x), _ptr(y))
    lin.rows = M
    return lin


def _check_rows(linears, M: int):
    for L in linears:
        rows = getattr(L, "rows", None)
        if rows is not None and rows != M:
            raise ValueError(f"a linear made for M = {rows} called with M = {M}")


def decode_linear_stack(linears, M: int, workspace, stream=None):
    """Run independent linears (a list of Linear) that share M."""
    _check_rows(linears, M)
    arr = _linear_array(linears)
    wp, wb = _ws(workspace)
    _check(lib().decode_linear_stack(arr, len(linears), M, wp, wb, _stream(stream)),
           "decode_linear_stack")


def decode_linear_stack_noalloc(linears, M: int, stream=None):
    """decode_linear_stack without a workspace: the partial sums go to the
    library's static device buffer (STATIC_SCRATCH_BYTES per GPU), shared by
    every call on that GPU, so calls that may overlap on one GPU race."""
    _check_rows(linears, M)
    arr = _linear_array(linears)
    _check(lib().decode_linear_stack_noalloc(arr, len(linears), M, _stream(stream)),
           "decode_linear_stack_noalloc")


def linear_run(linears, M: int, workspace, variant: int = VARIANT_AUTO, waves: int = 0,
               stream=None):
    """decode_linear_stack with a forced variant and/or persistent wave count."""
    _check_rows(linears, M)
    arr = _linear_array(linears)
    plan = Plan(variant, waves)
    wp, wb = _ws(workspace)
    _check(lib().skinny_linear_run(arr, len(linears), M, ctypes.byref(plan), wp, wb,
                                   _stream(stream)), "skinny_linear_run")


def band_rows(dtype: int, variant: int, M: int) -> int:
    """Rows per band of the main kernel: the workspace slot layout is [slot][M][band_rows]."""
    return lib().skinny_band_rows(dtype, variant, M)


def launch_count(linears) -> int:
    arr = _linear_array(linears)
    return lib().skinny_launch_count(arr, len(linears))


def linear_run_timed(linears, M: int, workspace, events, variant: int = VARIANT_AUTO,
                     waves: int = 0, stream=None):
    """linear_run recording events[2g] / events[2g+1] (hipEvent_t addresses) around
    main-kernel launch g."""
    _check_rows(linears, M)
    arr = _linear_array(linears)
    plan = Plan(variant, waves)
    ev = (ctypes.c_void_p * len(events))(*events)
    wp, wb = _ws(workspace)
    _check(lib().skinny_linear_run_timed(arr, len(linears), M, ctypes.byref(plan), ev, len(events),
                                         wp, wb, _stream(stream)), "skinny_linear_run_timed")


def plan_query(linears, M: int) -> Plan:
    arr = _linear_array(linears)
    plan = Plan()
    _check(lib().skinny_plan_query(arr, len(linears), M, ctypes.byref(plan)), "skinny_plan_query")
    return plan


def argmax_workspace_bytes(M: int, N: int) -> int:
    return lib().skinny_argmax_workspace_bytes(M, N)


def argmax_bf16(y, idx, workspace, stream=None):
    """idx[m] = smallest index of the largest value of y[m] (bf16 [M][N] and
    int32 [M] tensors on the GPU; idx written in place)."""
    M, N = _shape2(y)
    _need(y, (M, N), _BF16, "y")
    _need(idx, (M,), _I32, "idx")
    wp, wb = _ws(workspace)
    _check(lib().skinny_argmax_bf16(_ptr(y), M, N, _ptr(idx), wp, wb, _stream(stream)),
           "skinny_argmax_bf16")
    return idx


def lm_head_workspace_bytes(head: Linear, M: int) -> int:
    return lib().skinny_lm_head_workspace_bytes(_linear_array([head]), M)


def lm_head_argmax(head: Linear, M: int, next_token, workspace, stream=None):
    """Run the vocabulary projection `head` (its y = logits) and write the
    greedy token of each of the M rows into next_token (int32 [M] on the GPU)."""
    _check_rows([head], M)
    _need(next_token, (M,), _I32, "next_token")
    arr = _linear_array([head])
    wp, wb = _ws(workspace)
    _check(lib().skinny_lm_head_argmax(arr, M, _ptr(next_token), wp, wb, _stream(stream)),
           "skinny_lm_head_argmax")
    return next_token


def make_mlp(x, w_gate_up, w_down, y, s_gate_up=None, s_down=None) -> Mlp:
    """A skinny_mlp from GPU tensors x [M][H], w_gate_up [2I][H] (gate rows
    first), w_down [H][I], y [M][H] (scales for FP8)."""
    H, I = _shape2(w_down)
    dtype = FP8_BS128 if s_gate_up is not None else BF16
    wd = _BF16 if dtype == BF16 else _FP8
    _need(w_gate_up, (2 * I, H), wd, "w_gate_up")
    _need(w_down, (H, I), wd, "w_down")
    if dtype == FP8_BS128:
        _need(s_gate_up, _scale_shape(2 * I, H), _F32, "s_gate_up")
        _need(s_down, _scale_shape(H, I), _F32, "s_down")
    M = None
    if not isinstance(x, int):
        M, _ = _shape2(x)
        _need(x, (M, H), _BF16, "x")
        _need(y, (M, H), _BF16, "y")
    mlp = Mlp(dtype, H, I, 0, _ptr(w_gate_up), _ptr(s_gate_up), _ptr(w_down), _ptr(s_down),
              _ptr(x), _ptr(y))
    mlp.rows = M
    return mlp


def mlp_workspace_bytes(mlp: Mlp, M: int) -> int:
    return lib().skinny_mlp_workspace_bytes(ctypes.byref(mlp), M)


def mlp_swiglu(mlp: Mlp, M: int, workspace, stream=None):
    """y = down(silu(gate) * up) with [gate | up] = x . W_gate_up^T."""
    _check_rows([mlp], M)
    wp, wb = _ws(workspace)
    _check(lib().skinny_mlp_swiglu(ctypes.byref(mlp), M, wp, wb, _stream(stream)),
           "skinny_mlp_swiglu")


def make_experts(w, w_scale=None) -> Experts:
    """A skinny_experts from GPU tensors w [E][N][K] (bf16, or uint8 E4M3FN
    codes with w_scale [E][ceil(N/128)][ceil(K/128)] fp32)."""
    if isinstance(w, int) or w.dim() != 3:
        raise ValueError("w must be a 3-D tensor [E][N][K]")
    E, N, K = (int(v) for v in w.shape)
    _need(w, (E, N, K), _BF16 if w_scale is None else _FP8, "w")
    if w_scale is not None:
        _need(w_scale, (E, *_scale_shape(N, K)), _F32, "w_scale")
    return Experts(FP8_BS128 if w_scale is not None else BF16, E, N, K, _ptr(w), _ptr(w_scale))


def _moe_flags(x_per_route: bool, swiglu: bool) -> int:
    return (MOE_X_PER_ROUTE if x_per_route else 0) | (MOE_SWIGLU if swiglu else 0)


def _check_moe(experts: Experts, x, ids, y, x_per_route: bool, swiglu: bool):
    T, topk = _shape2(ids)
    _need(ids, (T, topk), _I32, "ids")
    _need(x, ((T * topk if x_per_route else T), (2 if swiglu else 1) * experts.K), _BF16, "x")
    _need(y, (T * topk, experts.N), _BF16, "y")
    return T, topk


def moe_workspace_bytes(experts: Experts, T: int, topk: int, x_per_route: bool = False,
                        swiglu: bool = False) -> int:
    return lib().skinny_moe_workspace_bytes(ctypes.byref(experts), T, topk,
                                            _moe_flags(x_per_route, swiglu))


def moe_linear(experts: Experts, x, ids, y, workspace, x_per_route: bool = False,
               swiglu: bool = False, stream=None):
    """y[t * topk + j] = x_r . W_{ids[t][j]}^T for the T x topk routes of ids
    (int32 [T][topk] on the GPU); x_r = x[t], or x[r] with x_per_route, or
    silu(g) * u of that row [g | u] with swiglu."""
    T, topk = _check_moe(experts, x, ids, y, x_per_route, swiglu)
    wp, wb = _ws(workspace)
    _check(lib().skinny_moe_linear(ctypes.byref(experts), _ptr(x), _ptr(ids), T, topk,
                                   _moe_flags(x_per_route, swiglu), _ptr(y), wp, wb,
                                   _stream(stream)), "skinny_moe_linear")
    return y


def moe_linear_timed(experts: Experts, x, ids, y, workspace, events, x_per_route: bool = False,
                     swiglu: bool = False, stream=None):
    """moe_linear recording the two hipEvent_t handles in `events` around its
    main launch."""
    T, topk = _check_moe(experts, x, ids, y, x_per_route, swiglu)
    wp, wb = _ws(workspace)
    ev = (ctypes.c_void_p * 2)(*events)
    _check(lib().skinny_moe_linear_timed(ctypes.byref(experts), _ptr(x), _ptr(ids), T, topk,
                                         _moe_flags(x_per_route, swiglu), _ptr(y), ev, wp, wb,
                                         _stream(stream)), "skinny_moe_linear_timed")
    return y


def _check_moe_mlp(gate_up: Experts, down: Experts, x, ids, y):
    T, topk = _shape2(ids)
    _need(ids, (T, topk), _I32, "ids")
    _need(x, (T, gate_up.K), _BF16, "x")
    _need(y, (T * topk, down.N), _BF16, "y")
    return T, topk


def moe_mlp_workspace_bytes(gate_up: Experts, down: Experts, T: int, topk: int) -> int:
    """Bytes of workspace moe_mlp_swiglu needs; allocate it zeroed (its first
    256 bytes are counters that must start at zero)."""
    return lib().skinny_moe_mlp_workspace_bytes(ctypes.byref(gate_up), ctypes.byref(down), T,
                                                topk)


def moe_mlp_swiglu(gate_up: Experts, down: Experts, x, ids, y, workspace, stream=None):
    """y[r] = bf16(silu(g) * u) . Wdown_e^T with [g | u] = x[t] . Wgate_up_e^T
    (bf16) for route r = t * topk + j, e = ids[t][j]; one launch for one token."""
    T, topk = _check_moe_mlp(gate_up, down, x, ids, y)
    wp, wb = _ws(workspace)
    _check(lib().skinny_moe_mlp_swiglu(ctypes.byref(gate_up), ctypes.byref(down), _ptr(x),
                                       _ptr(ids), T, topk, _ptr(y), wp, wb, _stream(stream)),
           "skinny_moe_mlp_swiglu")
    return y


def moe_mlp_swiglu_timed(gate_up: Experts, down: Experts, x, ids, y, workspace, events,
                         stream=None):
    """moe_mlp_swiglu recording the two hipEvent_t handles in `events` around
    its main launch (the one launch for one token, else gate_up's)."""
    T, topk = _check_moe_mlp(gate_up, down, x, ids, y)
    wp, wb = _ws(workspace)
    ev = (ctypes.c_void_p * 2)(*events)
    _check(lib().skinny_moe_mlp_swiglu_timed(ctypes.byref(gate_up), ctypes.byref(down), _ptr(x),
                                             _ptr(ids), T, topk, _ptr(y), ev, wp, wb,
                                             _stream(stream)), "skinny_moe_mlp_swiglu_timed")
    return y


def moe_mlp_plan_query(gate_up: Experts, down: Experts, T: int, topk: int) -> Plan:
    """The main launch moe_mlp_swiglu makes (kernel 7 = the one launch)."""
    plan = Plan()
    _check(lib().skinny_moe_mlp_plan_query(ctypes.byref(gate_up), ctypes.byref(down), T, topk,
                                           ctypes.byref(plan)), "skinny_moe_mlp_plan_query")
    return plan


def moe_mlp_set_spin_limit(polls: int) -> None:
    """Polls before the one-token launch's wait gives up (< 0: it does not
    wait); for tests of that path."""
    lib().skinny_moe_mlp_set_spin_limit(int(polls))


def moe_mlp_gave_up(workspace) -> bool:
    """Whether a wait of the one-token launch on this workspace gave up (its
    counter word 2; synchronizes with the device)."""
    import torch
    return bool(int(workspace[:16].view(torch.int32)[2].item()))


def moe_plan_query(experts: Experts, T: int, topk: int, x_per_route: bool = False,
                   swiglu: bool = False) -> Plan:
    """The main kernel moe_linear takes for these experts and T x topk routes
    (variant VARIANT_VECTOR or VARIANT_MFMA)."""
    plan = Plan()
    _check(lib().skinny_moe_plan_query(ctypes.byref(experts), T, topk,
                                       _moe_flags(x_per_route, swiglu), ctypes.byref(plan)),
           "skinny_moe_plan_query")
    return plan


class _Torch:
    """What the calls below ask torch for each time, looked up once."""

    def __init__(self):
        import torch
        self.bf16, self.f32, self.i32 = torch.bfloat16, torch.float32, torch.int32
        self.device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        # The stream's handle without a Stream object around it (a microsecond
        # of the host's time per call), where this torch has that.
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_torch = None


def _operand(t, shape, dtype, what, dev):
    """Device address of a tensor after the checks of _need and _ptr (which
    name what is wrong), and that it lies on GPU `dev`."""
    if t.shape != shape or t.dtype is not dtype:
        _need(t, shape, {str(dtype).replace("torch.", "")}, what)
    if not t.is_contiguous() or t.get_device() != dev:
        _ptr(t)
        raise ValueError(f"{what} is on {t.device}, the call's other tensors on GPU {dev}")
    return t.data_ptr()


def _call_device(t):
    """GPU of a call's tensors, which has to be the current one: the library
    launches there, on that device's current stream."""
    global _torch
    if _torch is None:
        _torch = _Torch()
    dev = t.get_device()
    if dev >= 0 and dev != _torch.device():
        raise ValueError(f"tensors on {t.device}, but the current device is GPU {_torch.device()}")
    return _torch, dev


def _call_stream(tt, dev, stream, cache=None, batch=None):
    if dev < 0:
        raise ValueError("tensors passed to the library must be on the GPU, not cpu")
    if cache is not None and (cache.gpu not in (None, dev) or batch.gpu not in (None, dev)):
        raise ValueError(f"cache on GPU {cache.gpu} and batch on GPU {batch.gpu}, the call's "
                         f"tensors on GPU {dev}")
    return tt.raw_stream(dev) if stream is None else _stream(stream)


def _space(workspace, dev):
    """A call's workspace as the library takes it, on the call's GPU."""
    if workspace is None or isinstance(workspace, tuple):
        return _ws(workspace)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _ptr(workspace)
        raise ValueError(f"workspace is on {workspace.device}, the call's other tensors on GPU {dev}")
    return workspace.data_ptr(), workspace.nbytes


def _one_gpu(struct, *tensors):
    """`struct` with the tensors' GPU and the tensors, whose memory it points to."""
    struct.gpu = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != struct.gpu:
            raise ValueError(f"tensors on {tensors[0].device} and on {t.device}")
    struct.tensors = tensors
    return struct


def make_kv_cache(k, v, k_scale=None, v_scale=None) -> KvCache:
    """A skinny_kv_cache from GPU tensors k and v [pages][kv_heads][page_tokens]
    [head_dim]: bf16, or e4m3 codes (uint8 / float8_e4m3fn) with k_scale and
    v_scale [pages][kv_heads] float32."""
    if isinstance(k, int) or k.dim() != 4:
        raise ValueError("k must be a 4-D tensor [pages][kv_heads][page_tokens][head_dim]")
    shape = tuple(int(n) for n in k.shape)
    if (k_scale is None) != (v_scale is None):
        raise ValueError("k_scale and v_scale come together")
    fp8 = k_scale is not None
    for t, what in ((k, "k"), (v, "v")):
        _need(t, shape, _FP8 if fp8 else _BF16, what)
    if fp8:
        _need(k_scale, shape[:2], _F32, "k_scale")
        _need(v_scale, shape[:2], _F32, "v_scale")
    return _one_gpu(KvCache(KV_FP8 if fp8 else KV_BF16, *shape, 0, _ptr(k), _ptr(v),
                            _ptr(k_scale), _ptr(v_scale)),
                    *((k, v, k_scale, v_scale) if fp8 else (k, v)))


def make_batch(q_start, kv_len, page_table, tokens: int) -> KvBatch:
    """A skinny_kv_batch from int32 GPU tensors q_start [seqs + 1], kv_len [seqs]
    and page_table [seqs][max_pages], for steps of `tokens` rows.  The tensors
    may change between calls (their values are read on the device)."""
    if isinstance(page_table, int):
        raise TypeError("pass tensors, or call the raw C entry points through lib()")
    seqs, width = _shape2(page_table)
    _need(q_start, (seqs + 1,), _I32, "q_start")
    _need(kv_len, (seqs,), _I32, "kv_len")
    _need(page_table, (seqs, width), _I32, "page_table")
    return _one_gpu(KvBatch(seqs, int(tokens), width, 0, _ptr(q_start), _ptr(kv_len),
                            _ptr(page_table)), q_start, kv_len, page_table)


def _heads(cache: KvCache, batch: KvBatch, t, what: str, extra: int = 0) -> int:
    """Query heads of a [tokens][(q_heads + extra) * head_dim] tensor."""
    dim = cache.head_dim
    shape = t.shape
    heads = shape[-1] // dim - extra
    if shape != (batch.tokens, (heads + extra) * dim):
        _need(t, (batch.tokens, (heads + extra) * dim), _BF16, what)
    return heads


def kv_append(cache: KvCache, batch: KvBatch, qkv, inv_freq, q_out, interleaved: bool = False,
              stream=None):
    """Write a step's keys and values into the paged cache and its rotated
    queries into q_out [tokens][q_heads * head_dim].  qkv [tokens][(q_heads +
    2 kv_heads) * head_dim] is the QKV linear's y; inv_freq [rotary_dim / 2]
    float32, or None for no rotation."""
    tt, dev = _call_device(qkv)
    heads = _heads(cache, batch, qkv, "qkv", 2 * cache.kv_heads)
    x = _operand(qkv, qkv.shape, tt.bf16, "qkv", dev)
    y = _operand(q_out, (batch.tokens, heads * cache.head_dim), tt.bf16, "q_out", dev)
    rot, f = 0, None
    if inv_freq is not None:
        rot = 2 * inv_freq.shape[0]
        f = _operand(inv_freq, (rot // 2,), tt.f32, "inv_freq", dev)
    _check(lib().skinny_kv_append(cache, batch, x, heads, f, rot, int(interleaved), y,
                                  _call_stream(tt, dev, stream, cache, batch)), "skinny_kv_append")
    return q_out


def kv_attention_workspace_bytes(cache: KvCache, batch: KvBatch, q_heads: int) -> int:
    return lib().skinny_kv_attention_workspace_bytes(cache, batch, q_heads)


def kv_attention(cache: KvCache, batch: KvBatch, q, out, workspace, scale: float | None = None,
                 stream=None):
    """out = softmax(scale q k^T) v over each sequence's cache, causal within
    the step's rows; q and out bf16 [tokens][q_heads * head_dim], scale
    1 / sqrt(head_dim) unless given."""
    tt, dev = _call_device(q)
    heads = _heads(cache, batch, q, "q")
    x = _operand(q, q.shape, tt.bf16, "q", dev)
    y = _operand(out, q.shape, tt.bf16, "out", dev)
    wp, wb = _space(workspace, dev)
    _check(lib().skinny_kv_attention(cache, batch, x, heads,
                                     cache.head_dim ** -0.5 if scale is None else scale, y, wp, wb,
                                     _call_stream(tt, dev, stream, cache, batch)),
           "skinny_kv_attention")
    return out


def verify_workspace_bytes(rows: int, seqs: int, vocab: int) -> int:
    return lib().skinny_verify_workspace_bytes(rows, seqs, vocab)


def verify_draft(q_start, logits, tokens, accept_u, sample_u, out_tokens, accepted, workspace,
                 draft_logits=None, temperature=None, stream=None):
    """Which drafted tokens the target keeps and the token that follows them.
    logits (and draft_logits) [rows][vocab] bf16 or float32, tokens int32 [rows]
    (the step's input tokens), q_start int32 [seqs + 1], accept_u float32 [rows],
    sample_u and temperature float32 [seqs]; out_tokens int32 [rows] gets each
    sequence's kept drafts, its next token, then -1, and accepted int32 [seqs]
    the number kept (-1 if a wait inside the launch gave up)."""
    tt, dev = _call_device(logits)
    rows, vocab = _shape2(logits)
    seqs = sample_u.shape[0]
    kind = logits.dtype
    if kind is not tt.bf16 and kind is not tt.f32:
        _need(logits, (rows, vocab), _BF16 | _F32, "logits")
    per_row, per_seq, i32, f32 = (rows,), (seqs,), tt.i32, tt.f32
    v = Verify(
        LOGITS_BF16 if kind is tt.bf16 else LOGITS_F32, vocab, rows, seqs,
        _operand(q_start, (seqs + 1,), i32, "q_start", dev),
        _operand(logits, logits.shape, kind, "logits", dev),
        None if draft_logits is None else _operand(draft_logits, (rows, vocab), kind,
                                                   "draft_logits", dev),
        _operand(tokens, per_row, i32, "tokens", dev),
        None if temperature is None else _operand(temperature, per_seq, f32, "temperature", dev),
        _operand(accept_u, per_row, f32, "accept_u", dev),
        _operand(sample_u, per_seq, f32, "sample_u", dev),
        _operand(out_tokens, per_row, i32, "out_tokens", dev),
        _operand(accepted, per_seq, i32, "accepted", dev))
    wp, wb = _space(workspace, dev)
    _check(lib().skinny_verify_draft(v, wp, wb, _call_stream(tt, dev, stream)),
           "skinny_verify_draft")
    return out_tokens


def verify_set_spin_limit(polls: int) -> None:
    """Polls before a sampling sequence's wait for another workgroup's sums gives
    up (< 0: it does not wait); for tests of that path."""
    lib().skinny_verify_set_spin_limit(int(polls))


def _values(t, tt, what) -> int:
    """VALUES_BF16 or VALUES_F32 of a tensor."""
    if t.dtype is tt.bf16:
        return VALUES_BF16
    if t.dtype is not tt.f32:
        _need(t, t.shape, _BF16 | _F32, what)
    return VALUES_F32


# struct skinny_norm and struct skinny_route as bytes: a ctypes structure of as many
# fields takes three times as long to make (2 us of a call's host time).
_NORM = struct.Struct("8i4f10P")
_ROUTE = struct.Struct("8ifi4P")


def block_norm(out, weight, residual=None, block=None, residual_out=None, bias=None,
               post_weight=None, post_bias=None, gate=None, route_weights=None,
               kind: int = NORM_RMS, eps: float = 1e-6, residual_scale: float = 1.0,
               block_scale: float = 1.0, weight_offset: float = 0.0, stream=None):
    """h = residual_scale * residual + block_scale * gate * norm(block) into
    residual_out, and norm(h) * weight + bias into out [rows][width] bf16, the
    next linear's x.  block [rows * routes][width] bf16 is a linear's y, or the
    experts' routes, summed with route_weights float32 [rows][routes]; its norm is
    taken only with a post_weight.  residual and residual_out (which may be the
    same tensor) are bf16 or float32; weights and biases [width], and gate
    [width] or [rows][width], are all bf16 or all float32, weights counting as
    weight_offset + weight.  What is None takes no part; out None only updates
    the residual."""
    first = out if out is not None else residual_out
    if first is None:
        raise ValueError("one of out and residual_out is needed")
    tt, dev = _call_device(first)
    shape = first.shape
    if len(shape) != 2:
        raise ValueError("expected a 2-D tensor")
    rows, width = shape
    rt, routes, gate_rows, wt = VALUES_BF16, 1, 0, None
    y = h = r = b = rw = g = 0
    if out is not None:
        y = _operand(out, shape, tt.bf16, "out", dev)
    if residual is not None:
        rt = _values(residual, tt, "residual")
        h = _operand(residual, shape, residual.dtype, "residual", dev)
    if residual_out is not None:
        kept = residual_out if residual is None else residual
        rt = _values(kept, tt, "residual_out")
        r = _operand(residual_out, shape, kept.dtype, "residual_out", dev)
    if block is not None:
        if route_weights is not None:
            routes = _shape2(route_weights)[1]
            rw = _operand(route_weights, (rows, routes), tt.f32, "route_weights", dev)
        elif block.shape != shape and rows:
            routes = max(1, block.shape[0] // rows)
        b = _operand(block, (rows * routes, width), tt.bf16, "block", dev)
    elif route_weights is not None or gate is not None or post_weight is not None:
        raise ValueError("route_weights, gate and post_weight need a block")
    w = wb = pw = pb = 0
    if weight is not None:
        wt = weight.dtype
        w = _operand(weight, (width,), wt, "weight", dev)
    if bias is not None:
        wt = wt or bias.dtype
        wb = _operand(bias, (width,), wt, "bias", dev)
    if post_weight is not None:
        wt = wt or post_weight.dtype
        pw = _operand(post_weight, (width,), wt, "post_weight", dev)
    if post_bias is not None:
        wt = wt or post_bias.dtype
        pb = _operand(post_bias, (width,), wt, "post_bias", dev)
    if gate is not None:
        wt = wt or gate.dtype
        gate_rows = int(gate.dim() == 2)
        g = _operand(gate, shape if gate_rows else (width,), wt, "gate", dev)
    if wt is not None and wt is not tt.bf16 and wt is not tt.f32:
        raise ValueError(f"weights, biases and gate: dtype {str(wt).replace('torch.', '')}, expected "
                         "bfloat16 or float32")
    n = _NORM.pack(kind, rows, width, routes, rt, VALUES_F32 if wt is tt.f32 else VALUES_BF16,
                   gate_rows, 0, eps, residual_scale, block_scale, weight_offset, b, rw, pw, pb, g,
                   h, r, w, wb, y)
    _check(lib().norm_of_bytes(n, _call_stream(tt, dev, stream)), "skinny_block_norm")
    return first


def make_lora(a, b, scale=None, ranks=None) -> Lora:
    """A skinny_lora from lists of GPU tensors a [adapters][rank][K] and b
    [adapters][n][rank], bf16, one of each per slice of the projection (or one
    tensor each for a projection of one); a slice without adapters has None in a
    and its width in b.  scale float32 and ranks int32 [adapters]."""
    a, b = ([t] if not isinstance(t, (list, tuple)) else list(t) for t in (a, b))
    if len(a) != len(b) or not 1 <= len(a) <= MAX_LORA_SLICES:
        raise ValueError(f"a and b need the same number of slices, 1 to {MAX_LORA_SLICES}")
    used = [t for t in a if t is not None]
    if not used or any(t.dim() != 3 for t in used):
        raise ValueError("a must be 3-D tensors [adapters][rank][K], and one at least")
    E, R, K = (int(v) for v in used[0].shape)
    for i, (p, q) in enumerate(zip(a, b)):
        if p is None:
            if not isinstance(q, int):
                raise ValueError(f"b[{i}] must be the width of a slice without adapters")
            continue
        _need(p, (E, R, K), _BF16, f"a[{i}]")
        if isinstance(q, int) or q is None or q.dim() != 3:
            raise ValueError(f"b[{i}] must be a 3-D tensor [adapters][n][rank]")
        _need(q, (E, int(q.shape[1]), R), _BF16, f"b[{i}]")
    _need(ranks, (E,), _I32, "ranks")
    _need(scale, (E,), _F32, "scale")
    lora = Lora(E, R, K, len(a))
    for i, (p, q) in enumerate(zip(a, b)):
        lora.n[i] = q if p is None else int(q.shape[1])
        if p is not None:
            lora.a[i], lora.b[i] = _ptr(p), _ptr(q)
    lora.ranks, lora.scale = _ptr(ranks), _ptr(scale)
    kept = [t for t in (*a, *b, ranks, scale) if t is not None and not isinstance(t, int)]
    lora.width = sum(lora.n[:len(a)])
    return _one_gpu(lora, *kept)


def lora_workspace_bytes(lora: Lora, rows: int) -> int:
    return lib().skinny_lora_workspace_bytes(lora, rows)


def lora_linear(lora: Lora, x, ids, y, workspace, base=None, stream=None):
    """y[t] = base[t] + scale[e] * B_e (A_e x[t]) for e = ids[t] (int32 [rows] on
    the GPU; rows with an id that is no adapter's keep base): x [rows][K] and y
    [rows][sum of the slices' n] bf16.  base None adds to y in place."""
    tt, dev = _call_device(x)
    rows = x.shape[0]
    xp = _operand(x, (rows, lora.K), tt.bf16, "x", dev)
    ip = _operand(ids, (rows,), tt.i32, "ids", dev)
    shape = (rows, lora.width or sum(lora.n[:max(lora.slices, 0)]))
    yp = _operand(y, shape, tt.bf16, "y", dev)
    bp = None if base is None else _operand(base, shape, tt.bf16, "base", dev)
    wp, wb = _space(workspace, dev)
    if lora.gpu not in (None, dev) and dev >= 0:
        raise ValueError(f"lora on GPU {lora.gpu}, the call's tensors on GPU {dev}")
    _check(lib().skinny_lora_linear(lora, xp, ip, rows, bp, yp, wp, wb,
                                    _call_stream(tt, dev, stream)), "skinny_lora_linear")
    return y


def moe_route(logits, ids, weights, scoring: int = ROUTE_SOFTMAX, bias=None, groups: int = 1,
              top_groups: int = 1, renormalize: bool = True, scale: float = 1.0, stream=None):
    """The topk experts of each row of logits [rows][experts] (bf16 or float32)
    into ids int32 [rows][topk], for moe_linear and moe_mlp_swiglu, and their
    weights into weights float32 [rows][topk], for block_norm's sum of the routes."""
    tt, dev = _call_device(logits)
    shape, chosen = logits.shape, ids.shape
    if len(shape) != 2 or len(chosen) != 2:
        raise ValueError("expected 2-D tensors")
    rows, experts = shape
    topk = chosen[1]
    each = (rows, topk)
    r = _ROUTE.pack(_values(logits, tt, "logits"), scoring, rows, experts, topk, groups, top_groups,
                    bool(renormalize), scale, 0,
                    _operand(logits, shape, logits.dtype, "logits", dev),
                    0 if bias is None else _operand(bias, (experts,), tt.f32, "bias", dev),
                    _operand(ids, each, tt.i32, "ids", dev),
                    _operand(weights, each, tt.f32, "weights", dev))
    _check(lib().route_of_bytes(r, _call_stream(tt, dev, stream)), "skinny_moe_route")
    return ids
