"""ctypes binding of libw4a16.so (argument marshalling only).

Every function takes torch tensors that already live on the GPU, checks
dtypes/shapes, and passes raw pointers, sizes and the current CUDA stream to
the C ABI declared in include/w4a16.h.  No arithmetic of the method happens
here, and there is no fallback: if the library is missing, ``load()`` raises.
"""

from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libw4a16.so")

W4_FLAG_PDL = 1
W4_FLAG_CUDA_CORES = 2
W4_FLAG_TENSOR_CORES = 4
W4_FLAG_SILU_MUL = 8
W4_FLAG_IDS_FINAL = 16


def _id_flags(pdl: bool, ids_final: bool) -> int:
    """ids_final: the ids were written before the previous kernel began
    (W4_FLAG_IDS_FINAL; only meaningful with pdl)."""
    return (W4_FLAG_PDL if pdl else 0) | (W4_FLAG_IDS_FINAL if ids_final else 0)
_PATH_FLAGS = {None: 0, "cuda": W4_FLAG_CUDA_CORES, "tensor": W4_FLAG_TENSOR_CORES}
STATUS = {0: "W4_OK", 1: "W4_ERR_ARG", 2: "W4_ERR_ALIGN", 3: "W4_ERR_SHAPE",
          4: "W4_ERR_WORKSPACE", 5: "W4_ERR_LAUNCH", 6: "W4_ERR_INDEX", 7: "W4_ERR_VALUE",
          8: "W4_ERR_TIMEOUT", 9: "W4_ERR_DEVICE", 10: "W4_ERR_STATE", 11: "W4_ERR_OWNER"}
STATUS_CODE = {v: k for k, v in STATUS.items()}

EXPORTS = ("w4_status_str", "w4_abi_version", "w4_last_cuda_error", "w4a16_gemv", "w4a16_gemv_workspace_bytes", "w4a16_gemv_workspace_bytes_flags",
           "w4a16_gemv_id", "w4a16_gemv_id_scaled", "w4_embed_gather", "w4_pack", "w4_quantize",
           "w4_slot_pool_create", "w4_slot_pool_destroy", "w4_slot_pool_remap",
           "w4_slot_pool_stage", "w4_slot_pool_stats", "w4a16_gemv_plan",
           "w4a16_gemv_static_scratch", "w4_dev_pool_state_bytes", "w4_dev_pool_init",
           "w4_dev_pool_stage", "w4_dev_pool_stats", "w4a16_gemv_chain",
           "w4a16_gemv_chain_workspace_bytes", "w4a16_gemv_chain_plan",
           "w4a16_gemv_chain_task_plan", "w4a16_gemv_id_plan", "w4a16_gemv_prefetch_l2",
           "w4a16_gemv_plan_flags", "w4_kv8_append", "w4_kv8_attn", "w4_kv8_attn_workspace_bytes",
           "w4_kv8_select", "w4_kv8_select_workspace_bytes", "w4_kv8_weigh", "w4_kv8_weigh_pages",
           "w4_kv8_evict", "w4_kv8_evict_workspace_bytes", "w4_route", "w4_moe_combine",
           "w4_logits_adjust", "w4_kv8_fork", "w4_kv8_reserve", "w4_kv8_compact",
           "w4_kv8_pages_workspace_bytes")
W4_TASK_SILU_MUL = 1
W4_MAX_L2_RANGES = 4
CHAIN_MAX_TASKS = 320


class W4Error(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        self.name = STATUS.get(code, str(code))
        super().__init__(f"{what}: {self.name}")


class PlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("path", "ctas", "slices", "threads", "team",
                                            "unit_rows", "chunk_groups", "rows_per_lane",
                                            "smem_bytes", "rows_per_call", "chunk_steps",
                                            "stages", "ctas_per_sm", "tmpl_team",
                                            "tmpl_chunk", "dynamic_windows")]


class GemvTask(ctypes.Structure):
    """struct w4_gemv_task of include/w4a16.h."""
    _fields_ = [("y", ctypes.c_void_p), ("qw", ctypes.c_void_p), ("st", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("qw_stride", ctypes.c_size_t),
                ("st_stride", ctypes.c_size_t), ("num_experts", ctypes.c_int),
                ("n_ids", ctypes.c_int), ("x_rows", ctypes.c_int), ("N", ctypes.c_int),
                ("K", ctypes.c_int), ("dep", ctypes.c_int), ("flags", ctypes.c_uint)]


class L2Range(ctypes.Structure):
    """struct w4_l2_range of include/w4a16.h."""
    _fields_ = [("ptr", ctypes.c_void_p), ("bytes", ctypes.c_size_t)]


class ChainPlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("ctas", "threads", "instantiation", "stages",
                                            "stage_bytes", "smem_bytes", "windows")]


class ChainTaskInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("rows_per_window", "rows_per_lane", "team",
                                            "chunk_steps", "chunks", "windows_per_item", "dot")]


class KV8CacheStruct(ctypes.Structure):
    """struct w4_kv8_cache of include/w4a16.h."""
    _fields_ = [("kc", ctypes.c_void_p), ("vc", ctypes.c_void_p), ("ks", ctypes.c_void_p),
                ("vs", ctypes.c_void_p), ("ranges", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("num_pages", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_stride", ctypes.c_size_t), ("head_stride", ctypes.c_size_t)]


class KV8BatchStruct(ctypes.Structure):
    """struct w4_kv8_batch of include/w4a16.h."""
    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("batch", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("rows", ctypes.c_int), ("max_new", ctypes.c_int), ("max_len", ctypes.c_int)]


class RouterStruct(ctypes.Structure):
    """struct w4_router of include/w4a16.h."""
    _fields_ = [("experts", ctypes.c_int), ("top_k", ctypes.c_int), ("groups", ctypes.c_int),
                ("top_groups", ctypes.c_int), ("group_best", ctypes.c_int),
                ("score", ctypes.c_int), ("renorm", ctypes.c_int), ("scale", ctypes.c_float)]


class LogitRulesStruct(ctypes.Structure):
    """struct w4_logit_rules of include/w4a16.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("tokens", "lens", "prompt", "repetition",
                                               "presence", "frequency", "bias_ids", "bias",
                                               "n_bias", "mask", "mask_rows")] + \
               [(n, ctypes.c_size_t) for n in ("token_stride", "bias_stride", "mask_stride")] + \
               [(n, ctypes.c_int) for n in ("max_tokens", "max_bias", "num_masks")]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    vp, i32, sz, u32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint
    i32p = ctypes.POINTER(ctypes.c_int32)
    lib.w4_status_str.restype = ctypes.c_char_p
    lib.w4_status_str.argtypes = [i32]
    lib.w4_abi_version.restype = i32
    lib.w4_last_cuda_error.restype = ctypes.c_char_p
    lib.w4_last_cuda_error.argtypes = []
    lib.w4a16_gemv.restype = i32
    lib.w4a16_gemv.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, sz, vp, u32, vp]
    lib.w4a16_gemv_prefetch_l2.restype = i32
    lib.w4a16_gemv_prefetch_l2.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, sz, vp, u32,
                                           ctypes.POINTER(L2Range), i32, vp]
    lib.w4a16_gemv_static_scratch.restype = i32
    lib.w4a16_gemv_static_scratch.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, u32, vp]
    lib.w4a16_gemv_workspace_bytes.restype = sz
    lib.w4a16_gemv_workspace_bytes.argtypes = [i32, i32, i32]
    lib.w4a16_gemv_workspace_bytes_flags.restype = sz
    lib.w4a16_gemv_workspace_bytes_flags.argtypes = [i32, i32, i32, ctypes.c_uint]
    lib.w4a16_gemv_id.restype = i32
    lib.w4a16_gemv_id.argtypes = [vp, vp, sz, vp, sz, i32, vp, i32, vp, i32, i32, i32, vp, u32, vp]
    lib.w4a16_gemv_id_scaled.restype = i32
    lib.w4a16_gemv_id_scaled.argtypes = [vp, vp, sz, vp, sz, i32, vp, i32, vp, i32, i32, i32,
                                         vp, i32, vp, vp, vp, vp, u32, vp]
    lib.w4_embed_gather.restype = i32
    lib.w4_embed_gather.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, u32, vp]
    lib.w4_pack.restype = i32
    lib.w4_pack.argtypes = [vp, vp, i32, i32, vp, vp]
    lib.w4_quantize.restype = i32
    lib.w4_quantize.argtypes = [vp, vp, vp, i32, i32, vp]
    lib.w4_slot_pool_create.restype = i32
    lib.w4_slot_pool_create.argtypes = [ctypes.POINTER(vp), i32, i32]
    lib.w4_slot_pool_destroy.restype = None
    lib.w4_slot_pool_destroy.argtypes = [vp]
    lib.w4_slot_pool_remap.restype = i32
    lib.w4_slot_pool_remap.argtypes = [vp, i32p, i32, i32p, i32p, i32p, ctypes.POINTER(i32)]
    lib.w4_slot_pool_stage.restype = i32
    lib.w4_slot_pool_stage.argtypes = [vp, i32p, i32, vp, vp, sz, sz, vp, vp, sz, sz, vp, vp,
                                       i32p, ctypes.POINTER(i32), vp]
    lib.w4_slot_pool_stats.restype = None
    lib.w4_slot_pool_stats.argtypes = [vp] + [ctypes.POINTER(ctypes.c_longlong)] * 3
    lib.w4_dev_pool_state_bytes.restype = sz
    lib.w4_dev_pool_state_bytes.argtypes = [i32, i32]
    lib.w4_dev_pool_init.restype = i32
    lib.w4_dev_pool_init.argtypes = [vp, i32, i32, vp]
    lib.w4_dev_pool_stage.restype = i32
    lib.w4_dev_pool_stage.argtypes = [vp, i32, i32, vp, i32, vp, vp, sz, sz, vp, vp, sz, sz, vp,
                                      vp, vp, u32, vp]
    lib.w4_dev_pool_stats.restype = i32
    lib.w4_dev_pool_stats.argtypes = [vp, i32, i32] + [ctypes.POINTER(ctypes.c_longlong)] * 3
    lib.w4a16_gemv_plan.restype = i32
    lib.w4a16_gemv_plan.argtypes = [i32, i32, i32, ctypes.POINTER(PlanInfo)]
    lib.w4a16_gemv_plan_flags.restype = i32
    lib.w4a16_gemv_plan_flags.argtypes = [i32, i32, i32, u32, ctypes.POINTER(PlanInfo)]
    lib.w4a16_gemv_id_plan.restype = i32
    lib.w4a16_gemv_id_plan.argtypes = [i32, i32, i32, i32, ctypes.POINTER(PlanInfo)]
    lib.w4a16_gemv_chain.restype = i32
    lib.w4a16_gemv_chain.argtypes = [ctypes.POINTER(GemvTask), i32, vp, sz, vp, u32, vp]
    lib.w4a16_gemv_chain_workspace_bytes.restype = sz
    lib.w4a16_gemv_chain_workspace_bytes.argtypes = [ctypes.POINTER(GemvTask), i32]
    lib.w4a16_gemv_chain_plan.restype = i32
    lib.w4a16_gemv_chain_plan.argtypes = [ctypes.POINTER(GemvTask), i32,
                                          ctypes.POINTER(ChainPlanInfo)]
    lib.w4a16_gemv_chain_task_plan.restype = i32
    lib.w4a16_gemv_chain_task_plan.argtypes = [ctypes.POINTER(GemvTask), i32, i32,
                                               ctypes.POINTER(ChainTaskInfo)]
    cp, bp, f32 = ctypes.POINTER(KV8CacheStruct), ctypes.POINTER(KV8BatchStruct), ctypes.c_float
    lib.w4_kv8_append.restype = i32
    lib.w4_kv8_append.argtypes = [cp, bp, vp, vp, sz, vp, u32, vp]
    lib.w4_kv8_attn.restype = i32
    lib.w4_kv8_attn.argtypes = [vp, vp, vp, sz, i32, cp, bp, f32, i32, vp, vp, i32, vp, sz, vp,
                                u32, vp]
    lib.w4_kv8_attn_workspace_bytes.restype = sz
    lib.w4_kv8_attn_workspace_bytes.argtypes = [cp, bp, i32, i32]
    lib.w4_kv8_select.restype = i32
    lib.w4_kv8_select.argtypes = [vp, vp, i32, i32, i32, vp, sz, i32, cp, bp, vp, sz, vp, u32, vp]
    lib.w4_kv8_select_workspace_bytes.restype = sz
    lib.w4_kv8_select_workspace_bytes.argtypes = [cp, bp]
    lib.w4_kv8_weigh.restype = i32
    lib.w4_kv8_weigh.argtypes = [vp, sz, i32, vp, cp, bp, f32, i32, vp, u32, vp]
    lib.w4_kv8_weigh_pages.restype = i32
    lib.w4_kv8_weigh_pages.argtypes = [vp, sz, i32, vp, cp, bp, f32, i32, vp, vp, i32, vp, u32, vp]
    lib.w4_kv8_evict.restype = i32
    lib.w4_kv8_evict.argtypes = [vp, vp, vp, i32, i32, i32, cp, bp, vp, sz, vp, u32, vp]
    lib.w4_kv8_evict_workspace_bytes.restype = sz
    lib.w4_kv8_evict_workspace_bytes.argtypes = [cp, bp, i32]
    lib.w4_route.restype = i32
    lib.w4_route.argtypes = [vp, vp, ctypes.POINTER(RouterStruct), vp, i32, sz, vp, i32, vp, u32, vp]
    lib.w4_moe_combine.restype = i32
    lib.w4_moe_combine.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, u32, vp]
    lib.w4_logits_adjust.restype = i32
    lib.w4_logits_adjust.argtypes = [vp, i32, sz, i32, i32, ctypes.POINTER(LogitRulesStruct), vp,
                                     u32, vp]
    lib.w4_kv8_fork.restype = i32
    lib.w4_kv8_fork.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, cp, i32, vp, sz, vp,
                                u32, vp]
    lib.w4_kv8_reserve.restype = i32
    lib.w4_kv8_reserve.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, sz, vp, u32, vp]
    lib.w4_kv8_compact.restype = i32
    lib.w4_kv8_compact.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, cp, i32, vp, sz, vp, u32, vp]
    lib.w4_kv8_pages_workspace_bytes.restype = sz
    lib.w4_kv8_pages_workspace_bytes.argtypes = [i32, i32]
    _lib = lib
    return lib


def _check(code: int, what: str):
    if code != 0:
        if code in (5, 10):
            what = f"{what} ({load().w4_last_cuda_error().decode()})"
        raise W4Error(code, what)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _as_words(qw: torch.Tensor) -> torch.Tensor:
    if qw.dtype not in (torch.int32, torch.uint32):
        raise ValueError("qw must hold 32-bit words (int32 or uint32)")
    return qw


# ------------------------------------------------------------------ calls
def workspace_bytes(M: int, N: int, K: int, path: str = None) -> int:
    """Zero-filled scratch a gemv call of this shape (and path choice) needs."""
    if path is None:
        return int(load().w4a16_gemv_workspace_bytes(M, N, K))
    return int(load().w4a16_gemv_workspace_bytes_flags(M, N, K, _PATH_FLAGS[path]))


def plan(M: int, N: int, K: int, path: str = None) -> dict:
    """Launch plan of a w4a16_gemv call (path: None, "cuda" or "tensor")."""
    info = PlanInfo()
    _check(load().w4a16_gemv_plan_flags(M, N, K, _PATH_FLAGS[path], ctypes.byref(info)),
           "w4a16_gemv_plan_flags")
    return {n: getattr(info, n) for n, _ in PlanInfo._fields_}


def id_plan(n_ids: int, x_rows: int, N: int, K: int) -> dict:
    """Launch plan of a w4a16_gemv_id call."""
    info = PlanInfo()
    _check(load().w4a16_gemv_id_plan(n_ids, x_rows, N, K, ctypes.byref(info)),
           "w4a16_gemv_id_plan")
    return {n: getattr(info, n) for n, _ in PlanInfo._fields_}


def l2_ranges(ranges):
    """A ctypes array of w4_l2_range from (tensor, bytes) or (address, bytes)
    pairs (bytes None: the whole tensor)."""
    arr = (L2Range * max(1, len(ranges)))()
    for i, (t, nbytes) in enumerate(ranges):
        if isinstance(t, torch.Tensor):
            _need(t, t.dtype, "prefetch range")
            full = t.numel() * t.element_size()
            nbytes = full if nbytes is None else min(int(nbytes), full)
            arr[i] = L2Range(t.data_ptr(), nbytes)
        else:
            arr[i] = L2Range(int(t), int(nbytes))
    return arr


def gemv(qw: torch.Tensor, st: torch.Tensor, x: torch.Tensor, y: torch.Tensor = None,
         workspace: torch.Tensor = None, status: torch.Tensor = None, pdl: bool = False,
         stream=None, path: str = None, silu_mul: bool = False, l2_next=None) -> torch.Tensor:
    """y[M, N] = x[M, K] @ W^T with W from (qw [N, K/8], st [N, K/32]).

    path: None (the library's choice), "cuda" (CUDA cores) or "tensor"
    (tcgen05 tensor cores; K a multiple of 256).
    silu_mul: x is [M, 2K] (gate then up) and the product takes
    silu(gate) * up, formed while the activations are staged.
    l2_next: up to 4 (tensor or address, bytes) ranges, normally the next
    call's codes and steps, brought into L2 once this call has requested its
    own weights (w4a16_gemv_prefetch_l2)."""
    qw = _as_words(qw)
    _need(qw, qw.dtype, "qw")
    _need(st, torch.bfloat16, "st")
    _need(x, torch.bfloat16, "x")
    x2 = x if x.dim() == 2 else x.view(1, -1)
    M, K = x2.shape
    if silu_mul:
        if K % 2:
            raise ValueError("silu_mul needs x rows of [gate | up]")
        K //= 2
    N = qw.shape[0]
    if qw.shape != (N, K // 8) or st.shape != (N, K // 32):
        raise ValueError("qw/st shapes do not match x")
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(y, torch.bfloat16, "y")
    # workspace: zero-filled, workspace_bytes(M, N, K, path) large.  The
    # library refuses a call whose K split needs it (W4_ERR_WORKSPACE); a
    # tensor-core call that only uses it for balanced runs runs without it.
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    flags = (W4_FLAG_PDL if pdl else 0) | _PATH_FLAGS[path] | (W4_FLAG_SILU_MUL if silu_mul else 0)
    if l2_next:
        if len(l2_next) > W4_MAX_L2_RANGES:
            raise ValueError(f"at most {W4_MAX_L2_RANGES} prefetch ranges")
        rs = l2_next if isinstance(l2_next, ctypes.Array) else l2_ranges(l2_next)
        _check(load().w4a16_gemv_prefetch_l2(_ptr(y), _ptr(qw), _ptr(st), _ptr(x2), M, N, K,
                                             _ptr(workspace), ws_bytes, _ptr(status), flags, rs,
                                             len(rs), _stream(stream)),
               "w4a16_gemv_prefetch_l2")
        return y
    _check(load().w4a16_gemv(_ptr(y), _ptr(qw), _ptr(st), _ptr(x2), M, N, K, _ptr(workspace),
                             ws_bytes, _ptr(status), flags, _stream(stream)),
           "w4a16_gemv")
    return y


def gemv_id(qw_base: torch.Tensor, st_base: torch.Tensor, ids: torch.Tensor, x: torch.Tensor,
            N: int, K: int, num_experts: int, qw_stride_bytes: int, st_stride_bytes: int,
            y: torch.Tensor = None, status: torch.Tensor = None, pdl: bool = False,
            stream=None, ids_final: bool = False) -> torch.Tensor:
    """y[i] = W_{ids[i]} @ x[i or 0]; experts at base + id * stride (bytes)."""
    _need(ids, torch.int32, "ids")
    _need(x, torch.bfloat16, "x")
    if not (qw_base.is_cuda and st_base.is_cuda):
        raise ValueError("bases must be CUDA tensors")
    x2 = x if x.dim() == 2 else x.view(1, -1)
    n_ids = ids.numel()
    if y is None:
        y = torch.empty((n_ids, N), dtype=torch.bfloat16, device=x.device)
    _need(y, torch.bfloat16, "y")
    _check(load().w4a16_gemv_id(_ptr(y), _ptr(qw_base), qw_stride_bytes, _ptr(st_base),
                                st_stride_bytes, num_experts, _ptr(ids), n_ids, _ptr(x2),
                                x2.shape[0], N, K, _ptr(status), _id_flags(pdl, ids_final),
                                _stream(stream)), "w4a16_gemv_id")
    return y


def bind_gemv_id(qw_base: torch.Tensor, st_base: torch.Tensor, ids: torch.Tensor,
                 x: torch.Tensor, N: int, K: int, num_experts: int, qw_stride_bytes: int,
                 st_stride_bytes: int, y: torch.Tensor, status: torch.Tensor = None):
    """w4a16_gemv_id with its arguments marshalled once, for decode loops.

    Returns call(pdl=False, stream=None), which enqueues the same routed
    product again (reading whatever the tensors hold at that time; they must
    stay allocated and in place).
    """
    _need(ids, torch.int32, "ids")
    _need(x, torch.bfloat16, "x")
    _need(y, torch.bfloat16, "y")
    if not (qw_base.is_cuda and st_base.is_cuda):
        raise ValueError("bases must be CUDA tensors")
    x2 = x if x.dim() == 2 else x.view(1, -1)
    fn = load().w4a16_gemv_id
    args = (_ptr(y), _ptr(qw_base), qw_stride_bytes, _ptr(st_base), st_stride_bytes, num_experts,
            _ptr(ids), ids.numel(), _ptr(x2), x2.shape[0], N, K, _ptr(status))

    def call(pdl: bool = False, stream=None, ids_final: bool = False):
        _check(fn(*args, _id_flags(pdl, ids_final), _stream(stream)), "w4a16_gemv_id")

    call.tensors = (qw_base, st_base, ids, x2, y, status)   # keep them alive
    return call


def _scaled_args(y, qw_base, qw_stride_bytes, st_base, st_stride_bytes, num_slots, ids, x, N, K,
                 expert_ids, num_experts, slot_expert, scale, bias, status):
    _need(ids, torch.int32, "ids")
    _need(expert_ids, torch.int32, "expert_ids")
    _need(x, torch.bfloat16, "x")
    _need(y, torch.bfloat16, "y")
    if expert_ids.numel() != ids.numel():
        raise ValueError("expert_ids must have one entry per id")
    if slot_expert is not None:
        _need(slot_expert, torch.int32, "slot_expert")
    for name, t in (("scale", scale), ("bias", bias)):
        if t is not None:
            _need(t, torch.bfloat16, name)
            if t.numel() != num_experts * N:
                raise ValueError(f"{name} must be [num_experts][N]")
    if not (qw_base.is_cuda and st_base.is_cuda):
        raise ValueError("bases must be CUDA tensors")
    x2 = x if x.dim() == 2 else x.view(1, -1)
    return x2, (_ptr(y), _ptr(qw_base), qw_stride_bytes, _ptr(st_base), st_stride_bytes,
                num_slots, _ptr(ids), ids.numel(), _ptr(x2), x2.shape[0], N, K, _ptr(expert_ids),
                num_experts, _ptr(slot_expert), _ptr(scale), _ptr(bias), _ptr(status))


def gemv_id_scaled(qw_base: torch.Tensor, st_base: torch.Tensor, ids: torch.Tensor,
                   x: torch.Tensor, N: int, K: int, num_slots: int, qw_stride_bytes: int,
                   st_stride_bytes: int, expert_ids: torch.Tensor, num_experts: int,
                   slot_expert: torch.Tensor = None, scale: torch.Tensor = None,
                   bias: torch.Tensor = None, y: torch.Tensor = None,
                   status: torch.Tensor = None, pdl: bool = False, stream=None,
                   ids_final: bool = False) -> torch.Tensor:
    """y[i] = bf16(fma(W_{ids[i]} @ x[i or 0], scale[e], bias[e])), e = expert_ids[i]:
    weights through slot (or expert) ids, per-expert vectors through real ids."""
    if y is None:
        y = torch.empty((ids.numel(), N), dtype=torch.bfloat16, device=x.device)
    _, args = _scaled_args(y, qw_base, qw_stride_bytes, st_base, st_stride_bytes, num_slots, ids,
                           x, N, K, expert_ids, num_experts, slot_expert, scale, bias, status)
    _check(load().w4a16_gemv_id_scaled(*args, _id_flags(pdl, ids_final), _stream(stream)),
           "w4a16_gemv_id_scaled")
    return y


def bind_gemv_id_scaled(qw_base, st_base, ids, x, N, K, num_slots, qw_stride_bytes,
                        st_stride_bytes, expert_ids, num_experts, y, slot_expert=None,
                        scale=None, bias=None, status=None):
    """w4a16_gemv_id_scaled with its arguments marshalled once: returns
    call(pdl=False, stream=None)."""
    x2, args = _scaled_args(y, qw_base, qw_stride_bytes, st_base, st_stride_bytes, num_slots,
                            ids, x, N, K, expert_ids, num_experts, slot_expert, scale, bias,
                            status)
    fn = load().w4a16_gemv_id_scaled

    def call(pdl: bool = False, stream=None, ids_final: bool = False):
        _check(fn(*args, _id_flags(pdl, ids_final), _stream(stream)), "w4a16_gemv_id_scaled")

    call.tensors = (qw_base, st_base, ids, x2, y, expert_ids, slot_expert, scale, bias, status)
    return call


def embed_gather(qw: torch.Tensor, st: torch.Tensor, ids: torch.Tensor, out: torch.Tensor = None,
                 status: torch.Tensor = None, pdl: bool = False, stream=None) -> torch.Tensor:
    qw = _as_words(qw)
    _need(qw, qw.dtype, "qw")
    _need(st, torch.bfloat16, "st")
    _need(ids, torch.int32, "ids")
    V, K = qw.shape[0], qw.shape[1] * 8
    T = ids.numel()
    if out is None:
        out = torch.empty((T, K), dtype=torch.bfloat16, device=qw.device)
    _need(out, torch.bfloat16, "out")
    _check(load().w4_embed_gather(_ptr(out), _ptr(qw), _ptr(st), _ptr(ids), T, V, K, _ptr(status),
                                  W4_FLAG_PDL if pdl else 0, _stream(stream)), "w4_embed_gather")
    return out


def pack(codes: torch.Tensor, qw: torch.Tensor = None, status: torch.Tensor = None,
         stream=None) -> torch.Tensor:
    _need(codes, torch.uint8, "codes")
    N, K = codes.shape
    if qw is None:
        qw = torch.empty((N, K // 8), dtype=torch.int32, device=codes.device)
    _check(load().w4_pack(_ptr(qw), _ptr(codes), N, K, _ptr(status), _stream(stream)), "w4_pack")
    return qw


def quantize(w: torch.Tensor, stream=None):
    _need(w, torch.float32, "w")
    N, K = w.shape
    qw = torch.empty((N, K // 8), dtype=torch.int32, device=w.device)
    st = torch.empty((N, K // 32), dtype=torch.bfloat16, device=w.device)
    _check(load().w4_quantize(_ptr(qw), _ptr(st), _ptr(w), N, K, _stream(stream)), "w4_quantize")
    return qw, st


class DevSlotPool:
    """Device-side LFU expert-slot pool: state in a device buffer, remap and
    fills enqueued on a stream (graph-capturable)."""

    def __init__(self, num_experts: int, num_slots: int, device="cuda", stream=None):
        self._lib = load()
        n = self._lib.w4_dev_pool_state_bytes(num_experts, num_slots)
        if n == 0:
            raise W4Error(3, "w4_dev_pool_state_bytes")
        self.state = torch.empty(n, dtype=torch.uint8, device=device)
        self.num_experts, self.num_slots = num_experts, num_slots
        self.reset(stream)

    def reset(self, stream=None):
        """Every slot free, every count 0 (enqueued on `stream`)."""
        _check(self._lib.w4_dev_pool_init(_ptr(self.state), self.num_experts, self.num_slots,
                                          _stream(stream)), "w4_dev_pool_init")

    def bind_stage(self, ids_dev: torch.Tensor, pool_qw, full_qw, qw_stride, qw_bytes, pool_st,
                   full_st, st_stride, st_bytes, slot_ids_dev: torch.Tensor, slot_expert=None,
                   status=None):
        """Returns call(pdl=False, stream=None) that enqueues the remap of the
        ids then held by ids_dev (device int32 [k]) and the fills."""
        _need(ids_dev, torch.int32, "ids_dev")
        _need(slot_ids_dev, torch.int32, "slot_ids_dev")
        fn = self._lib.w4_dev_pool_stage
        args = (_ptr(self.state), self.num_experts, self.num_slots, _ptr(ids_dev), ids_dev.numel(),
                _ptr(pool_qw), _ptr(full_qw), qw_stride, qw_bytes, _ptr(pool_st), _ptr(full_st),
                st_stride, st_bytes, _ptr(slot_ids_dev), _ptr(slot_expert), _ptr(status))

        def call(pdl: bool = False, stream=None):
            _check(fn(*args, W4_FLAG_PDL if pdl else 0, _stream(stream)), "w4_dev_pool_stage")

        call.tensors = (self.state, ids_dev, pool_qw, full_qw, pool_st, full_st, slot_ids_dev,
                        slot_expert, status)
        return call

    def stats(self):
        r, h, m = ctypes.c_longlong(), ctypes.c_longlong(), ctypes.c_longlong()
        _check(self._lib.w4_dev_pool_stats(_ptr(self.state), self.num_experts, self.num_slots,
                                           ctypes.byref(r), ctypes.byref(h), ctypes.byref(m)),
               "w4_dev_pool_stats")
        return {"requests": r.value, "hits": h.value, "misses": m.value}


class SlotPool:
    """Host LFU expert-slot pool (C++ in the library)."""

    def __init__(self, num_experts: int, num_slots: int):
        self._lib = load()
        h = ctypes.c_void_p()
        _check(self._lib.w4_slot_pool_create(ctypes.byref(h), num_experts, num_slots),
               "w4_slot_pool_create")
        self._h = h
        self.num_experts, self.num_slots = num_experts, num_slots

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._lib.w4_slot_pool_destroy(h)
            self._h = None

    def remap(self, ids):
        ids = [int(v) for v in ids]
        k = len(ids)
        arr = (ctypes.c_int32 * k)(*ids)
        slots = (ctypes.c_int32 * k)()
        me = (ctypes.c_int32 * k)()
        ms = (ctypes.c_int32 * k)()
        nm = ctypes.c_int()
        _check(self._lib.w4_slot_pool_remap(self._h, arr, k, slots, me, ms, ctypes.byref(nm)),
               "w4_slot_pool_remap")
        return list(slots), [(me[i], ms[i]) for i in range(nm.value)]

    def stage(self, ids, pool_qw, full_qw, qw_stride, qw_bytes, pool_st, full_st, st_stride,
              st_bytes, slot_ids_dev: torch.Tensor, stream=None, slot_expert=None):
        """Remap, copy missed experts into the pool and write slot ids (and, when
        given, the device slot table), all on `stream`.  full_qw / full_st may
        be CUDA tensors or page-locked CPU tensors."""
        ids = [int(v) for v in ids]
        k = len(ids)
        arr = (ctypes.c_int32 * k)(*ids)
        slots = (ctypes.c_int32 * k)()
        nm = ctypes.c_int()
        _check(self._lib.w4_slot_pool_stage(self._h, arr, k, _ptr(pool_qw), _ptr(full_qw),
                                            qw_stride, qw_bytes, _ptr(pool_st), _ptr(full_st),
                                            st_stride, st_bytes, _ptr(slot_ids_dev),
                                            _ptr(slot_expert), slots, ctypes.byref(nm),
                                            _stream(stream)),
               "w4_slot_pool_stage")
        return list(slots), nm.value

    def bind_stage(self, k: int, pool_qw, full_qw, qw_stride, qw_bytes, pool_st, full_st,
                   st_stride, st_bytes, slot_ids_dev: torch.Tensor, slot_expert=None):
        """stage() with the buffers marshalled once: returns call(ids, stream=None)
        for requests of k ids (any int sequence), which returns the misses."""
        arr = (ctypes.c_int32 * k)()
        slots = (ctypes.c_int32 * k)()
        nm = ctypes.c_int()
        fixed = (_ptr(pool_qw), _ptr(full_qw), qw_stride, qw_bytes, _ptr(pool_st), _ptr(full_st),
                 st_stride, st_bytes, _ptr(slot_ids_dev), _ptr(slot_expert), slots,
                 ctypes.byref(nm))
        fn, h = self._lib.w4_slot_pool_stage, self._h

        def call(ids, stream=None) -> int:
            if len(ids) != k:
                raise ValueError(f"expected {k} ids")
            for i, v in enumerate(ids):
                arr[i] = int(v)
            _check(fn(h, arr, k, *fixed, _stream(stream)), "w4_slot_pool_stage")
            return nm.value

        call.tensors = (pool_qw, full_qw, pool_st, full_st, slot_ids_dev, slot_expert)
        return call

    def stats(self):
        r, h, m = ctypes.c_longlong(), ctypes.c_longlong(), ctypes.c_longlong()
        self._lib.w4_slot_pool_stats(self._h, ctypes.byref(r), ctypes.byref(h), ctypes.byref(m))
        return {"requests": r.value, "hits": h.value, "misses": m.value}


# ------------------------------------------------------------------ chains
def gemv_task(qw: torch.Tensor, st: torch.Tensor, x: torch.Tensor, y: torch.Tensor, dep: int = -1,
              silu_mul: bool = False) -> dict:
    """A dense task of a chain: y[N] = W x (x [K], or [2K] = [gate | up] with silu_mul)."""
    qw = _as_words(qw)
    for t, dt, name in ((qw, qw.dtype, "qw"), (st, torch.bfloat16, "st"),
                        (x, torch.bfloat16, "x"), (y, torch.bfloat16, "y")):
        _need(t, dt, name)
    N, K = qw.shape[0], qw.shape[-1] * 8
    if st.shape[0] != N or st.shape[-1] != K // 32 or y.numel() != N:
        raise ValueError("qw, st and y disagree on N or K")
    if x.numel() != K * (2 if silu_mul else 1):
        raise ValueError("x must hold one activation row")
    return {"y": y, "qw": qw, "st": st, "x": x, "ids": None, "qw_stride": 0, "st_stride": 0,
            "num_experts": 0, "n_ids": 1, "x_rows": 1, "N": N, "K": K, "dep": dep,
            "flags": W4_TASK_SILU_MUL if silu_mul else 0}


def gemv_id_task(qw_base: torch.Tensor, st_base: torch.Tensor, ids: torch.Tensor,
                 x: torch.Tensor, y: torch.Tensor, N: int, K: int, num_experts: int,
                 qw_stride_bytes: int, st_stride_bytes: int, dep: int = -1,
                 silu_mul: bool = False) -> dict:
    """A routed task of a chain: y[i] = W_{ids[i]} x_i (x_i: row i when x has
    n_ids rows, else row 0; [gate | up] rows of 2K with silu_mul)."""
    _need(ids, torch.int32, "ids")
    _need(x, torch.bfloat16, "x")
    _need(y, torch.bfloat16, "y")
    n_ids = ids.numel()
    row = K * (2 if silu_mul else 1)
    if x.numel() % row or x.numel() // row not in (1, n_ids):
        raise ValueError("x must hold 1 or n_ids activation rows")
    if y.numel() != n_ids * N:
        raise ValueError("y must be [n_ids, N]")
    return {"y": y, "qw": qw_base, "st": st_base, "x": x, "ids": ids,
            "qw_stride": qw_stride_bytes, "st_stride": st_stride_bytes,
            "num_experts": num_experts, "n_ids": n_ids, "x_rows": x.numel() // row, "N": N,
            "K": K, "dep": dep, "flags": W4_TASK_SILU_MUL if silu_mul else 0}


def _task_array(tasks):
    arr = (GemvTask * len(tasks))()
    for i, t in enumerate(tasks):
        g = arr[i]
        for name in ("y", "qw", "st", "x", "ids"):
            setattr(g, name, None if t[name] is None else t[name].data_ptr())
        for name in ("qw_stride", "st_stride", "num_experts", "n_ids", "x_rows", "N", "K", "dep",
                     "flags"):
            setattr(g, name, int(t[name]))
    return arr


def chain_workspace_bytes(tasks) -> int:
    """Bytes of the zero-initialised workspace a chain of these tasks needs."""
    return int(load().w4a16_gemv_chain_workspace_bytes(_task_array(tasks), len(tasks)))


def chain_plan(tasks) -> dict:
    arr = _task_array(tasks)
    info = ChainPlanInfo()
    _check(load().w4a16_gemv_chain_plan(arr, len(tasks), ctypes.byref(info)),
           "w4a16_gemv_chain_plan")
    return {n: getattr(info, n) for n, _ in ChainPlanInfo._fields_}


def chain_task_plan(tasks, task: int) -> dict:
    arr = _task_array(tasks)
    info = ChainTaskInfo()
    _check(load().w4a16_gemv_chain_task_plan(arr, len(tasks), task, ctypes.byref(info)),
           "w4a16_gemv_chain_task_plan", "w4a16_gemv_id_plan")
    return {n: getattr(info, n) for n, _ in ChainTaskInfo._fields_}


def bind_gemv_chain(tasks, workspace: torch.Tensor, status: torch.Tensor = None):
    """w4a16_gemv_chain with the task list marshalled once: returns
    call(pdl=False, stream=None).  `workspace` (uint8, zeroed once) must hold
    chain_workspace_bytes(tasks) bytes."""
    _need(workspace, torch.uint8, "workspace")
    arr = _task_array(tasks)
    n = len(tasks)
    fn = load().w4a16_gemv_chain
    ws_ptr, ws_bytes = _ptr(workspace), workspace.numel()

    def call(pdl: bool = False, stream=None):
        _check(fn(arr, n, ws_ptr, ws_bytes, _ptr(status), W4_FLAG_PDL if pdl else 0,
                  _stream(stream)), "w4a16_gemv_chain")

    call.tensors = (tasks, workspace, status)   # keep the buffers alive with the binding
    return call


def gemv_chain(tasks, workspace: torch.Tensor, status: torch.Tensor = None, pdl: bool = False,
               stream=None):
    """Run the tasks (dicts from gemv_task / gemv_id_task) as one launch."""
    bind_gemv_chain(tasks, workspace, status)(pdl=pdl, stream=stream)


# ------------------------------------------------------------------ 8-bit key/value cache
class KV8Cache:
    """The pages of an 8-bit key/value cache (struct w4_kv8_cache).

    kc, vc: uint8 [pages, kv_heads, page_tokens, head_dim], the last two dimensions dense, both
    with the same strides (views of one larger tensor, of a layer say, are fine); ks, vs: fp32
    [pages, kv_heads]; ranges: uint8 [pages, kv_heads, 2, head_dim] or None (kv8_select needs
    it); weight: fp32 [pages, kv_heads, page_tokens] or None (kv8_weigh and kv8_evict need it).
    A value is (code - 128) * step."""

    def __init__(self, kc: torch.Tensor, vc: torch.Tensor, ks: torch.Tensor, vs: torch.Tensor,
                 ranges: torch.Tensor = None, weight: torch.Tensor = None):
        for t, name in ((kc, "kc"), (vc, "vc")):
            if not t.is_cuda or t.dtype != torch.uint8 or t.dim() != 4:
                raise ValueError(f"{name} must be a 4-dimensional uint8 CUDA tensor")
        if kc.shape != vc.shape or kc.stride() != vc.stride():
            raise ValueError("kc and vc must have the same shape and strides")
        n, h, p, d = kc.shape
        if kc.stride(3) != 1 or kc.stride(2) != d:
            raise ValueError("tokens and channels of a block must be dense")
        for t, name, shape, dtype in ((ks, "ks", (n, h), torch.float32),
                                      (vs, "vs", (n, h), torch.float32),
                                      (ranges, "ranges", (n, h, 2, d), torch.uint8),
                                      (weight, "weight", (n, h, p), torch.float32)):
            if t is None and name in ("ranges", "weight"):
                continue
            _need(t, dtype, name)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {list(shape)}")
        self.tensors = (kc, vc, ks, vs, ranges, weight)
        self.pages, self.kv_heads, self.page_tokens, self.head_dim = n, h, p, d
        self.device = kc.device
        self.struct = KV8CacheStruct(
            *[None if t is None else t.data_ptr() for t in self.tensors], n, h, p, d,
            kc.stride(0) if n > 1 else h * p * d, kc.stride(1) if h > 1 else p * d)


class KV8Batch:
    """The sequences of a call (struct w4_kv8_batch): table int32 [batch, max_pages], lens int32
    [batch] (the new tokens included), offsets int32 [batch + 1] of the packed new rows or None
    (one row per sequence); rows, max_new and max_len bound them (the tensors may change between
    calls, within the bounds)."""

    def __init__(self, table: torch.Tensor, lens: torch.Tensor, offsets: torch.Tensor = None,
                 rows: int = None, max_new: int = 1, max_len: int = None, page_tokens: int = None):
        _need(table, torch.int32, "table")
        _need(lens, torch.int32, "lens")
        if table.dim() != 2 or lens.shape != (table.shape[0],):
            raise ValueError("table must be [batch, max_pages] and lens [batch]")
        if offsets is not None:
            _need(offsets, torch.int32, "offsets")
            if offsets.shape != (table.shape[0] + 1,):
                raise ValueError("offsets must be [batch + 1]")
        self.batch, self.max_pages = table.shape
        self.rows = rows if rows is not None else (self.batch if offsets is None else None)
        self.max_new = max_new
        if max_len is None:
            if page_tokens is None:
                raise ValueError("max_len (or page_tokens) is needed")
            max_len = self.max_pages * page_tokens
        self.max_len = max_len
        self.tensors = (table, lens, offsets)
        self._structs = {}

    def struct(self, rows: int) -> KV8BatchStruct:
        """The C struct for calls on `rows` packed rows."""
        if self.rows is not None and rows != self.rows:
            raise ValueError(f"expected {self.rows} packed rows, got {rows}")
        if rows not in self._structs:
            self._structs[rows] = KV8BatchStruct(
                *[None if t is None else t.data_ptr() for t in self.tensors], self.batch,
                self.max_pages, rows, self.max_new, self.max_len)
        return self._structs[rows]


def _kv8_rows(t: torch.Tensor, name: str, heads: int, d: int):
    """Packed rows [T, heads, head_dim] of bf16, heads and channels dense: (row stride, T)."""
    if not t.is_cuda or t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a CUDA tensor of bfloat16")
    if t.dim() != 3 or t.shape[2] != d or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [rows, heads, head_dim]")
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != d):
        raise ValueError(f"heads and channels of {name} must be dense")
    return (t.stride(0) if t.shape[0] > 1 else t.shape[1] * d), t.shape[0]


def _kv8_bytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


_handles = {}   # stream handles as ctypes pointers
_CONVERTED = (ctypes._SimpleCData, ctypes.Array, type(ctypes.byref(ctypes.c_int())))


def _kv8_call(fn, name, args, keep):
    """call(pdl=False, stream=None) that enqueues fn(*args) again."""
    dev = keep[0].device.index
    if dev is None:
        dev = torch.cuda.current_device()
    raw = torch._C._cuda_getCurrentRawStream   # current_stream() builds an object each time
    # the arguments converted once: the same function, without types to convert by at each call
    bare = load()[name]
    bare.restype = ctypes.c_int
    args = tuple(a if isinstance(a, _CONVERTED) else t(a) for t, a in zip(fn.argtypes, args))

    def call(pdl: bool = False, stream=None):
        handle = raw(dev) if stream is None else stream.cuda_stream
        at = _handles.get(handle)
        if at is None:
            at = _handles[handle] = ctypes.c_void_p(handle)
        code = bare(*args, W4_FLAG_PDL if pdl else 0, at)
        if code:
            _check(code, name)

    call.tensors = keep
    return call


def kv8_attn_workspace_bytes(cache: KV8Cache, batch: KV8Batch, q_heads: int, rows: int = None,
                             max_sel: int = 0) -> int:
    """Zero-filled scratch of a kv8_attn call (rows: packed rows, if the batch does not say)."""
    rows = rows if rows is not None else batch.rows if batch.rows is not None else \
        batch.batch * batch.max_new
    return int(load().w4_kv8_attn_workspace_bytes(ctypes.byref(cache.struct),
                                                  ctypes.byref(batch.struct(rows)), q_heads,
                                                  max_sel))


def kv8_select_workspace_bytes(cache: KV8Cache, batch: KV8Batch) -> int:
    return int(load().w4_kv8_select_workspace_bytes(ctypes.byref(cache.struct),
                                                    ctypes.byref(batch.struct(batch.batch))))


def kv8_evict_workspace_bytes(cache: KV8Cache, batch: KV8Batch, budget: int) -> int:
    rows = batch.rows if batch.rows is not None else batch.batch
    return int(load().w4_kv8_evict_workspace_bytes(ctypes.byref(cache.struct),
                                                   ctypes.byref(batch.struct(rows)), budget))


def bind_kv8_append(cache: KV8Cache, batch: KV8Batch, k: torch.Tensor, v: torch.Tensor,
                    status: torch.Tensor = None):
    """w4_kv8_append with its arguments marshalled once: returns call(pdl=False, stream=None),
    which stores whatever rows k and v ([rows, kv_heads, head_dim]) hold at that time."""
    stride, rows = _kv8_rows(k, "k", cache.kv_heads, cache.head_dim)
    if _kv8_rows(v, "v", cache.kv_heads, cache.head_dim) != (stride, rows):
        raise ValueError("k and v must have the same rows and row stride")
    bs = batch.struct(rows)
    args = (ctypes.byref(cache.struct), ctypes.byref(bs), _ptr(k), _ptr(v), stride, _ptr(status))
    return _kv8_call(load().w4_kv8_append, "w4_kv8_append", args, (cache, batch, bs, k, v, status))


def kv8_append(cache: KV8Cache, batch: KV8Batch, k: torch.Tensor, v: torch.Tensor,
               status: torch.Tensor = None, pdl: bool = False, stream=None):
    """Store the new tokens' keys and values ([rows, kv_heads, head_dim] bf16) in the pages."""
    bind_kv8_append(cache, batch, k, v, status)(pdl, stream)


def _kv8_sel(cache: KV8Cache, batch: KV8Batch, sel, n_sel) -> int:
    """max_sel of a selection (0: none)."""
    if sel is None and n_sel is None:
        return 0
    if sel is None or n_sel is None:
        raise ValueError("sel and n_sel go together")
    _need(sel, torch.int32, "sel")
    _need(n_sel, torch.int32, "n_sel")
    max_sel = sel.shape[-1]
    if tuple(sel.shape) != (batch.batch, cache.kv_heads, max_sel) or \
            tuple(n_sel.shape) != (batch.batch, cache.kv_heads):
        raise ValueError("sel must be [batch, kv_heads, max_sel] and n_sel [batch, kv_heads]")
    return max_sel


def bind_kv8_attn(cache: KV8Cache, batch: KV8Batch, q: torch.Tensor, scale: float,
                  out: torch.Tensor, lse: torch.Tensor = None, window: int = 0,
                  sel: torch.Tensor = None, n_sel: torch.Tensor = None,
                  workspace: torch.Tensor = None, status: torch.Tensor = None):
    """w4_kv8_attn with its arguments marshalled once: returns call(pdl=False, stream=None)."""
    stride, rows = _kv8_rows(q, "q", None, cache.head_dim)
    q_heads = q.shape[1]
    _need(out, torch.bfloat16, "out")
    if tuple(out.shape) != (rows, q_heads, cache.head_dim):
        raise ValueError("out must be [rows, q_heads, head_dim]")
    if lse is not None:
        _need(lse, torch.float32, "lse")
        if tuple(lse.shape) != (rows, q_heads):
            raise ValueError("lse must be [rows, q_heads]")
    max_sel = _kv8_sel(cache, batch, sel, n_sel)
    bs = batch.struct(rows)
    args = (_ptr(out), _ptr(lse), _ptr(q), stride, q_heads, ctypes.byref(cache.struct),
            ctypes.byref(bs), scale, window, _ptr(sel), _ptr(n_sel), max_sel, _ptr(workspace),
            _kv8_bytes(workspace), _ptr(status))
    return _kv8_call(load().w4_kv8_attn, "w4_kv8_attn", args,
                     (cache, batch, bs, q, out, lse, sel, n_sel, workspace, status))


def kv8_attn(cache: KV8Cache, batch: KV8Batch, q: torch.Tensor, scale: float,
             out: torch.Tensor = None, lse: torch.Tensor = None, window: int = 0,
             sel: torch.Tensor = None, n_sel: torch.Tensor = None,
             workspace: torch.Tensor = None, status: torch.Tensor = None, pdl: bool = False,
             stream=None) -> torch.Tensor:
    """Attention of the new rows q [rows, q_heads, head_dim] over their sequences' cached tokens
    (causal; within `window` tokens if > 0; over the pages of sel / n_sel if given)."""
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    bind_kv8_attn(cache, batch, q, scale, out, lse, window, sel, n_sel, workspace,
                  status)(pdl, stream)
    return out


def bind_kv8_select(cache: KV8Cache, batch: KV8Batch, q: torch.Tensor, sel: torch.Tensor,
                    n_sel: torch.Tensor, sink: int = 1, recent: int = 1,
                    workspace: torch.Tensor = None, status: torch.Tensor = None):
    """w4_kv8_select with its arguments marshalled once: returns call(pdl=False, stream=None)."""
    stride, rows = _kv8_rows(q, "q", None, cache.head_dim)
    _need(sel, torch.int32, "sel")
    _need(n_sel, torch.int32, "n_sel")
    if sel.dim() != 3 or tuple(sel.shape[:2]) != (batch.batch, cache.kv_heads) or \
            tuple(n_sel.shape) != (batch.batch, cache.kv_heads):
        raise ValueError("sel must be [batch, kv_heads, max_sel] and n_sel [batch, kv_heads]")
    bs = batch.struct(rows)
    args = (_ptr(sel), _ptr(n_sel), sel.shape[2], sink, recent, _ptr(q), stride, q.shape[1],
            ctypes.byref(cache.struct), ctypes.byref(bs), _ptr(workspace), _kv8_bytes(workspace),
            _ptr(status))
    return _kv8_call(load().w4_kv8_select, "w4_kv8_select", args,
                     (cache, batch, bs, q, sel, n_sel, workspace, status))


def kv8_select(cache: KV8Cache, batch: KV8Batch, q: torch.Tensor, max_sel: int, sink: int = 1,
               recent: int = 1, workspace: torch.Tensor = None, status: torch.Tensor = None,
               pdl: bool = False, stream=None):
    """(sel, n_sel): the logical pages of highest score bound for each sequence's new row."""
    sel = torch.empty((batch.batch, cache.kv_heads, max_sel), dtype=torch.int32, device=q.device)
    n_sel = torch.empty((batch.batch, cache.kv_heads), dtype=torch.int32, device=q.device)
    bind_kv8_select(cache, batch, q, sel, n_sel, sink, recent, workspace, status)(pdl, stream)
    return sel, n_sel


def bind_kv8_weigh(cache: KV8Cache, batch: KV8Batch, q: torch.Tensor, lse: torch.Tensor,
                   scale: float, window: int = 0, status: torch.Tensor = None,
                   sel: torch.Tensor = None, n_sel: torch.Tensor = None):
    """w4_kv8_weigh (over the pages of sel / n_sel if given: w4_kv8_weigh_pages) with its arguments
    marshalled once: returns call(pdl=False, stream=None)."""
    stride, rows = _kv8_rows(q, "q", None, cache.head_dim)
    _need(lse, torch.float32, "lse")
    if tuple(lse.shape) != (rows, q.shape[1]):
        raise ValueError("lse must be [rows, q_heads]")
    bs = batch.struct(rows)
    args = (_ptr(q), stride, q.shape[1], _ptr(lse), ctypes.byref(cache.struct), ctypes.byref(bs),
            scale, window)
    max_sel = _kv8_sel(cache, batch, sel, n_sel)
    if max_sel == 0 and sel is None:
        return _kv8_call(load().w4_kv8_weigh, "w4_kv8_weigh", (*args, _ptr(status)),
                         (cache, batch, bs, q, lse, status))
    return _kv8_call(load().w4_kv8_weigh_pages, "w4_kv8_weigh_pages",
                     (*args, _ptr(sel), _ptr(n_sel), max_sel, _ptr(status)),
                     (cache, batch, bs, q, lse, sel, n_sel, status))


def kv8_weigh(cache: KV8Cache, batch: KV8Batch, q: torch.Tensor, lse: torch.Tensor, scale: float,
              window: int = 0, status: torch.Tensor = None, pdl: bool = False, stream=None,
              sel: torch.Tensor = None, n_sel: torch.Tensor = None):
    """Add the attention weight that each cached token receives from the new rows to
    cache.weight (lse as given by kv8_attn for the same rows, with the same selection).  No two
    sequences of the batch may share a page (as rows that kv8_fork made do): they would race on its
    weights."""
    bind_kv8_weigh(cache, batch, q, lse, scale, window, status, sel, n_sel)(pdl, stream)


def bind_kv8_evict(cache: KV8Cache, batch: KV8Batch, dst_table: torch.Tensor, kept: torch.Tensor,
                   new_lens: torch.Tensor, sink: int = 0, recent: int = 0,
                   workspace: torch.Tensor = None, status: torch.Tensor = None):
    """w4_kv8_evict with its arguments marshalled once: returns call(pdl=False, stream=None)."""
    for t, name in ((dst_table, "dst_table"), (kept, "kept"), (new_lens, "new_lens")):
        _need(t, torch.int32, name)
    if kept.dim() != 3 or tuple(kept.shape[:2]) != (batch.batch, cache.kv_heads):
        raise ValueError("kept must be [batch, kv_heads, budget]")
    budget = kept.shape[2]
    if tuple(dst_table.shape) != (batch.batch, -(-budget // cache.page_tokens)) or \
            tuple(new_lens.shape) != (batch.batch,):
        raise ValueError("dst_table must be [batch, ceil(budget / page_tokens)], new_lens [batch]")
    bs = batch.struct(batch.rows if batch.rows is not None else batch.batch)
    args = (_ptr(dst_table), _ptr(kept), _ptr(new_lens), budget, sink, recent,
            ctypes.byref(cache.struct), ctypes.byref(bs), _ptr(workspace), _kv8_bytes(workspace),
            _ptr(status))
    return _kv8_call(load().w4_kv8_evict, "w4_kv8_evict", args,
                     (cache, batch, bs, dst_table, kept, new_lens, workspace, status))


def kv8_evict(cache: KV8Cache, batch: KV8Batch, budget: int, dst_table: torch.Tensor,
              sink: int = 0, recent: int = 0, workspace: torch.Tensor = None,
              status: torch.Tensor = None, pdl: bool = False, stream=None):
    """(kept, new_lens): the `budget` tokens of most accumulated weight of each sequence and head,
    gathered into the pages of dst_table."""
    kept = torch.empty((batch.batch, cache.kv_heads, budget), dtype=torch.int32,
                       device=cache.device)
    new_lens = torch.empty((batch.batch,), dtype=torch.int32, device=cache.device)
    bind_kv8_evict(cache, batch, dst_table, kept, new_lens, sink, recent, workspace,
                   status)(pdl, stream)
    return kept, new_lens


# ------------------------------------------------------------------ pages of the cache
def _same_device(*tensors):
    """The tensors' device, which must be the current one (a call launches there)."""
    devs = {t.device for t in tensors if t is not None}
    if len(devs) != 1:
        raise ValueError("all tensors of a call must be on one device")
    dev = devs.pop()
    if dev.type != "cuda" or dev.index not in (None, torch.cuda.current_device()):
        raise ValueError(f"the tensors are on {dev}, which is not the current CUDA device")
    return dev


def _caches(caches):
    """An array of w4_kv8_cache of one cache or several."""
    caches = [caches] if isinstance(caches, KV8Cache) else list(caches)
    if not caches:
        raise ValueError("at least one cache is needed")
    return caches, (KV8CacheStruct * len(caches))(*[c.struct for c in caches])


def _kv8_table(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor):
    for t, name in ((table, "table"), (lens, "lens"), (refs, "refs")):
        _need(t, torch.int32, name)
    if table.dim() != 2 or lens.shape != (table.shape[0],) or refs.dim() != 1:
        raise ValueError("table must be [batch, max_pages], lens [batch] and refs [pages]")


def kv8_pages_workspace_bytes(batch: int, num_pages: int) -> int:
    """Scratch of kv8_fork, kv8_reserve and kv8_compact calls of up to `batch` rows (old or new)
    on a pool of num_pages pages."""
    return int(load().w4_kv8_pages_workspace_bytes(batch, num_pages))


def bind_kv8_fork(caches, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                  parents: torch.Tensor, new_table: torch.Tensor, new_lens: torch.Tensor,
                  new_refs: torch.Tensor, workspace: torch.Tensor, status: torch.Tensor = None):
    """w4_kv8_fork with its arguments marshalled once: returns call(pdl=False, stream=None).
    caches: a KV8Cache or several of one shape (a model's layers)."""
    caches, arr = _caches(caches)
    _kv8_table(table, lens, refs)
    _kv8_table(new_table, new_lens, new_refs)
    _need(parents, torch.int32, "parents")
    if refs.shape != (caches[0].pages,) or new_refs.shape != refs.shape:
        raise ValueError("refs and new_refs must be [pages]")
    if new_table.shape[1] != table.shape[1] or parents.shape != new_lens.shape:
        raise ValueError("new_table must be [new_batch, max_pages] and parents [new_batch]")
    _same_device(*[c.tensors[0] for c in caches], table, lens, refs, parents, new_table, new_lens,
                 new_refs, workspace, status)
    args = (_ptr(new_table), _ptr(new_lens), _ptr(new_refs), new_table.shape[0], _ptr(parents),
            _ptr(table), _ptr(lens), _ptr(refs), *table.shape, arr, len(caches), _ptr(workspace),
            _kv8_bytes(workspace), _ptr(status))
    return _kv8_call(load().w4_kv8_fork, "w4_kv8_fork", args,
                     (table, caches, lens, refs, parents, new_table, new_lens, new_refs, workspace,
                      status))


def kv8_fork(caches, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
             parents: torch.Tensor, workspace: torch.Tensor, status: torch.Tensor = None,
             pdl: bool = False, stream=None):
    """(new_table, new_lens, new_refs): row b goes on from row parents[b] of the old table (-1:
    it is empty); the pages that rows will write to are their own.  Entries past a row's pages
    are -1.  Rows that share pages cannot be weighed in one kv8_weigh call."""
    shape = (parents.numel(), table.shape[1])
    new_table = torch.full(shape, -1, dtype=torch.int32, device=table.device)
    new_lens, new_refs = torch.empty_like(parents), torch.empty_like(refs)
    _on(stream, new_table, new_lens, new_refs)
    bind_kv8_fork(caches, table, lens, refs, parents, new_table, new_lens, new_refs, workspace,
                  status)(pdl, stream)
    return new_table, new_lens, new_refs


def _on(stream, *tensors):
    """Fresh tensors whose first use is on another stream than the one they were allocated (and
    filled) on: that stream waits for the current one, and the memory is not reused before it is
    done."""
    if stream is None or stream == torch.cuda.current_stream():
        return
    stream.wait_stream(torch.cuda.current_stream())
    for t in tensors:
        t.record_stream(stream)


def bind_kv8_reserve(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                     page_tokens: int, grow: torch.Tensor = None, workspace: torch.Tensor = None,
                     status: torch.Tensor = None):
    """w4_kv8_reserve with its arguments marshalled once: returns call(pdl=False, stream=None).
    workspace: kv8_pages_workspace_bytes(batch, pages) bytes."""
    _kv8_table(table, lens, refs)
    if workspace is None:
        raise ValueError("workspace must be a tensor of kv8_pages_workspace_bytes(batch, pages) bytes")
    if grow is not None:
        _need(grow, torch.int32, "grow")
        if grow.shape != lens.shape:
            raise ValueError("grow must be [batch]")
    _same_device(table, lens, refs, grow, workspace, status)
    args = (_ptr(table), _ptr(lens), _ptr(refs), _ptr(grow), *table.shape, refs.shape[0],
            page_tokens, _ptr(workspace), _kv8_bytes(workspace), _ptr(status))
    return _kv8_call(load().w4_kv8_reserve, "w4_kv8_reserve", args,
                     (table, lens, refs, grow, workspace, status))


def kv8_reserve(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_tokens: int,
                grow: torch.Tensor = None, workspace: torch.Tensor = None,
                status: torch.Tensor = None, pdl: bool = False, stream=None):
    """lens += grow (None: one token for each row that has any), with pages for the new tokens, in
    place.  workspace: None allocates one for this call."""
    if workspace is None:
        _kv8_table(table, lens, refs)
        workspace = torch.empty(kv8_pages_workspace_bytes(lens.numel(), refs.numel()),
                                dtype=torch.uint8, device=table.device)
        _on(stream, workspace)
    bind_kv8_reserve(table, lens, refs, page_tokens, grow, workspace, status)(pdl, stream)


def bind_kv8_compact(caches, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                     new_table: torch.Tensor, new_refs: torch.Tensor, used: torch.Tensor,
                     workspace: torch.Tensor, status: torch.Tensor = None):
    """w4_kv8_compact with its arguments marshalled once: returns call(pdl=False, stream=None)."""
    caches, arr = _caches(caches)
    _kv8_table(table, lens, refs)
    _kv8_table(new_table, lens, new_refs)
    _need(used, torch.int32, "used")
    if refs.shape != (caches[0].pages,) or new_refs.shape != refs.shape or used.numel() != 1:
        raise ValueError("refs and new_refs must be [pages] and used [1]")
    if new_table.shape != table.shape:
        raise ValueError("new_table must have the shape of table")
    _same_device(*[c.tensors[0] for c in caches], table, lens, refs, new_table, new_refs, used,
                 workspace, status)
    args = (_ptr(new_table), _ptr(new_refs), _ptr(used), _ptr(table), _ptr(lens), _ptr(refs),
            *table.shape, arr, len(caches), _ptr(workspace), _kv8_bytes(workspace), _ptr(status))
    return _kv8_call(load().w4_kv8_compact, "w4_kv8_compact", args,
                     (table, caches, lens, refs, new_table, new_refs, used, workspace, status))


def kv8_compact(caches, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                workspace: torch.Tensor, status: torch.Tensor = None, pdl: bool = False,
                stream=None):
    """(new_table, new_refs, used): the pages in use moved to the lowest numbers.  Entries past a
    row's pages are -1."""
    new_table, new_refs = torch.full_like(table, -1), torch.empty_like(refs)
    used = torch.empty((1,), dtype=torch.int32, device=table.device)
    _on(stream, new_table, new_refs, used)
    bind_kv8_compact(caches, table, lens, refs, new_table, new_refs, used, workspace,
                     status)(pdl, stream)
    return new_table, new_refs, used


# ------------------------------------------------------------------ routing and logits
_TYPES = {torch.bfloat16: 0, torch.float32: 1}   # W4_TYPE_*


def _float_rows(t: torch.Tensor, name: str):
    """(W4_TYPE_*, row stride) of [rows, n] logits, dense within a row."""
    if not t.is_cuda or t.dtype not in _TYPES:
        raise ValueError(f"{name} must be a CUDA tensor of bfloat16 or float32")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [rows, n], each row dense")
    return _TYPES[t.dtype], t.stride(0) if t.shape[0] > 1 else t.shape[1]


class Router:
    """How tokens choose experts (struct w4_router): scores "softmax" or "sigmoid" of the logits;
    with groups > 1 only experts of the top_groups groups whose group_best largest scores sum
    highest; weights scale * score, divided by the chosen scores' sum with renorm."""

    def __init__(self, experts: int, top_k: int, groups: int = 1, top_groups: int = 1,
                 group_best: int = 2, score: str = "softmax", renorm: bool = True,
                 scale: float = 1.0):
        if score not in ("softmax", "sigmoid"):
            raise ValueError('score must be "softmax" or "sigmoid"')
        self.experts, self.top_k = experts, top_k
        self.struct = RouterStruct(experts, top_k, groups, top_groups, group_best,
                                   int(score == "sigmoid"), int(renorm), scale)


def bind_route(router: Router, logits: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
               bias: torch.Tensor = None, status: torch.Tensor = None):
    """w4_route with its arguments marshalled once: returns call(pdl=False, stream=None)."""
    kind, stride = _float_rows(logits, "logits")
    _need(ids, torch.int32, "ids")
    _need(weights, torch.float32, "weights")
    if logits.shape[1] != router.experts:
        raise ValueError("logits must be [rows, experts]")
    if tuple(ids.shape) != (logits.shape[0], router.top_k) or weights.shape != ids.shape:
        raise ValueError("ids and weights must be [rows, top_k]")
    if bias is not None:
        _need(bias, torch.float32, "bias")
        if bias.shape != (router.experts,):
            raise ValueError("bias must be [experts]")
    _same_device(logits, ids, weights, bias, status)
    args = (_ptr(ids), _ptr(weights), ctypes.byref(router.struct), _ptr(logits), kind, stride,
            _ptr(bias), logits.shape[0], _ptr(status))
    return _kv8_call(load().w4_route, "w4_route", args,
                     (logits, ids, weights, bias, status, router))


def route(router: Router, logits: torch.Tensor, bias: torch.Tensor = None,
          status: torch.Tensor = None, pdl: bool = False, stream=None):
    """(ids, weights): int32 and fp32 [rows, top_k], the experts of each row of logits [rows,
    experts] (bf16 or fp32), by score + bias."""
    shape = (logits.shape[0], router.top_k)
    ids = torch.empty(shape, dtype=torch.int32, device=logits.device)
    weights = torch.empty(shape, dtype=torch.float32, device=logits.device)
    _on(stream, ids, weights)
    bind_route(router, logits, ids, weights, bias, status)(pdl, stream)
    return ids, weights


def bind_moe_combine(y: torch.Tensor, weights: torch.Tensor, out: torch.Tensor,
                     add: torch.Tensor = None, ids: torch.Tensor = None, num_experts: int = 0,
                     status: torch.Tensor = None):
    """w4_moe_combine with its arguments marshalled once: returns call(pdl=False, stream=None)."""
    _need(y, torch.bfloat16, "y")
    _need(weights, torch.float32, "weights")
    _need(out, torch.bfloat16, "out")
    if y.dim() != 2 or weights.dim() != 2 or y.shape[0] != weights.numel() or \
            tuple(out.shape) != (weights.shape[0], y.shape[1]):
        raise ValueError("weights must be [rows, top_k], y [rows * top_k, N] and out [rows, N]")
    if add is not None:
        _need(add, torch.bfloat16, "add")
        if add.shape != out.shape:
            raise ValueError("add must be [rows, N]")
    if ids is not None:
        _need(ids, torch.int32, "ids")
        if ids.numel() != weights.numel():
            raise ValueError("ids must be [rows, top_k]")
    _same_device(y, weights, out, add, ids, status)
    args = (_ptr(out), _ptr(y), _ptr(weights), _ptr(ids), num_experts, _ptr(add),
            *weights.shape, y.shape[1], _ptr(status))
    return _kv8_call(load().w4_moe_combine, "w4_moe_combine", args,
                     (y, weights, out, add, ids, status))


def moe_combine(y: torch.Tensor, weights: torch.Tensor, out: torch.Tensor = None,
                add: torch.Tensor = None, ids: torch.Tensor = None, num_experts: int = 0,
                status: torch.Tensor = None, pdl: bool = False, stream=None) -> torch.Tensor:
    """out[t] = add[t] + sum_j weights[t, j] * y[t * top_k + j] (y as gemv_id writes it)."""
    if out is None:
        out = torch.empty((weights.shape[0], y.shape[1]), dtype=torch.bfloat16, device=y.device)
        _on(stream, out)
    bind_moe_combine(y, weights, out, add, ids, num_experts, status)(pdl, stream)
    return out


class LogitRules:
    """What w4_logits_adjust does to each row (struct w4_logit_rules); None where there is no such
    rule.

    tokens int32 [rows, max_tokens] with lens int32 [rows]: the histories; prompt int32 [rows]:
    how many of their tokens, from the first on, were the prompt.  repetition, presence,
    frequency: fp32 [rows].  bias_ids int32 and bias fp32 [rows, max_bias], n_bias int32 [rows]
    (None: all).  mask int32 or uint32 [masks, words]: bit v % 32 of word v / 32 allows token v;
    mask_rows int32 [rows]: each row's mask, -1: none (None: row b's is b).  The tensors may
    change between calls, in place."""

    def __init__(self, tokens: torch.Tensor = None, lens: torch.Tensor = None,
                 prompt: torch.Tensor = None, repetition: torch.Tensor = None,
                 presence: torch.Tensor = None, frequency: torch.Tensor = None,
                 bias_ids: torch.Tensor = None, bias: torch.Tensor = None,
                 n_bias: torch.Tensor = None, mask: torch.Tensor = None,
                 mask_rows: torch.Tensor = None):
        if (tokens is None) != (lens is None) or (bias_ids is None) != (bias is None):
            raise ValueError("tokens go with lens, and bias_ids with bias")
        per_row = (("lens", lens, torch.int32), ("prompt", prompt, torch.int32),
                   ("repetition", repetition, torch.float32),
                   ("presence", presence, torch.float32),
                   ("frequency", frequency, torch.float32), ("n_bias", n_bias, torch.int32),
                   ("mask_rows", mask_rows, torch.int32))
        for name, t, dtype in per_row:
            if t is not None:
                _need(t, dtype, name)
                if t.dim() != 1:
                    raise ValueError(f"{name} must be [rows]")
        lists = (("tokens", tokens, (torch.int32,)), ("bias_ids", bias_ids, (torch.int32,)),
                 ("bias", bias, (torch.float32,)), ("mask", mask, (torch.int32, torch.uint32)))
        strides, widths = {}, {}
        for name, t, dtypes in lists:
            strides[name] = widths[name] = 0
            if t is None:
                continue
            if not t.is_cuda or t.dtype not in dtypes or t.dim() != 2 or \
                    (t.shape[1] > 1 and t.stride(1) != 1):
                raise ValueError(f"{name} must be a CUDA tensor [rows, n] of {dtypes[0]}, each "
                                 "row dense")
            widths[name] = t.shape[1]
            strides[name] = t.stride(0) if t.shape[0] > 1 else t.shape[1]
        if bias is not None and (bias.shape != bias_ids.shape or
                                 strides["bias"] != strides["bias_ids"]):
            raise ValueError("bias_ids and bias must have the same shape and row stride")
        self.row_counts = {t.shape[0] for t in (tokens, bias_ids, *(t for _, t, _ in per_row))
                           if t is not None}
        self.words = widths["mask"]
        self.masks = 0 if mask is None else mask.shape[0]
        self.per_row_mask = mask is not None and mask_rows is None
        self.tensors = (tokens, lens, prompt, repetition, presence, frequency, bias_ids, bias,
                        n_bias, mask, mask_rows)
        # a list of no columns has no address, and a null one would say that there is no such rule: its
        # counts' stands for it, since nothing is read there
        def place(t, counts):
            t = counts if t is not None and t.dim() == 2 and t.shape[1] == 0 else t
            return None if t is None else t.data_ptr()

        self.struct = LogitRulesStruct(place(tokens, lens),
                                       *[place(t, None) for t in self.tensors[1:6]],
                                       place(bias_ids, n_bias), place(bias, n_bias),
                                       *[place(t, None) for t in self.tensors[8:]],
                                       strides["tokens"], strides["bias"], strides["mask"],
                                       widths["tokens"], widths["bias"], self.masks)


def bind_adjust_logits(logits: torch.Tensor, rules: LogitRules, status: torch.Tensor = None):
    """w4_logits_adjust with its arguments marshalled once: returns call(pdl=False,
    stream=None)."""
    kind, stride = _float_rows(logits, "logits")
    rows, V = logits.shape
    if rules.row_counts - {rows}:
        raise ValueError(f"the rules are for {sorted(rules.row_counts)} rows, the logits have {rows}")
    if rules.masks and rules.words < (V + 31) // 32:
        raise ValueError("mask must hold a bit for each token")
    if rules.per_row_mask and rules.masks < rows:
        raise ValueError("mask must have a row for each row of logits")
    _same_device(logits, *rules.tensors, status)
    args = (_ptr(logits), kind, stride, rows, V, ctypes.byref(rules.struct), _ptr(status))
    return _kv8_call(load().w4_logits_adjust, "w4_logits_adjust", args, (logits, rules, status))


def adjust_logits(logits: torch.Tensor, rules: LogitRules, status: torch.Tensor = None,
                  pdl: bool = False, stream=None) -> torch.Tensor:
    """Penalties for repeated tokens, biases and masks on logits [rows, V] (bf16 or fp32), in
    place."""
    bind_adjust_logits(logits, rules, status)(pdl, stream)
    return logits
