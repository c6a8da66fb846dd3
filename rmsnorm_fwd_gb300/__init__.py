"""Row-wise RMSNorm forward for GB300 (sm_103a): hand-written CUDA kernels
behind the C ABI of ``include/rmsnorm.h`` (``librmsnorm.so``).

This module is the thin Python binding: the functions below have the C
names and only marshal arguments (pointers, sizes, the stream handle) into
the library.  Every step of the computation runs in the library's kernels;
there is no Python, PyTorch or CPU fallback.  If the library cannot be built
or loaded, the first call raises.

PyTorch is used only for device memory and streams (``rms_norm`` takes
tensors, reads their data pointers and the current stream, and calls
``rmsnorm_fwd``).
"""
from __future__ import annotations

import ctypes
import functools
import struct
import threading

# element types (rmsnorm_dtype_t)
F32, BF16, F16 = 0, 1, 2
DTYPE_NAMES = {F32: "f32", BF16: "bf16", F16: "f16"}
DTYPE_CODES = {"f32": F32, "bf16": BF16, "f16": F16}

# status codes (rmsnorm_status_t)
OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED_DTYPE = 2
ERR_NOT_INITIALIZED = 3
ERR_ALIASING = 4
ERR_CUDA = 5
ERR_DEVICE_TIMEOUT = 6
ERR_MISALIGNED = 7
ERR_UNSUPPORTED_DEVICE = 8
ERR_VARIANT = 9
ERR_TOO_LARGE = 10
ERR_BAD_INDEX = 11

# variants (rmsnorm_variant_t)
VARIANT_AUTO = 0
VARIANT_WARP_PER_ROW = 1
VARIANT_CTA_PER_ROW = 2
VARIANT_STAGED = 3
VARIANT_PERSISTENT = 4
VARIANT_GENERIC = 5
VARIANT_CLUSTER = 6
VARIANT_GRID = 7
VARIANT_NAMES = {0: "auto", 1: "warp_per_row", 2: "cta_per_row", 3: "staged", 4: "persistent",
                 5: "generic", 6: "cluster", 7: "grid"}

# epilogues (rmsnorm_epilogue_t)
EPI_PLAIN, EPI_BIAS, EPI_MXFP8, EPI_MXFP4, EPI_NVFP4 = 0, 1, 2, 3, 4
EPI_NAMES = {EPI_PLAIN: "plain", EPI_BIAS: "bias", EPI_MXFP8: "mxfp8", EPI_MXFP4: "mxfp4",
             EPI_NVFP4: "nvfp4"}
EPI_CODES = {v: k for k, v in EPI_NAMES.items()}
# block-scaled outputs: (elements per scale block, bits per element code)
QUANT_FORMATS = {EPI_MXFP8: (32, 8), EPI_MXFP4: (32, 4), EPI_NVFP4: (16, 4)}


class RmsnormError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({rmsnorm_status_string(status)})")


class Plan(ctypes.Structure):
    """rmsnorm_plan_t."""
    _fields_ = [(name, ctypes.c_int32) for name in (
        "variant", "vec_bytes", "threads_per_row", "vecs_per_thread", "block_threads",
        "rows_per_block", "stages", "grid", "smem_bytes", "kernel_index")]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class QkPlan(ctypes.Structure):
    """rmsnorm_qk_plan_t."""
    _fields_ = [(name, ctypes.c_int32) for name in (
        "lanes_per_head", "vecs_per_lane", "heads_per_group", "grid")]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class KernelInfo(ctypes.Structure):
    """rmsnorm_kernel_info_t."""
    _fields_ = [(name, ctypes.c_int32) for name in (
        "variant", "dtype", "vec_bytes", "tpr", "nv", "block", "min_blocks", "cache_policy",
        "epilogue")]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class Heads(ctypes.Structure):
    """rmsnorm_heads_t."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class Rope(ctypes.Structure):
    """rmsnorm_rope_t."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("max_position", ctypes.c_int64), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class PagedCache(ctypes.Structure):
    """rmsnorm_paged_cache_t."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("e4m3", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    from . import _build
    return _build.LIB


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        from . import _build
        path = _build.build()  # compiles in-tree if stale; raises if nvcc is missing
        lib = ctypes.CDLL(path, mode=ctypes.RTLD_GLOBAL)
        vp, i64, i32, f32, u64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                                  ctypes.c_uint64)
        pp = ctypes.POINTER(Plan)
        # pointers to rmsnorm_heads_t, rmsnorm_rope_t, rmsnorm_paged_cache_t: addresses or byref()
        hp = rp = cp = vp
        szp = ctypes.POINTER(ctypes.c_size_t)
        sig = {
            "rmsnorm_create": ([], i32),
            "rmsnorm_destroy": ([], i32),
            "rmsnorm_fwd": ([vp, vp, vp, i64, i64, f32, i32, vp], i32),
            "rmsnorm_fwd_ex": ([vp, vp, vp, i64, i64, f32, i32, vp, i32, pp], i32),
            "rmsnorm_plan": ([vp, vp, vp, i64, i64, i32, i32, i32, i32, pp], i32),
            "rmsnorm_plan_host_mapped": ([vp, vp, vp, i64, i64, i32, i32, i32, pp], i32),
            "rmsnorm_fwd_host": ([vp, vp, vp, i64, i64, f32, i32, vp, ctypes.c_size_t, i64, vp],
                                 i32),
            "rmsnorm_qk_norm": ([vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, f32, f32, i32, vp],
                                i32),
            "rmsnorm_qk_norm_ex": ([vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, f32, f32, i32, vp,
                                    ctypes.POINTER(QkPlan)], i32),
            "rmsnorm_fwd_bias": ([vp, vp, vp, i64, i64, f32, f32, i32, vp], i32),
            "rmsnorm_fwd_mxfp8": ([vp, vp, vp, vp, i64, i64, f32, f32, i32, vp], i32),
            "rmsnorm_fwd_mxfp4": ([vp, vp, vp, vp, i64, i64, f32, f32, i32, vp], i32),
            "rmsnorm_fwd_nvfp4": ([vp, vp, vp, vp, i64, i64, f32, f32, f32, i32, vp], i32),
            "rmsnorm_fwd_epilogue_ex": ([vp, vp, vp, vp, i64, i64, i32, f32, f32, f32, i32, vp,
                                         i32, pp], i32),
            "rmsnorm_plan_epilogue": ([vp, vp, vp, i64, i64, i32, i32, i32, i32, i32, pp], i32),
            "rmsnorm_validate_plan_epilogue": ([pp, vp, vp, vp, i64, i64, i32, i32, i32, i32],
                                               i32),
            "rmsnorm_qk_norm_rope": ([hp, hp, hp, hp, vp, vp, rp, i64, i64, i64, i64, f32, f32,
                                      i32, vp], i32),
            "rmsnorm_qk_norm_rope_bwd": ([hp, hp, hp, hp, hp, hp, vp, vp, vp, vp, rp, vp,
                                          ctypes.c_size_t, i64, i64, i64, i64, f32, f32, i32,
                                          vp], i32),
            "rmsnorm_qk_norm_rope_bwd_workspace": ([i64, i32, szp], i32),
            "rmsnorm_qk_norm_rope_append": ([hp, hp, hp, hp, vp, vp, rp, cp, vp, i64, i64, i64, i64,
                                             f32, f32, i32, vp], i32),
            "rmsnorm_bwd": ([vp, vp, vp, vp, vp, vp, ctypes.c_size_t, i64, i64, f32, f32, i32,
                             vp], i32),
            "rmsnorm_bwd_workspace": ([i64, i64, i32, i32, szp], i32),
            "rmsnorm_last_variant": ([], i32),
            "rmsnorm_kernel_count": ([], i32),
            "rmsnorm_validate_plan": ([pp, vp, vp, vp, i64, i64, i32, i32, i32], i32),
            "rmsnorm_device_limits": ([ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)],
                                      i32),
            "rmsnorm_kernel_info": ([i32, ctypes.POINTER(KernelInfo)], i32),
            "rmsnorm_get_device_status": ([ctypes.POINTER(ctypes.c_int)], i32),
            "rmsnorm_set_wait_limit_ns": ([u64], i32),
            "rmsnorm_set_pdl": ([i32], i32),
            "rmsnorm_get_pdl": ([], i32),
            "rmsnorm_test_staged_timeout": ([vp, vp, vp, i64, i64, i32, u64, vp], i32),
            "rmsnorm_test_grid_timeout": ([vp, vp, vp, i64, i64, i32, u64, vp], i32),
            "rmsnorm_fwd_staged_noalloc": ([vp, vp, vp, i64, i64, f32, i32, vp], i32),
            "rmsnorm_test_staged_noalloc_timeout": ([vp, vp, vp, i64, i64, i32, u64, vp], i32),
            "rmsnorm_noalloc_block_status": ([ctypes.POINTER(ctypes.c_int), i32], i32),
            "rmsnorm_status_string": ([i32], ctypes.c_char_p),
            "rmsnorm_version": ([], i32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _check(rc: int, where: str) -> None:
    if rc != OK:
        raise RmsnormError(rc, where)


# ------------------------------------------------------------------ C names

def rmsnorm_create() -> None:
    _check(_load().rmsnorm_create(), "rmsnorm_create")


def rmsnorm_destroy() -> None:
    _check(_load().rmsnorm_destroy(), "rmsnorm_destroy")


def rmsnorm_fwd(x: int, weight: int, y: int, rows: int, hidden: int, eps: float, dtype: int,
                stream: int | None) -> None:
    """Raw call: device pointers as integers, stream as a cudaStream_t integer."""
    _check(_load().rmsnorm_fwd(x, weight, y, rows, hidden, eps, dtype, stream or None),
           "rmsnorm_fwd")


def rmsnorm_fwd_ex(x: int, weight: int, y: int, rows: int, hidden: int, eps: float, dtype: int,
                   stream: int | None, variant: int = VARIANT_AUTO,
                   plan: Plan | None = None) -> Plan | None:
    ref = ctypes.byref(plan) if plan is not None else None
    _check(_load().rmsnorm_fwd_ex(x, weight, y, rows, hidden, eps, dtype, stream or None,
                                  variant, ref), "rmsnorm_fwd_ex")
    return plan


def rmsnorm_fwd_host(x_host: int, weight: int, y_host: int, rows: int, hidden: int, eps: float,
                     dtype: int, workspace: int, workspace_bytes: int, chunk_rows: int,
                     stream: int | None) -> None:
    """Host-buffer call: host x/y (pinned for overlap), device weight and
    workspace, chunked upload / kernel / download pipeline."""
    _check(_load().rmsnorm_fwd_host(x_host, weight, y_host, rows, hidden, eps, dtype, workspace,
                                    workspace_bytes, chunk_rows, stream or None),
           "rmsnorm_fwd_host")


def rmsnorm_qk_norm(q: int, k: int, q_weight: int, k_weight: int, tokens: int, q_heads: int,
                    k_heads: int, head_dim: int, q_token_stride: int, k_token_stride: int,
                    weight_bias: float, eps: float, dtype: int, stream: int | None) -> None:
    """Per-head QK norm in place (device pointers as integers)."""
    _check(_load().rmsnorm_qk_norm(q or None, k or None, q_weight or None, k_weight or None,
                                   tokens, q_heads, k_heads, head_dim, q_token_stride,
                                   k_token_stride, weight_bias, eps, dtype, stream or None),
           "rmsnorm_qk_norm")


def rmsnorm_qk_norm_ex(q: int, k: int, q_weight: int, k_weight: int, tokens: int, q_heads: int,
                       k_heads: int, head_dim: int, q_token_stride: int, k_token_stride: int,
                       weight_bias: float, eps: float, dtype: int, stream: int | None,
                       plan: QkPlan | None = None) -> QkPlan | None:
    _check(_load().rmsnorm_qk_norm_ex(q or None, k or None, q_weight or None, k_weight or None,
                                      tokens, q_heads, k_heads, head_dim, q_token_stride,
                                      k_token_stride, weight_bias, eps, dtype, stream or None,
                                      ctypes.byref(plan) if plan is not None else None),
           "rmsnorm_qk_norm_ex")
    return plan


def qk_norm(q, k, q_weight, k_weight, head_dim: int, eps: float, weight_bias: float = 0.0,
            stream=None) -> None:
    """In-place per-head norm of PyTorch CUDA tensors q [..., q_heads * head_dim]
    and k [..., k_heads * head_dim] (the last dimension holds a token's heads;
    the token dimension may be strided, e.g. views into a fused QKV tensor)."""
    import torch
    for t in (q, k):
        if not t.is_cuda or t.stride(-1) != 1:
            raise ValueError("q and k must be CUDA tensors with a contiguous last dimension")
    tokens = q.numel() // q.shape[-1]
    if k.numel() // k.shape[-1] != tokens:
        raise ValueError("q and k must hold the same number of tokens")
    qs = q.stride(-2) if q.dim() > 1 else q.shape[-1]
    ks = k.stride(-2) if k.dim() > 1 else k.shape[-1]
    ensure_context(q.device.index)
    s = stream if stream is not None else torch.cuda.current_stream(q.device)
    with torch.cuda.device(q.device.index):
        rmsnorm_qk_norm(q.data_ptr(), k.data_ptr(), q_weight.data_ptr(), k_weight.data_ptr(),
                        tokens, q.shape[-1] // head_dim, k.shape[-1] // head_dim, head_dim, qs, ks,
                        float(weight_bias), float(eps), torch_dtype_code(q.dtype), s.cuda_stream)


def rmsnorm_fwd_bias(x: int, weight: int, y: int, rows: int, hidden: int, weight_bias: float,
                     eps: float, dtype: int, stream: int | None) -> None:
    _check(_load().rmsnorm_fwd_bias(x, weight, y, rows, hidden, weight_bias, eps, dtype,
                                    stream or None), "rmsnorm_fwd_bias")


def rmsnorm_fwd_mxfp8(x: int, weight: int, q: int, scales: int, rows: int, hidden: int,
                      weight_bias: float, eps: float, dtype: int, stream: int | None) -> None:
    _check(_load().rmsnorm_fwd_mxfp8(x, weight, q, scales, rows, hidden, weight_bias, eps, dtype,
                                     stream or None), "rmsnorm_fwd_mxfp8")


def rmsnorm_fwd_mxfp4(x: int, weight: int, q: int, scales: int, rows: int, hidden: int,
                      weight_bias: float, eps: float, dtype: int, stream: int | None) -> None:
    _check(_load().rmsnorm_fwd_mxfp4(x, weight, q, scales, rows, hidden, weight_bias, eps, dtype,
                                     stream or None), "rmsnorm_fwd_mxfp4")


def rmsnorm_fwd_nvfp4(x: int, weight: int, q: int, scales: int, rows: int, hidden: int,
                      global_scale: float, weight_bias: float, eps: float, dtype: int,
                      stream: int | None) -> None:
    _check(_load().rmsnorm_fwd_nvfp4(x, weight, q, scales, rows, hidden, global_scale,
                                     weight_bias, eps, dtype, stream or None), "rmsnorm_fwd_nvfp4")


def rmsnorm_fwd_epilogue_ex(x: int, weight: int, y: int, scales: int | None, rows: int,
                            hidden: int, epilogue: int, weight_bias: float, eps: float,
                            dtype: int, stream: int | None, variant: int = VARIANT_AUTO,
                            plan: Plan | None = None, global_scale: float = 1.0) -> None:
    _check(_load().rmsnorm_fwd_epilogue_ex(x, weight, y, scales or None, rows, hidden, epilogue,
                                           weight_bias, global_scale, eps, dtype, stream or None,
                                           variant,
                                           ctypes.byref(plan) if plan is not None else None),
           "rmsnorm_fwd_epilogue_ex")


def rmsnorm_plan_epilogue_status(x: int, weight: int, y: int, rows: int, hidden: int, dtype: int,
                                 epilogue: int, sm_count: int, smem_optin: int,
                                 variant: int = VARIANT_AUTO):
    """(status, plan) of the selector for an epilogue, without raising."""
    p = Plan()
    rc = _load().rmsnorm_plan_epilogue(x, weight, y, rows, hidden, dtype, epilogue, sm_count,
                                       smem_optin, variant, ctypes.byref(p))
    return rc, p


def rmsnorm_validate_plan_epilogue(plan: Plan, x: int, weight: int, y: int, rows: int,
                                   hidden: int, dtype: int, epilogue: int, sm_count: int,
                                   smem_optin: int) -> int:
    return _load().rmsnorm_validate_plan_epilogue(ctypes.byref(plan), x, weight, y, rows, hidden,
                                                  dtype, epilogue, sm_count, smem_optin)


def _ref(structure):
    return None if structure is None else ctypes.byref(structure)


def rmsnorm_qk_norm_rope(q: Heads | None, k: Heads | None, q_out: Heads | None,
                         k_out: Heads | None, q_weight: int, k_weight: int, rope: Rope,
                         tokens: int, q_heads: int, k_heads: int, head_dim: int,
                         weight_bias: float, eps: float, dtype: int,
                         stream: int | None) -> None:
    """Per-head QK norm and position rotation (structures with device pointers)."""
    _check(_load().rmsnorm_qk_norm_rope(_ref(q), _ref(k), _ref(q_out), _ref(k_out),
                                        q_weight or None, k_weight or None, _ref(rope), tokens,
                                        q_heads, k_heads, head_dim, weight_bias, eps, dtype,
                                        stream or None), "rmsnorm_qk_norm_rope")


def rmsnorm_qk_norm_rope_bwd(dq_out: Heads | None, dk_out: Heads | None, q: Heads | None,
                             k: Heads | None, dq: Heads | None, dk: Heads | None, q_weight: int,
                             k_weight: int, dq_weight: int, dk_weight: int, rope: Rope,
                             workspace: int, workspace_bytes: int, tokens: int, q_heads: int,
                             k_heads: int, head_dim: int, weight_bias: float, eps: float,
                             dtype: int, stream: int | None) -> None:
    _check(_load().rmsnorm_qk_norm_rope_bwd(_ref(dq_out), _ref(dk_out), _ref(q), _ref(k),
                                            _ref(dq), _ref(dk), q_weight or None,
                                            k_weight or None, dq_weight or None,
                                            dk_weight or None, _ref(rope), workspace or None,
                                            workspace_bytes, tokens, q_heads, k_heads, head_dim,
                                            weight_bias, eps, dtype, stream or None),
           "rmsnorm_qk_norm_rope_bwd")


def rmsnorm_qk_norm_rope_bwd_workspace(head_dim: int, sm_count: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_load().rmsnorm_qk_norm_rope_bwd_workspace(head_dim, sm_count, ctypes.byref(n)),
           "rmsnorm_qk_norm_rope_bwd_workspace")
    return n.value


def rmsnorm_qk_norm_rope_append(q: Heads | None, k: Heads, v: Heads, q_out: Heads | None,
                                q_weight: int, k_weight: int, rope: Rope, cache: PagedCache,
                                slots: int, tokens: int, q_heads: int, k_heads: int,
                                head_dim: int, weight_bias: float, eps: float, dtype: int,
                                stream: int | None) -> None:
    _check(_load().rmsnorm_qk_norm_rope_append(_ref(q), _ref(k), _ref(v), _ref(q_out),
                                               q_weight or None, k_weight or None, _ref(rope),
                                               _ref(cache), slots or None, tokens, q_heads,
                                               k_heads, head_dim, weight_bias, eps, dtype,
                                               stream or None), "rmsnorm_qk_norm_rope_append")


def rmsnorm_bwd(dy: int, x: int, weight: int, dx: int, dweight: int, workspace: int,
                workspace_bytes: int, rows: int, hidden: int, weight_bias: float, eps: float,
                dtype: int, stream: int | None) -> None:
    _check(_load().rmsnorm_bwd(dy or None, x or None, weight or None, dx or None,
                               dweight or None, workspace or None, workspace_bytes, rows, hidden,
                               weight_bias, eps, dtype, stream or None), "rmsnorm_bwd")


def rmsnorm_bwd_workspace(rows: int, hidden: int, dtype: int, sm_count: int) -> int:
    n = ctypes.c_size_t(0)
    _check(_load().rmsnorm_bwd_workspace(rows, hidden, dtype, sm_count, ctypes.byref(n)),
           "rmsnorm_bwd_workspace")
    return n.value


def rmsnorm_plan(x: int, weight: int, y: int, rows: int, hidden: int, dtype: int, sm_count: int,
                 smem_optin: int, variant: int = VARIANT_AUTO) -> Plan:
    p = Plan()
    _check(_load().rmsnorm_plan(x, weight, y, rows, hidden, dtype, sm_count, smem_optin, variant,
                                ctypes.byref(p)), "rmsnorm_plan")
    return p


def rmsnorm_plan_status(x: int, weight: int, y: int, rows: int, hidden: int, dtype: int,
                        sm_count: int, smem_optin: int, variant: int = VARIANT_AUTO):
    """(status, plan) without raising."""
    p = Plan()
    rc = _load().rmsnorm_plan(x, weight, y, rows, hidden, dtype, sm_count, smem_optin, variant,
                              ctypes.byref(p))
    return rc, p


def rmsnorm_plan_host_mapped_status(x_host: int, weight: int, y_host: int, rows: int,
                                    hidden: int, dtype: int, sm_count: int, smem_optin: int):
    """(status, plan) of rmsnorm_fwd_host's page-locked path, without raising."""
    p = Plan()
    rc = _load().rmsnorm_plan_host_mapped(x_host, weight, y_host, rows, hidden, dtype, sm_count,
                                          smem_optin, ctypes.byref(p))
    return rc, p


def rmsnorm_device_limits() -> tuple[int, int]:
    """(SM count, opt-in shared memory per block) of the current device."""
    a, b = ctypes.c_int(0), ctypes.c_int(0)
    _check(_load().rmsnorm_device_limits(ctypes.byref(a), ctypes.byref(b)),
           "rmsnorm_device_limits")
    return a.value, b.value


def rmsnorm_validate_plan(plan: Plan, x: int, weight: int, y: int, rows: int, hidden: int,
                          dtype: int, sm_count: int, smem_optin: int) -> int:
    """Status rmsnorm_fwd_ex would give this explicit plan (host only)."""
    return _load().rmsnorm_validate_plan(ctypes.byref(plan), x, weight, y, rows, hidden, dtype,
                                         sm_count, smem_optin)


def rmsnorm_kernel_count() -> int:
    return _load().rmsnorm_kernel_count()


def rmsnorm_kernel_info(index: int) -> KernelInfo:
    k = KernelInfo()
    _check(_load().rmsnorm_kernel_info(index, ctypes.byref(k)), "rmsnorm_kernel_info")
    return k


def kernels() -> list[dict]:
    """Every compiled instantiation, with its index."""
    return [dict(index=i, **rmsnorm_kernel_info(i).as_dict()) for i in range(rmsnorm_kernel_count())]


def rmsnorm_last_variant() -> int:
    return _load().rmsnorm_last_variant()


def rmsnorm_get_device_status() -> int:
    v = ctypes.c_int(0)
    _check(_load().rmsnorm_get_device_status(ctypes.byref(v)), "rmsnorm_get_device_status")
    return v.value


def rmsnorm_set_wait_limit_ns(limit_ns: int) -> None:
    _check(_load().rmsnorm_set_wait_limit_ns(limit_ns), "rmsnorm_set_wait_limit_ns")


def rmsnorm_set_pdl(enable: bool) -> None:
    _check(_load().rmsnorm_set_pdl(1 if enable else 0), "rmsnorm_set_pdl")


def rmsnorm_get_pdl() -> bool:
    return bool(_load().rmsnorm_get_pdl())


def rmsnorm_test_staged_timeout(x: int, weight: int, y: int, rows: int, hidden: int, dtype: int,
                                limit_ns: int, stream: int | None) -> None:
    _check(_load().rmsnorm_test_staged_timeout(x, weight, y, rows, hidden, dtype, limit_ns,
                                               stream or None), "rmsnorm_test_staged_timeout")


def rmsnorm_test_grid_timeout(x: int, weight: int, y: int, rows: int, hidden: int, dtype: int,
                              limit_ns: int, stream: int | None) -> None:
    _check(_load().rmsnorm_test_grid_timeout(x, weight, y, rows, hidden, dtype, limit_ns,
                                             stream or None), "rmsnorm_test_grid_timeout")


def rmsnorm_fwd_staged_noalloc(x: int, weight: int, y: int, rows: int, hidden: int, eps: float,
                               dtype: int, stream: int | None) -> None:
    """The allocation-free entry point (no context, no device allocation):
    device pointers as integers, stream as a cudaStream_t integer."""
    _check(_load().rmsnorm_fwd_staged_noalloc(x, weight, y, rows, hidden, eps, dtype,
                                              stream or None), "rmsnorm_fwd_staged_noalloc")


def rmsnorm_test_staged_noalloc_timeout(x: int, weight: int, y: int, rows: int, hidden: int,
                                        dtype: int, limit_ns: int, stream: int | None) -> None:
    _check(_load().rmsnorm_test_staged_noalloc_timeout(x, weight, y, rows, hidden, dtype,
                                                       limit_ns, stream or None),
           "rmsnorm_test_staged_noalloc_timeout")


def rmsnorm_noalloc_block_status(n: int) -> list[int]:
    """The first n words of the allocation-free entry point's static status
    array (one per block of its last launch)."""
    buf = (ctypes.c_int * max(n, 1))()
    _check(_load().rmsnorm_noalloc_block_status(buf, n), "rmsnorm_noalloc_block_status")
    return list(buf[:n])


def rmsnorm_status_string(status: int) -> str:
    return _load().rmsnorm_status_string(status).decode()


def rmsnorm_version() -> int:
    return _load().rmsnorm_version()


# ------------------------------------------------------------------ tensors

_created = set()


def ensure_context(device_index: int) -> None:
    """rmsnorm_create on `device_index` once per process."""
    if device_index in _created:
        return
    import torch
    with torch.cuda.device(device_index):
        rmsnorm_create()
    _created.add(device_index)


def torch_dtype_code(dt) -> int:
    import torch
    table = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
    if dt not in table:
        raise TypeError(f"unsupported dtype {dt}")
    return table[dt]


def rms_norm(x, weight, eps: float, out=None, variant: int = VARIANT_AUTO, plan: Plan | None = None,
             stream=None):
    """y = x * rsqrt(mean(x^2, -1) + eps) * weight through rmsnorm_fwd_ex.

    ``x``: CUDA tensor [..., hidden], contiguous; ``weight``: [hidden], same
    dtype and device; ``out``: optional preallocated output (may be ``x``).
    Runs on ``stream`` (default: PyTorch's current stream)."""
    import torch
    if not (x.is_cuda and weight.is_cuda):
        raise ValueError("rms_norm takes CUDA tensors (there is no CPU path)")
    if x.dtype != weight.dtype:
        raise TypeError("x and weight must share a dtype")
    if not x.is_contiguous() or not weight.is_contiguous():
        raise ValueError("x and weight must be contiguous")
    hidden = x.shape[-1]
    if weight.numel() != hidden:
        raise ValueError("weight must have hidden elements")
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
        raise ValueError("out must match x (shape, dtype, contiguous)")
    ensure_context(x.device.index)
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    rows = x.numel() // hidden if hidden else 0
    with torch.cuda.device(x.device.index):
        rmsnorm_fwd_ex(x.data_ptr(), weight.data_ptr(), out.data_ptr(), rows, hidden, float(eps),
                       torch_dtype_code(x.dtype), s.cuda_stream, variant, plan)
    return out


def rms_norm_bias(x, weight, weight_bias: float, eps: float, out=None, variant: int = VARIANT_AUTO,
                  plan: Plan | None = None, stream=None):
    """y = x * rsqrt(mean(x^2, -1) + eps) * (weight + weight_bias) through
    rmsnorm_fwd_epilogue_ex (tensors as for ``rms_norm``)."""
    import torch
    _check_rows(x, weight)
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
        raise ValueError("out must match x (shape, dtype, contiguous)")
    ensure_context(x.device.index)
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden else 0
    with torch.cuda.device(x.device.index):
        rmsnorm_fwd_epilogue_ex(x.data_ptr(), weight.data_ptr(), out.data_ptr(), None, rows, hidden,
                                EPI_BIAS, float(weight_bias), float(eps),
                                torch_dtype_code(x.dtype), s.cuda_stream, variant, plan, 1.0)
    return out


def rms_norm_quant(x, weight, eps: float, fmt: str = "mxfp8", weight_bias: float = -0.0,
                   global_scale: float = 1.0, out=None, scales=None,
                   variant: int = VARIANT_AUTO, plan: Plan | None = None, stream=None):
    """RMSNorm with a block-scaled output, fmt "mxfp8" | "mxfp4" | "nvfp4":
    (codes uint8 [..., hidden * bits / 8] -- E4M3 bytes, or two E2M1 codes per
    byte with the even element in the low nibble -- and scales uint8
    [..., hidden / block] -- E8M0 exponents, or E4M3 values for NVFP4, which
    stand for code * scale * global_scale)."""
    import torch
    _check_rows(x, weight)
    epi = EPI_CODES[fmt]
    block, bits = QUANT_FORMATS[epi]
    hidden = x.shape[-1]
    if hidden % block:
        raise ValueError(f"hidden must be a multiple of {block} for {fmt}")
    lead = tuple(x.shape[:-1])
    if out is None:
        out = torch.empty(lead + (hidden * bits // 8,), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(lead + (hidden // block,), dtype=torch.uint8, device=x.device)
    if out.dtype != torch.uint8 or out.numel() * 8 != x.numel() * bits or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous uint8 tensor of x.numel() * {bits} / 8 bytes")
    if scales.dtype != torch.uint8 or scales.numel() * block != x.numel() or \
            not scales.is_contiguous():
        raise ValueError(f"scales must be a contiguous uint8 tensor of x.numel() / {block} bytes")
    ensure_context(x.device.index)
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    rows = x.numel() // hidden if hidden else 0
    with torch.cuda.device(x.device.index):
        rmsnorm_fwd_epilogue_ex(x.data_ptr(), weight.data_ptr(), out.data_ptr(), scales.data_ptr(),
                                rows, hidden, epi, float(weight_bias), float(eps),
                                torch_dtype_code(x.dtype), s.cuda_stream, variant, plan,
                                float(global_scale))
    return out, scales


def rms_norm_mxfp8(x, weight, eps: float, weight_bias: float = -0.0, out=None, scales=None,
                   variant: int = VARIANT_AUTO, plan: Plan | None = None, stream=None):
    """RMSNorm with an MXFP8 output: (codes uint8 [..., hidden] holding E4M3
    bit patterns, scales uint8 [..., hidden / 32] holding E8M0 exponents)."""
    return rms_norm_quant(x, weight, eps, "mxfp8", weight_bias, 1.0, out, scales, variant, plan,
                          stream)


def _check_rows(x, weight):
    if not (x.is_cuda and weight.is_cuda):
        raise ValueError("CUDA tensors required (there is no CPU path)")
    if x.dtype != weight.dtype:
        raise TypeError("x and weight must share a dtype")
    if not x.is_contiguous() or not weight.is_contiguous():
        raise ValueError("x and weight must be contiguous")
    if weight.numel() != x.shape[-1]:
        raise ValueError("weight must have hidden elements")


# The structures of a call as bytes: ctypes hands the library their address
# (read during the call only), at a third of the time that building ctypes
# structures takes, which a decode step would notice.
_HEADS = struct.Struct("@Pqq")          # rmsnorm_heads_t
_ROPE = struct.Struct("@PPqii")         # rmsnorm_rope_t
_CACHE = struct.Struct("@PPqqqqqiff0q")  # rmsnorm_paged_cache_t, padded to its end


def _here(device, stream) -> bool:
    """Whether a call on `device` and `stream` (None: the current one) runs as
    things stand; else the caller calls itself again inside _there().  Short
    calls pay for every microsecond on the host."""
    import torch
    if device.index not in _created:
        ensure_context(device.index)
    return stream is None and torch.cuda.current_device() == device.index


def _there(device, stream, *tensors):
    """The context in which `stream` (and its device), or `device`, is current.
    Tensors made in it belong to that stream; `tensors` are used on it."""
    import torch
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError("stream must be on the device of the tensors")
    for t in tensors:  # their memory is not given out again before `stream` is done with it
        if t is not None:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _stream(device) -> int:
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


@functools.lru_cache(maxsize=None)
def _sm_count(index: int) -> int:
    """SM count of the current device, `index` (one that has a context)."""
    return rmsnorm_device_limits()[0]


@functools.lru_cache(maxsize=256)
def _heads_workspace(head_dim: int, sms: int) -> int:
    return rmsnorm_qk_norm_rope_bwd_workspace(head_dim, sms)


@functools.lru_cache(maxsize=1024)
def _rows_workspace(rows: int, hidden: int, code: int, sms: int) -> int:
    return rmsnorm_bwd_workspace(rows, hidden, code, sms)


def _heads(t, name: str, dtype, device) -> tuple[bytes, int]:
    """(rmsnorm_heads_t, tokens) of a CUDA tensor [..., heads, head_dim] whose
    leading dimensions step evenly over the tokens."""
    if t is None or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype is not dtype or t.device != device:
        raise TypeError(f"{name} must have the dtype and device of the other tensors")
    shape = t.shape
    if len(shape) == 3 and t.is_contiguous():
        return _HEADS.pack(t.data_ptr(), 0, 0), shape[0]
    strides = t.stride()
    if len(shape) == 3:
        tokens, heads, dim = shape
        step, head_step, last = strides
        if tokens == 1:
            step = 0
    elif len(shape) > 3:
        heads, dim = shape[-2:]
        head_step, last = strides[-2:]
        tokens, step = 1, 0
        for n, s in zip(shape[-3::-1], strides[-3::-1]):
            if n != 1:
                if tokens == 1:
                    step = s
                elif s != step * tokens and t.numel():
                    raise ValueError(f"the leading dimensions of {name} must step evenly")
                tokens *= n
    else:
        raise ValueError(f"{name} must be [..., tokens, heads, head_dim]")
    if last != 1 and dim > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if heads == 1:
        head_step = 0
    elif head_step == 0:
        raise ValueError(f"{name} must not be an expanded tensor")
    if step == 0 and tokens > 1:
        raise ValueError(f"{name} must not be an expanded tensor")
    return _HEADS.pack(t.data_ptr(), step, head_step), tokens


_NO_ROPE = _ROPE.pack(0, 0, 0, 0, 0)


def _rope(cos_sin, positions, tokens: int, interleaved: bool, device) -> bytes:
    """The rmsnorm_rope_t."""
    import torch
    if cos_sin is None:
        return _NO_ROPE
    if positions is None:
        raise ValueError("cos_sin without positions")
    if cos_sin.dtype != torch.float32 or positions.dtype != torch.int64:
        raise TypeError("cos_sin must be float32 and positions int64")
    if cos_sin.device != device or positions.device != device:
        raise ValueError("cos_sin and positions must be on the device of q and k")
    shape = cos_sin.shape
    if len(shape) != 2 or not cos_sin.is_contiguous() or not positions.is_contiguous():
        raise ValueError("cos_sin must be [max_position, rotary_dim], cos_sin and positions "
                         "contiguous")
    if positions.numel() != tokens:
        raise ValueError("positions must hold one position for each token")
    return _ROPE.pack(cos_sin.data_ptr(), positions.data_ptr(), shape[0], shape[1],
                      1 if interleaved else 0)


def _head_weight(w, name: str, head_dim: int, dtype, device):
    if w is None:
        return None
    if w.dtype is not dtype or w.device != device:
        raise TypeError(f"{name} must have the dtype and device of its heads")
    if w.numel() != head_dim or not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous, with head_dim elements")
    return w.data_ptr()


def _same_shape(t, like, name: str) -> None:
    if t is None or t.shape != like.shape:
        raise ValueError(f"{name} must be given, with the shape of its input")


def qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps: float,
                 weight_bias: float = 0.0, interleaved: bool = False, q_out=None, k_out=None,
                 stream=None):
    """Per-head norm and position rotation of q [..., q_heads, head_dim] and k
    [..., k_heads, head_dim] in one pass (rmsnorm_qk_norm_rope): in place, or
    into q_out / k_out.  Returns (q_out, k_out).

    Every tensor's leading dimensions are the tokens and must step evenly;
    heads may be strided (views into a fused QKV tensor, head-major layouts).
    ``cos_sin``: float32 [max_position, rotary_dim], a row holding the cosines
    of a position's rotary_dim / 2 angles and then their sines; ``positions``:
    int64, one for each token; both None: no rotation.  ``k`` may be None.
    A position outside the table leaves its token out and is reported by
    rmsnorm_get_device_status (ERR_BAD_INDEX).  Runs on ``stream`` (default:
    PyTorch's current stream)."""
    if q is None:
        raise ValueError("q must be a CUDA tensor (there is no CPU path)")
    device, dtype = q.device, q.dtype
    qh, tokens = _heads(q, "q", dtype, device)
    q_heads, head_dim = q.shape[-2:]
    kh, k_heads = None, 0
    if k is not None:
        kh, k_tokens = _heads(k, "k", dtype, device)
        k_heads, k_dim = k.shape[-2:]
        if k_tokens != tokens or k_dim != head_dim:
            raise ValueError("q and k must hold the same number of tokens and one head_dim")
    if not _here(device, stream):
        with _there(device, stream, q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out):
            return qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps, weight_bias,
                                interleaved, q_out, k_out)
    qo = ko = None
    if q_out is not None:
        _same_shape(q_out, q, "q_out")
        qo = _heads(q_out, "q_out", dtype, device)[0]
    if k_out is not None:
        if k is None:
            raise ValueError("k_out without k")
        _same_shape(k_out, k, "k_out")
        ko = _heads(k_out, "k_out", dtype, device)[0]
    _check(_load().rmsnorm_qk_norm_rope(
        qh, kh, qo, ko, _head_weight(q_weight, "q_weight", head_dim, dtype, device),
        _head_weight(k_weight, "k_weight", head_dim, dtype, device),
        _rope(cos_sin, positions, tokens, interleaved, device), tokens, q_heads, k_heads,
        head_dim, weight_bias, eps, torch_dtype_code(dtype), _stream(device)),
        "rmsnorm_qk_norm_rope")
    return q if q_out is None else q_out, k if k_out is None else k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos_sin, positions,
                          eps: float, weight_bias: float = 0.0, interleaved: bool = False,
                          dq=None, dk=None, weight_grads: bool = True, stream=None):
    """Gradient of ``qk_norm_rope`` (rmsnorm_qk_norm_rope_bwd): (dq, dk,
    dq_weight, dk_weight) from the gradients of its outputs and its inputs q
    and k as they were before the call (so that call must not be in place).
    dq / dk: optional outputs, which may be dq_out / dk_out or q / k
    themselves; by default new contiguous tensors.  Expanded gradients (stride
    0) are refused: make them contiguous.  The weights' gradients are
    float32 [head_dim] (None with ``weight_grads=False``).  k and dk_out may
    be None.  Other arguments as for ``qk_norm_rope``."""
    import torch
    if q is None:
        raise ValueError("q must be a CUDA tensor (there is no CPU path)")
    device, dtype = q.device, q.dtype
    qh, tokens = _heads(q, "q", dtype, device)
    q_heads, head_dim = q.shape[-2:]
    if not _here(device, stream):
        with _there(device, stream, dq_out, dk_out, q, k, q_weight, k_weight, cos_sin, positions,
                    dq, dk):
            return qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos_sin,
                                         positions, eps, weight_bias, interleaved, dq, dk,
                                         weight_grads)
    _same_shape(dq_out, q, "dq_out")
    qy = _heads(dq_out, "dq_out", dtype, device)[0]
    kh = ky = kd = None
    k_heads = 0
    if k is not None:
        kh, k_tokens = _heads(k, "k", dtype, device)
        k_heads, k_dim = k.shape[-2:]
        if k_tokens != tokens or k_dim != head_dim:
            raise ValueError("q and k must hold the same number of tokens and one head_dim")
        _same_shape(dk_out, k, "dk_out")
        ky = _heads(dk_out, "dk_out", dtype, device)[0]
        if dk is None:
            dk = torch.empty_like(k, memory_format=torch.contiguous_format)
            kd = _HEADS.pack(dk.data_ptr(), 0, 0)
        else:
            _same_shape(dk, k, "dk")
            kd = _heads(dk, "dk", dtype, device)[0]
    if dq is None:
        dq = torch.empty_like(q, memory_format=torch.contiguous_format)
        qd = _HEADS.pack(dq.data_ptr(), 0, 0)
    else:
        _same_shape(dq, q, "dq")
        qd = _heads(dq, "dq", dtype, device)[0]
    wp = qp = kp = qg = kg = None
    need = 0
    if weight_grads:
        need = _heads_workspace(head_dim, _sm_count(device.index))
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        qg = torch.empty(head_dim, dtype=torch.float32, device=device)
        kg = torch.empty(head_dim, dtype=torch.float32, device=device)
        wp, qp, kp = ws.data_ptr(), qg.data_ptr(), kg.data_ptr()
    _check(_load().rmsnorm_qk_norm_rope_bwd(
        qy, ky, qh, kh, qd, kd, _head_weight(q_weight, "q_weight", head_dim, dtype, device),
        _head_weight(k_weight, "k_weight", head_dim, dtype, device), qp, kp,
        _rope(cos_sin, positions, tokens, interleaved, device), wp, need, tokens, q_heads,
        k_heads, head_dim, weight_bias, eps, torch_dtype_code(dtype), _stream(device)),
        "rmsnorm_qk_norm_rope_bwd")
    return dq, dk, qg, kg


def qk_norm_rope_append(q, k, v, q_weight, k_weight, cos_sin, positions, slots, k_cache, v_cache,
                        eps: float, weight_bias: float = 0.0, interleaved: bool = False,
                        k_scale: float = 1.0, v_scale: float = 1.0, q_out=None, stream=None):
    """``qk_norm_rope`` with the keys and values appended to a paged cache in
    the same launch (rmsnorm_qk_norm_rope_append): q in place or into q_out, k
    and v into k_cache and v_cache [pages, page_size, k_heads, head_dim] (any
    strides but the last; head-first caches come as transposed views) at
    slots[t] = page * page_size + slot.  Returns q_out.

    ``slots``: int64, one for each token; a negative one marks padding, of
    which nothing is written and whose values and position have no effect; the
    others must differ.  Caches hold the elements' dtype, or E4M3 codes of
    value / scale (float8_e4m3fn or uint8).  Weights None: the rotation alone.
    k and v are left as they were; ``q`` may be None."""
    import torch
    if k is None:
        raise ValueError("k must be a CUDA tensor (there is no CPU path)")
    device, k_dtype = k.device, k.dtype
    kh, tokens = _heads(k, "k", k_dtype, device)
    vh, v_tokens = _heads(v, "v", k_dtype, device)
    k_heads, head_dim = k.shape[-2:]
    qh, q_heads, q_tokens, qo = None, 0, tokens, None
    if q is not None:
        qh, q_tokens = _heads(q, "q", k_dtype, device)
        q_heads = q.shape[-2]
        if q.shape[-1] != head_dim:
            raise ValueError("q and k must hold one head_dim")
    if v.shape[-2:] != k.shape[-2:] or v_tokens != tokens or q_tokens != tokens:
        raise ValueError("q, k and v must hold the same number of tokens, k and v the same heads")
    if q_out is not None:
        if q is None:
            raise ValueError("q_out without q")
        _same_shape(q_out, q, "q_out")
        qo = _heads(q_out, "q_out", k_dtype, device)[0]
    if not _here(device, stream):
        with _there(device, stream, q, k, v, q_weight, k_weight, cos_sin, positions, slots,
                    k_cache, v_cache, q_out):
            return qk_norm_rope_append(q, k, v, q_weight, k_weight, cos_sin, positions, slots,
                                       k_cache, v_cache, eps, weight_bias, interleaved, k_scale,
                                       v_scale, q_out)
    if slots is None or slots.dtype != torch.int64:
        raise TypeError("slots must be int64")
    if slots.device != device or slots.numel() != tokens or not slots.is_contiguous():
        raise ValueError("slots must be contiguous, one for each token, on the device of k")
    shape, st = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or shape[2] != k_heads or shape[3] != head_dim or \
            v_cache.shape != shape or v_cache.stride() != st:
        raise ValueError("k_cache and v_cache must be [pages, page_size, k_heads, head_dim] with "
                         "the same strides")
    dtype = k_cache.dtype
    if v_cache.dtype != dtype or k_cache.device != device or v_cache.device != device:
        raise TypeError("k_cache and v_cache must have one dtype and the device of k")
    if head_dim > 1 and st[3] != 1:
        raise ValueError("the last dimension of the caches must be contiguous")
    e4m3 = dtype is not k_dtype
    if e4m3 and dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError("the caches must hold the dtype of k, float8_e4m3fn or uint8")
    cache = _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), shape[0], shape[1], st[0], st[1],
                        st[2], e4m3, k_scale, v_scale)
    _check(_load().rmsnorm_qk_norm_rope_append(
        qh, kh, vh, qo, _head_weight(q_weight, "q_weight", head_dim, k_dtype, device),
        _head_weight(k_weight, "k_weight", head_dim, k_dtype, device),
        _rope(cos_sin, positions, tokens, interleaved, device), cache, slots.data_ptr(), tokens,
        q_heads, k_heads, head_dim, weight_bias, eps, torch_dtype_code(k_dtype),
        _stream(device)), "rmsnorm_qk_norm_rope_append")
    return q if q_out is None else q_out


def rms_norm_backward(dy, x, weight, eps: float, weight_bias: float = -0.0, dx=None,
                      weight_grad: bool = True, stream=None):
    """Gradient of ``rms_norm`` (of ``rms_norm_bias`` with ``weight_bias``)
    through rmsnorm_bwd: (dx, dweight) from dy, the gradient of the output, and
    x, the input.  Tensors as for ``rms_norm``; ``dx``: optional output, which
    may be dy or x itself; dweight is float32 [hidden] (None with
    ``weight_grad=False``)."""
    import torch
    _check_rows(x, weight)
    device, shape, dtype = x.device, x.shape, x.dtype
    if dy is None:
        raise ValueError("dy must be given")
    for t, name in ((dy, "dy"), (dx, "dx")):
        if t is not None and (t.shape != shape or t.dtype != dtype or t.device != device or
                              not t.is_contiguous()):
            raise ValueError(f"{name} must match x (shape, dtype, device, contiguous)")
    if weight.device != device:
        raise ValueError("weight must be on the device of x")
    if not _here(device, stream):
        with _there(device, stream, dy, x, weight, dx):
            return rms_norm_backward(dy, x, weight, eps, weight_bias, dx, weight_grad)
    hidden = shape[-1]
    rows = x.numel() // hidden if hidden else 0
    code = torch_dtype_code(dtype)
    if dx is None:
        dx = torch.empty_like(x)
    need = _rows_workspace(rows, hidden, code, _sm_count(device.index))
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    w_grad = torch.empty(hidden, dtype=torch.float32, device=device) if weight_grad else None
    _check(_load().rmsnorm_bwd(dy.data_ptr(), x.data_ptr(), weight.data_ptr(), dx.data_ptr(),
                               w_grad.data_ptr() if weight_grad else None, ws.data_ptr(), need,
                               rows, hidden, weight_bias, eps, code, _stream(device)),
           "rmsnorm_bwd")
    return dx, w_grad
