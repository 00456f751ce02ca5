"""ctypes binding of libpaged_decode.so (argument marshalling only).

The functions carry the names of the C entry points declared in
include/paged_decode.h and take torch tensors (device memory) or plain
integers; every step of the computation runs in the library's CUDA kernels.
There is no fallback: if the library is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading
from typing import Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libpaged_decode.so")

PD_OK = 0
PD_ERR_INVALID_ARG = 1
PD_ERR_UNSUPPORTED = 2
PD_ERR_WORKSPACE_TOO_SMALL = 3
PD_ERR_CUDA = 4
PD_ERR_DEVICE_FAULT = 5

# layout of pd_plan / pd_layer_desc this binding marshals (paged_decode_abi_version)
ABI_VERSION = 5

PD_KV_BF16 = 0
PD_KV_FP8_E4M3 = 1
PD_KV_FP4_E2M1 = 2

PD_DEVFLAG_BAD_PAGE = 0x1
PD_DEVFLAG_BAD_SEQLEN = 0x2
PD_DEVFLAG_WAIT_TIMEOUT = 0x4
PD_DEVFLAG_NO_PAGES = 0x8
PD_DEVFLAG_BAD_GROUP = 0x10

EXPORTED = (
    "paged_decode_plan",
    "paged_decode_global",
    "paged_decode_window",
    "paged_decode_merge",
    "paged_decode_check_device_error",
    "paged_decode_status_string",
    "paged_decode_abi_version",
    "paged_decode_noalloc",
    "paged_decode_global_fp8",
    "paged_decode_window_fp8",
    "paged_decode_plan_multi",
    "paged_decode_plan_partial",
    "paged_decode_global_partial",
    "paged_decode_combine",
    "paged_decode_rope_table",
    "paged_decode_qkv_norm_rope_write",
    "paged_decode_stage_copy",
    "paged_decode_append_slots_workspace",
    "paged_decode_append_slots",
    "paged_decode_write_slots",
    "paged_decode_write_slots_fp8",
    "paged_decode_plan_shared",
    "paged_decode_global_shared",
    "paged_decode_global_shared_fp8",
    "paged_decode_append_slots_args",
    "paged_decode_write_slots_args",
    "paged_decode_global_shared_args",
    "paged_decode_global_fp4",
    "paged_decode_window_fp4",
    "paged_decode_write_slots_fp4",
    "paged_decode_read_slots",
    "paged_decode_read_slots_fp8",
    "paged_decode_read_slots_fp4",
    "paged_decode_write_slots_fp4_args",
    "paged_decode_read_slots_args",
)


class LayerDesc(ctypes.Structure):
    _fields_ = [
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("kv_shared", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
    ]


class Plan(ctypes.Structure):
    _fields_ = [
        ("layer", LayerDesc),
        ("batch", ctypes.c_int32),
        ("num_splits", ctypes.c_int32),
        ("chunk_tokens", ctypes.c_int32),
        ("block_tokens", ctypes.c_int32),
        ("variant", ctypes.c_int32),
        ("grid_x", ctypes.c_int32),
        ("grid_y", ctypes.c_int32),
        ("grid_z", ctypes.c_int32),
        ("threads_per_cta", ctypes.c_int32),
        ("smem_bytes", ctypes.c_int32),
        ("sm_count", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
        ("merge_mode", ctypes.c_int32),
        ("test_stall_bytes", ctypes.c_int32),
        ("query_tokens", ctypes.c_int32),
        ("partial", ctypes.c_int32),
        ("early_kv", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_uint64),
        ("lse_offset", ctypes.c_uint64),
        ("opart_offset", ctypes.c_uint64),
        ("magic", ctypes.c_uint32),
        ("version", ctypes.c_uint32),
    ]


class SharedPlan(ctypes.Structure):
    _fields_ = [
        ("own", Plan),
        ("num_groups", ctypes.c_int32),
        ("max_prefix_pages", ctypes.c_int32),
        ("row_tile", ctypes.c_int32),
        ("tiles", ctypes.c_int32),
        ("num_pieces", ctypes.c_int32),
        ("chunk_tokens", ctypes.c_int32),
        ("max_prefix_len", ctypes.c_int32),
        ("variant", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_uint64),
        ("lse_offset", ctypes.c_uint64),
        ("o_offset", ctypes.c_uint64),
        ("magic", ctypes.c_uint32),
        ("version", ctypes.c_uint32),
    ]


class PagedDecodeError(RuntimeError):
    def __init__(self, status: int, where: str, flags: int = 0):
        self.status = status
        self.flags = flags
        msg = f"{where}: {status_string(status)} (status {status})"
        if flags:
            msg += f", device flags 0x{flags:x}"
        super().__init__(msg)


_lock = threading.Lock()
_lib = None


def load_library(path: Optional[str] = None):
    """Load the CUDA library; raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"CUDA library not found at {p}; build it with "
                "`python -m paged_gqa_decode_global_gb300.build` (no CPU fallback exists)")
        lib = ctypes.CDLL(p)
        vp, i32, u64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
        lib.paged_decode_plan.argtypes = [ctypes.POINTER(LayerDesc), i32, vp, i32, ctypes.POINTER(Plan)]
        lib.paged_decode_plan.restype = ctypes.c_int
        lib.paged_decode_global.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, vp, vp, f32, vp, u64, vp, vp]
        lib.paged_decode_global.restype = ctypes.c_int
        lib.paged_decode_window.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, vp, vp, i32, f32, vp, u64, vp, vp]
        lib.paged_decode_window.restype = ctypes.c_int
        lib.paged_decode_merge.argtypes = [ctypes.POINTER(Plan), vp, u64, vp, vp]
        lib.paged_decode_merge.restype = ctypes.c_int
        lib.paged_decode_check_device_error.argtypes = [ctypes.POINTER(Plan), vp, u64, vp,
                                                        ctypes.POINTER(ctypes.c_uint32)]
        lib.paged_decode_check_device_error.restype = ctypes.c_int
        lib.paged_decode_status_string.argtypes = [ctypes.c_int]
        lib.paged_decode_status_string.restype = ctypes.c_char_p
        lib.paged_decode_abi_version.argtypes = []
        lib.paged_decode_abi_version.restype = i32
        lib.paged_decode_noalloc.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, vp, vp, i32, f32, vp, vp, vp]
        lib.paged_decode_noalloc.restype = ctypes.c_int
        lib.paged_decode_global_fp8.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, vp, vp, vp, vp, f32, vp, u64, vp,
                                                vp]
        lib.paged_decode_global_fp8.restype = ctypes.c_int
        lib.paged_decode_window_fp8.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, vp, vp, vp, vp, i32, f32, vp, u64,
                                                vp, vp]
        lib.paged_decode_window_fp8.restype = ctypes.c_int
        lib.paged_decode_plan_multi.argtypes = [ctypes.POINTER(LayerDesc), i32, i32, vp, i32, ctypes.POINTER(Plan)]
        lib.paged_decode_plan_multi.restype = ctypes.c_int
        lib.paged_decode_plan_partial.argtypes = [ctypes.POINTER(LayerDesc), i32, vp, i32, ctypes.POINTER(Plan)]
        lib.paged_decode_plan_partial.restype = ctypes.c_int
        lib.paged_decode_global_partial.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, vp, vp, f32, vp, u64, vp, vp, vp]
        lib.paged_decode_global_partial.restype = ctypes.c_int
        lib.paged_decode_combine.argtypes = [i32, i32, i32, vp, vp, vp, vp]
        lib.paged_decode_combine.restype = ctypes.c_int
        lib.paged_decode_stage_copy.argtypes = [ctypes.c_void_p, i32, i32, vp]
        lib.paged_decode_stage_copy.restype = ctypes.c_int
        lib.paged_decode_rope_table.argtypes = [ctypes.c_double, i32, i32, vp, vp]
        lib.paged_decode_rope_table.restype = ctypes.c_int
        lib.paged_decode_qkv_norm_rope_write.argtypes = [ctypes.POINTER(LayerDesc), i32, i32, i32, f32] + [vp] * 14
        lib.paged_decode_qkv_norm_rope_write.restype = ctypes.c_int
        i64 = ctypes.c_int64
        lib.paged_decode_append_slots_workspace.argtypes = [i32]
        lib.paged_decode_append_slots_workspace.restype = u64
        lib.paged_decode_append_slots.argtypes = [i32] * 5 + [vp] * 3 + [i32] + [vp] * 9 + [u64, vp]
        lib.paged_decode_append_slots.restype = ctypes.c_int
        lib.paged_decode_write_slots.argtypes = [ctypes.POINTER(LayerDesc), i32, vp, vp, i64, i64] + [vp] * 5
        lib.paged_decode_write_slots.restype = ctypes.c_int
        lib.paged_decode_write_slots_fp8.argtypes = [ctypes.POINTER(LayerDesc), i32, vp, vp, i64, i64] + [vp] * 7
        lib.paged_decode_write_slots_fp8.restype = ctypes.c_int
        lib.paged_decode_plan_shared.argtypes = [ctypes.POINTER(LayerDesc), i32, i32, vp, i32, vp, vp, i32, i32,
                                                 ctypes.POINTER(SharedPlan)]
        lib.paged_decode_plan_shared.restype = ctypes.c_int
        lib.paged_decode_global_shared.argtypes = [ctypes.POINTER(SharedPlan)] + [vp] * 8 + [f32, vp, u64, vp, vp]
        lib.paged_decode_global_shared.restype = ctypes.c_int
        lib.paged_decode_global_shared_fp8.argtypes = [ctypes.POINTER(SharedPlan)] + [vp] * 10 + [f32, vp, u64, vp, vp]
        lib.paged_decode_global_shared_fp8.restype = ctypes.c_int
        lib.paged_decode_global_fp4.argtypes = [ctypes.POINTER(Plan)] + [vp] * 5 + [i32] * 2 + [vp] * 2 + [
            f32, vp, u64, vp, vp]
        lib.paged_decode_global_fp4.restype = ctypes.c_int
        lib.paged_decode_window_fp4.argtypes = [ctypes.POINTER(Plan)] + [vp] * 5 + [i32] * 2 + [vp] * 2 + [
            i32, f32, vp, u64, vp, vp]
        lib.paged_decode_window_fp4.restype = ctypes.c_int
        rows = [ctypes.POINTER(LayerDesc), i32]
        lib.paged_decode_write_slots_fp4.argtypes = rows + [vp] * 2 + [i64] * 2 + [vp] * 5 + [i32] * 2 + [vp] * 2
        lib.paged_decode_write_slots_fp4.restype = ctypes.c_int
        lib.paged_decode_read_slots.argtypes = rows + [vp] * 5 + [i64] * 2 + [vp] * 2
        lib.paged_decode_read_slots.restype = ctypes.c_int
        lib.paged_decode_read_slots_fp8.argtypes = rows + [vp] * 7 + [i64] * 2 + [vp] * 2
        lib.paged_decode_read_slots_fp8.restype = ctypes.c_int
        lib.paged_decode_read_slots_fp4.argtypes = rows + [vp] * 5 + [i32] * 2 + [vp] * 2 + [i64] * 2 + [vp] * 2
        lib.paged_decode_read_slots_fp4.restype = ctypes.c_int
        for fn in (lib.paged_decode_append_slots_args, lib.paged_decode_write_slots_args,
                   lib.paged_decode_global_shared_args, lib.paged_decode_write_slots_fp4_args,
                   lib.paged_decode_read_slots_args):
            fn.argtypes, fn.restype = [ctypes.c_char_p], ctypes.c_int
        found = int(lib.paged_decode_abi_version())
        if found != ABI_VERSION:
            raise RuntimeError(f"{p} has ABI version {found}, this binding marshals version {ABI_VERSION}: rebuild it "
                               "with `python -m paged_gqa_decode_global_gb300.build`")
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    try:
        return load_library().paged_decode_status_string(status).decode()
    except Exception:  # noqa: BLE001 - message formatting must not fail
        return f"status {status}"


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        torch = _torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the same without a Stream object
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != PD_OK:
        raise PagedDecodeError(status, where)


def layer_desc(num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int, num_pages: int,
               max_pages_per_seq: int, window: int = 0, kv_shared: bool = False,
               kv_dtype: int = PD_KV_BF16) -> LayerDesc:
    return LayerDesc(num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
                     window, 1 if kv_shared else 0, int(kv_dtype))


def paged_decode_plan(desc: LayerDesc, seq_lens_host: Sequence[int], sm_count: int) -> Plan:
    lib = load_library()
    n = len(seq_lens_host)
    arr = (ctypes.c_int32 * max(1, n))(*[int(x) for x in seq_lens_host])
    plan = Plan()
    st = lib.paged_decode_plan(ctypes.byref(desc), n, ctypes.cast(arr, ctypes.c_void_p) if n else None,
                               int(sm_count), ctypes.byref(plan))
    _check(st, "paged_decode_plan")
    return plan


def paged_decode_plan_multi(desc: LayerDesc, query_tokens: int, seq_lens_host: Sequence[int],
                            sm_count: int) -> Plan:
    """Plan for `query_tokens` new tokens per request (q / out [B, T, Hq, d])."""
    lib = load_library()
    n = len(seq_lens_host)
    arr = (ctypes.c_int32 * max(1, n))(*[int(x) for x in seq_lens_host])
    plan = Plan()
    st = lib.paged_decode_plan_multi(ctypes.byref(desc), n, int(query_tokens),
                                     ctypes.cast(arr, ctypes.c_void_p) if n else None, int(sm_count),
                                     ctypes.byref(plan))
    _check(st, "paged_decode_plan_multi")
    return plan


def paged_decode_global(plan: Plan, q, k_pool, v_pool, block_tables, seq_lens, scale: float, workspace,
                        out, stream=None, workspace_bytes: Optional[int] = None) -> None:
    lib = load_library()
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = lib.paged_decode_global(ctypes.byref(plan), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_tables),
                                 _ptr(seq_lens), float(scale), _ptr(workspace), int(wb), _ptr(out),
                                 _stream_ptr(stream))
    _check(st, "paged_decode_global")


def paged_decode_window(plan: Plan, q, k_pool, v_pool, block_tables, seq_lens, window: int, scale: float,
                        workspace, out, stream=None, workspace_bytes: Optional[int] = None) -> None:
    lib = load_library()
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = lib.paged_decode_window(ctypes.byref(plan), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_tables),
                                 _ptr(seq_lens), int(window), float(scale), _ptr(workspace), int(wb), _ptr(out),
                                 _stream_ptr(stream))
    _check(st, "paged_decode_window")


def paged_decode_global_fp8(plan: Plan, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens,
                            scale: float, workspace, out, stream=None, workspace_bytes: Optional[int] = None) -> None:
    lib = load_library()
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = lib.paged_decode_global_fp8(ctypes.byref(plan), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale),
                                     _ptr(v_scale), _ptr(block_tables), _ptr(seq_lens), float(scale),
                                     _ptr(workspace), int(wb), _ptr(out), _stream_ptr(stream))
    _check(st, "paged_decode_global_fp8")


def paged_decode_window_fp8(plan: Plan, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens, window: int,
                            scale: float, workspace, out, stream=None, workspace_bytes: Optional[int] = None) -> None:
    lib = load_library()
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = lib.paged_decode_window_fp8(ctypes.byref(plan), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale),
                                     _ptr(v_scale), _ptr(block_tables), _ptr(seq_lens), int(window), float(scale),
                                     _ptr(workspace), int(wb), _ptr(out), _stream_ptr(stream))
    _check(st, "paged_decode_window_fp8")


def paged_decode_global_fp4(plan: Plan, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens, scale: float,
                            workspace, out, stream=None, workspace_bytes: Optional[int] = None, *, k_exp: int = 0,
                            v_exp: int = 0) -> None:
    """Stage 1 over a 4-bit cache: k_pool / v_pool uint8 codes [pages, Hkv, P, d / 2], k_scale / v_scale uint8 (e4m3)
    [pages, Hkv, P, d / 16], values times 2^k_exp and 2^v_exp (fp4_exponent). On a K=V layer v_exp is k_exp."""
    _decode_fp4(plan, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens, None, scale, workspace, out, stream,
                workspace_bytes, k_exp, v_exp)


def paged_decode_window_fp4(plan: Plan, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens, window: int,
                            scale: float, workspace, out, stream=None, workspace_bytes: Optional[int] = None, *,
                            k_exp: int = 0, v_exp: int = 0) -> None:
    """The same on a sliding-window layer."""
    _decode_fp4(plan, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens, int(window), scale, workspace, out,
                stream, workspace_bytes, k_exp, v_exp)


def _decode_fp4(plan, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens, window, scale, workspace, out,
                stream, workspace_bytes, k_exp, v_exp) -> None:
    lib, ly = load_library(), plan.layer
    dev, nbytes = workspace.get_device(), workspace.nbytes if workspace_bytes is None else int(workspace_bytes)
    if workspace.nbytes < nbytes or not workspace.is_contiguous():
        _refuse_bytes("workspace", workspace, nbytes)
    torch = _torch()
    B, T, Hq, d = plan.batch, plan.query_tokens, ly.num_q_heads, ly.head_dim
    shape = (B, T, Hq, d) if T > 1 or (hasattr(q, "dim") and q.dim() == 4) else (B, Hq, d)
    pool, scales = _fp4_shapes(ly)
    _want_or_address(q, "q", torch.bfloat16, shape, dev)
    _want_or_address(out, "out", torch.bfloat16, shape, dev)
    _want_or_address(k_pool, "k_pool", torch.uint8, pool, dev)
    _want_or_address(v_pool, "v_pool", torch.uint8, pool, dev)
    _want_or_address(k_scale, "k_scale", torch.uint8, scales, dev)
    _want_or_address(v_scale, "v_scale", torch.uint8, scales, dev)
    _want_or_address(block_tables, "block_tables", torch.int32, (B, ly.max_pages_per_seq), dev)
    _want_or_address(seq_lens, "seq_lens", torch.int32, (B,), dev)
    raw = _launch_stream(stream, dev)
    head = (ctypes.byref(plan), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), k_exp, v_exp,
            _ptr(block_tables), _ptr(seq_lens))
    tail = (scale, workspace.data_ptr(), nbytes, _ptr(out), raw)
    if window is None:
        st = lib.paged_decode_global_fp4(*head, *tail)
    else:
        st = lib.paged_decode_window_fp4(*head, window, *tail)
    if st != PD_OK:
        raise PagedDecodeError(st, "paged_decode_global_fp4" if window is None else "paged_decode_window_fp4")


def _fp4_shapes(ly) -> tuple:
    """A layer's 4-bit pool and its block scales."""
    rows = (ly.num_pages, ly.num_kv_heads, ly.page_size)
    return rows + (ly.head_dim // 2,), rows + (ly.head_dim // 16,)


def fp4_exponent(largest: float) -> int:
    """The layer exponent for values of magnitudes up to `largest`: the smallest e in [-64, 64] with
    largest <= 6 * 448 * 2^e; 64 past them all (infinity too), 0 without a positive magnitude (NaN too)."""
    if not largest > 0.0:
        return 0
    if math.isinf(largest):
        return 64
    m, e = math.frexp(largest)  # (a quotient by 6 * 448 = 0.65625 * 2^12 would be 0 for the smallest numbers)
    return max(-64, min(64, e - 12 if m <= 0.65625 else e - 11))


def paged_decode_merge(plan: Plan, workspace, out, stream=None, workspace_bytes: Optional[int] = None) -> None:
    lib = load_library()
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = lib.paged_decode_merge(ctypes.byref(plan), _ptr(workspace), int(wb), _ptr(out), _stream_ptr(stream))
    _check(st, "paged_decode_merge")


def paged_decode_check_device_error(plan: Plan, workspace, stream=None) -> int:
    """Synchronise, read and clear the device error word; raises on a non-zero word."""
    lib = load_library()
    flags = ctypes.c_uint32(0)
    wb = workspace.numel() * workspace.element_size()
    st = lib.paged_decode_check_device_error(ctypes.byref(plan), _ptr(workspace), int(wb), _stream_ptr(stream),
                                             ctypes.byref(flags))
    if st != PD_OK:
        raise PagedDecodeError(st, "paged_decode_check_device_error", flags.value)
    return flags.value


def paged_decode_noalloc(plan: Plan, q, k_pool, v_pool, block_tables, seq_lens, window: int, scale: float, out,
                         device_flags=None, stream=None) -> None:
    """Stage 1 + merge using the library's own scratch array instead of a
    workspace, for callers that cannot allocate device memory (see the C
    header). `device_flags`: optional int32/uint32 device tensor receiving the
    call's device error word."""
    lib = load_library()
    st = lib.paged_decode_noalloc(ctypes.byref(plan), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_tables),
                                  _ptr(seq_lens), int(window), float(scale), _ptr(out), _ptr(device_flags),
                                  _stream_ptr(stream))
    _check(st, "paged_decode_noalloc")


def abi_version() -> int:
    return int(load_library().paged_decode_abi_version())


# ----------------------------------------------------------------------------
# Convenience: one layer-step (stage 1 + stage 2) on torch tensors
# ----------------------------------------------------------------------------

class LayerStep:
    """Plan + workspace for one layer, reusable across steps whose sequences
    are no longer than the planned ones."""

    def __init__(self, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
                 seq_lens_host, *, window=0, kv_shared=False, kv_dtype=PD_KV_BF16, sm_count=None, device=None,
                 query_tokens=1, early_kv=False):
        import torch
        device = torch.device("cuda") if device is None else torch.device(device)
        if sm_count is None:
            sm_count = torch.cuda.get_device_properties(device).multi_processor_count
        self.desc = layer_desc(num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
                               window, kv_shared, kv_dtype)
        self.fp8 = kv_dtype == PD_KV_FP8_E4M3
        self.fp4 = kv_dtype == PD_KV_FP4_E2M1
        self.query_tokens = int(query_tokens)
        if self.query_tokens > 1:
            self.plan = paged_decode_plan_multi(self.desc, self.query_tokens, list(seq_lens_host), sm_count)
        else:
            self.plan = paged_decode_plan(self.desc, list(seq_lens_host), sm_count)
        # the caller's promise about the kernel launched just before stage 1 (pd_plan.early_kv)
        self.plan.early_kv = 1 if early_kv else 0
        nbytes = int(self.plan.workspace_bytes)
        # zeroed once: the first word is the device error flag
        self.workspace = torch.zeros((nbytes + 255) // 256 * 256, dtype=torch.uint8, device=device)
        self.window = window

    @classmethod
    def for_inputs(cls, li, sm_count=None, query_tokens=1, early_kv=False):
        """A step for a LayerInputs (bf16 cache) or Fp8LayerInputs (e4m3 cache), which run() takes (a step over a 4-bit
        cache is called with its tensors); query_tokens > 1: q and out are [B, T, Hq, d]."""
        fp8 = hasattr(li, "k8")
        return cls(li.num_q_heads, li.num_kv_heads, li.head_dim, li.page_size, li.num_pages, li.max_pages,
                   li.seq_lens_list(), window=li.window, kv_shared=li.kv_shared,
                   kv_dtype=PD_KV_FP8_E4M3 if fp8 else PD_KV_BF16, sm_count=sm_count, device=li.q.device,
                   query_tokens=query_tokens, early_kv=early_kv)

    def __call__(self, q, k_pool, v_pool, block_tables, seq_lens, scale, out, stream=None, k_scale=None,
                 v_scale=None, k_exp=0, v_exp=0):
        if self.fp4:
            _decode_fp4(self.plan, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens, self.window or None,
                        scale, self.workspace, out, stream, None, k_exp, v_exp)
            return out  # joined in the launch
        if self.fp8:
            if self.window > 0:
                paged_decode_window_fp8(self.plan, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens,
                                        self.window, scale, self.workspace, out, stream)
            else:
                paged_decode_global_fp8(self.plan, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens,
                                        scale, self.workspace, out, stream)
        elif self.window > 0:
            paged_decode_window(self.plan, q, k_pool, v_pool, block_tables, seq_lens, self.window, scale,
                                self.workspace, out, stream)
        else:
            paged_decode_global(self.plan, q, k_pool, v_pool, block_tables, seq_lens, scale, self.workspace,
                                out, stream)
        paged_decode_merge(self.plan, self.workspace, out, stream)
        return out

    def run(self, li, out=None, stream=None):
        import torch
        if out is None:
            out = torch.empty_like(li.q)
        if self.fp8:
            return self(li.q, li.k8, li.v8, li.block_tables, li.seq_lens, li.scale, out, stream,
                        k_scale=li.k_scale, v_scale=li.v_scale)
        return self(li.q, li.k_pool, li.v_pool, li.block_tables, li.seq_lens, li.scale, out, stream)

    def check(self, stream=None) -> int:
        return paged_decode_check_device_error(self.plan, self.workspace, stream)


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)


def paged_decode_rope_table(theta: float, rotary_dim: int, num_positions: int, cos_sin, stream=None) -> None:
    """Fill cos_sin (fp32 [num_positions, rotary_dim], device) with the layer's RoPE table."""
    st = load_library().paged_decode_rope_table(float(theta), int(rotary_dim), int(num_positions), _ptr(cos_sin),
                                                _stream_ptr(stream))
    _check(st, "paged_decode_rope_table")


def paged_decode_qkv_norm_rope_write(desc: LayerDesc, rotary_dim: int, num_positions: int, eps: float, q_in, k_in,
                                     v_in, q_norm_weight, k_norm_weight, v_norm_weight, cos_sin, block_tables,
                                     seq_lens, q_out, k_pool, v_pool, device_flags, stream=None) -> None:
    """QKV norm + RoPE of the new tokens, k / v rows written into the pools, q into q_out."""
    batch = q_in.shape[0]
    st = load_library().paged_decode_qkv_norm_rope_write(
        ctypes.byref(desc), int(batch), int(rotary_dim), int(num_positions), float(eps), _ptr(q_in), _ptr(k_in),
        _ptr(v_in), _ptr(q_norm_weight), _ptr(k_norm_weight), _ptr(v_norm_weight), _ptr(cos_sin),
        _ptr(block_tables), _ptr(seq_lens), _ptr(q_out), _ptr(k_pool), _ptr(v_pool), _ptr(device_flags),
        _stream_ptr(stream))
    _check(st, "paged_decode_qkv_norm_rope_write")


def paged_decode_plan_partial(desc: LayerDesc, seq_lens_host: Sequence[int], sm_count: int) -> Plan:
    """Plan for paged_decode_global_partial (a global bf16 layer's local tokens)."""
    lib = load_library()
    n = len(seq_lens_host)
    arr = (ctypes.c_int32 * max(1, n))(*[int(x) for x in seq_lens_host])
    plan = Plan()
    st = lib.paged_decode_plan_partial(ctypes.byref(desc), n, ctypes.cast(arr, ctypes.c_void_p) if n else None,
                                       int(sm_count), ctypes.byref(plan))
    _check(st, "paged_decode_plan_partial")
    return plan


def paged_decode_global_partial(plan: Plan, q, k_pool, v_pool, block_tables, seq_lens, scale: float, workspace,
                                o_out, lse_out, stream=None, workspace_bytes: Optional[int] = None) -> None:
    """This rank's normalised fp32 partial output o_out [B, Hq, d] and its log-sum-exp lse_out [B, Hq]."""
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    st = load_library().paged_decode_global_partial(
        ctypes.byref(plan), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_tables), _ptr(seq_lens), float(scale),
        _ptr(workspace), int(wb), _ptr(o_out), _ptr(lse_out), _stream_ptr(stream))
    _check(st, "paged_decode_global_partial")


MAX_STAGE_COPIES = 4  # PD_MAX_STAGE_COPIES


class Copy(ctypes.Structure):
    _fields_ = [("dst", ctypes.c_void_p), ("src", ctypes.c_void_p), ("bytes", ctypes.c_size_t)]


def paged_decode_stage_copy(pairs, after_wait: int = 0, stream=None) -> None:
    """Copy each (dst, src) pair of tensors (equal byte sizes; device or
    page-locked host memory; a pair of Nones is skipped) as one kernel in the
    stream's chain of programmatic dependent launches; after_wait 1 waits for
    the launch in front first."""
    entries = []
    for dst, src in pairs:
        if dst is None and src is None:
            continue
        if dst is None or src is None:
            raise ValueError("a copy needs both its source and its destination")
        n = dst.numel() * dst.element_size()
        if src.numel() * src.element_size() != n:
            raise ValueError(f"copy of {src.numel() * src.element_size()} bytes into {n} bytes")
        entries.append(Copy(_ptr(dst), _ptr(src), n))
    arr = (Copy * max(1, len(entries)))(*entries)
    st = load_library().paged_decode_stage_copy(ctypes.cast(arr, ctypes.c_void_p), len(entries), int(after_wait),
                                                _stream_ptr(stream))
    _check(st, "paged_decode_stage_copy")


def paged_decode_combine(o_parts, lse_parts, out, stream=None) -> None:
    """Merge gathered partials o_parts [R, rows..., d] fp32, lse_parts [R, rows...] into bf16 out [rows..., d]."""
    R = o_parts.shape[0]
    d = o_parts.shape[-1]
    rows = o_parts[0].numel() // d
    st = load_library().paged_decode_combine(int(R), int(rows), int(d), _ptr(o_parts), _ptr(lse_parts), _ptr(out),
                                             _stream_ptr(stream))
    _check(st, "paged_decode_combine")


# ----------------------------------------------------------------------------
# Block tables and slot maps, the cache write by slot, shared-prefix decode
# ----------------------------------------------------------------------------

# pd_append_slots_args, pd_write_slots_args and pd_global_shared_args: one
# argument for ctypes to convert instead of up to twenty (~2 us)
_SLOTS_ARGS = struct.Struct("6i12PQP").pack
_WRITE_ARGS = struct.Struct("P2i2P2q7P").pack
_SHARED_ARGS = struct.Struct("P10PfiPQ2P").pack


def _refuse(name: str, t, dtype, shape) -> None:
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {shape}, got {t.dtype} "
                     f"{tuple(t.shape)}{'' if t.is_contiguous() else ' (not contiguous)'} on {t.device}")


def _want(t, name: str, dtype, shape, device: int) -> None:
    """A tensor handed to the library is contiguous, of the type and shape its C argument has, on the call's device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        _refuse(name, t, dtype, shape)


def _refuse_bytes(name: str, t, nbytes: int) -> None:
    raise ValueError(f"{name}: expected a contiguous tensor of at least {nbytes} bytes on the GPU of the call's other "
                     f"tensors, got {t.dtype} {tuple(t.shape)}{'' if t.is_contiguous() else ' (not contiguous)'} on "
                     f"{t.device}")


def _is_word(t, device: int) -> bool:
    """Whether a flag word fits a tensor, of any type, on the call's device."""
    return t.nbytes >= 4 and t.is_contiguous() and t.get_device() == device


def _launch_stream(stream, device: int) -> int:
    """The raw stream of a call whose tensors are all on GPU `device`: it launches on the current device, which has to
    be that one."""
    torch = _torch()
    if device < 0:
        raise ValueError("every tensor, device_flags and workspace among them, has to be on the call's GPU")
    current = torch.cuda.current_device()
    if device != current:
        raise ValueError(f"the call's tensors are on cuda:{device}, but it would launch on the current device, "
                         f"cuda:{current}: call it under torch.cuda.device({device})")
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the same without a Stream object
        if raw is not None:
            return raw(device)
    elif getattr(stream, "device_index", device) != device:
        raise ValueError(f"the call's tensors are on cuda:{device}, its stream is cuda:{stream.device_index}'s")
    return _stream_ptr(stream) or 0


def paged_decode_append_slots_workspace(batch: int) -> int:
    """Bytes of the (zeroed) workspace paged_decode_append_slots takes."""
    return int(load_library().paged_decode_append_slots_workspace(int(batch)))


def paged_decode_append_slots(page_size: int, num_pages: int, cached_lens, new_tokens, free_pages, free_range,
                              block_tables, seq_lens, token_starts, slot_map, positions, free_range_out, device_flags,
                              workspace, stream=None) -> None:
    """Hand out the pages the requests' new tokens need and write their slots:
    block_tables [B, max_pages] is extended in place; seq_lens [B],
    token_starts [B + 1], slot_map and positions (None: not wanted) [max_tokens]
    and free_range_out [2] are written. All int32; seq_lens may be cached_lens
    and free_range_out may be free_range."""
    i32 = _torch().int32
    dev, (B,), (n,), (free,) = cached_lens.get_device(), cached_lens.shape, slot_map.shape, free_pages.shape
    width = block_tables.shape[-1]
    _want(cached_lens, "cached_lens", i32, (B,), dev)
    _want(new_tokens, "new_tokens", i32, (B,), dev)
    _want(free_pages, "free_pages", i32, (free,), dev)
    _want(free_range, "free_range", i32, (2,), dev)
    _want(block_tables, "block_tables", i32, (B, width), dev)
    _want(seq_lens, "seq_lens", i32, (B,), dev)
    _want(token_starts, "token_starts", i32, (B + 1,), dev)
    _want(slot_map, "slot_map", i32, (n,), dev)
    if positions is not None:
        _want(positions, "positions", i32, (n,), dev)
    _want(free_range_out, "free_range_out", i32, (2,), dev)
    if not _is_word(device_flags, dev):
        _refuse_bytes("device_flags", device_flags, 4)
    if not workspace.is_contiguous() or workspace.get_device() != dev:
        _refuse_bytes("workspace", workspace, 4)
    raw = _launch_stream(stream, dev)
    st = load_library().paged_decode_append_slots_args(_SLOTS_ARGS(
        B, page_size, num_pages, width, n, free, cached_lens.data_ptr(), new_tokens.data_ptr(), free_pages.data_ptr(),
        free_range.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(), token_starts.data_ptr(),
        slot_map.data_ptr(), _ptr(positions) or 0, free_range_out.data_ptr(), device_flags.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, raw))
    if st != PD_OK:
        raise PagedDecodeError(st, "paged_decode_append_slots")


def _token_rows(t, name: str, dtype, shape, device: int) -> int:
    """The token stride (elements) of k / v rows [tokens, Hkv, d] whose heads are contiguous."""
    n, heads, d = shape
    token, head, one = t.stride() if t.dim() == 3 else (0, 0, 0)
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or one != 1 or (heads > 1 and head != d):
        raise ValueError(f"{name}: expected {dtype} {shape} with each token's heads contiguous, got {t.dtype} "
                         f"{tuple(t.shape)}, strides {t.stride()} on {t.device}")
    return token if n > 1 else heads * d  # (one token's stride may be anything)


def _write_slots(fp8: bool, desc, k_in, v_in, slot_map, k_pool, v_pool, k_scale, v_scale, device_flags, stream):
    torch = _torch()
    (n,), dev, heads, d = slot_map.shape, slot_map.get_device(), desc.num_kv_heads, desc.head_dim
    _want(slot_map, "slot_map", torch.int32, (n,), dev)
    pool_type = torch.uint8 if fp8 else torch.bfloat16
    pool, rows = (desc.num_pages, heads, desc.page_size, d), (n, heads, d)
    _want(k_pool, "k_pool", pool_type, pool, dev)
    ks, vs = _token_rows(k_in, "k_in", torch.bfloat16, rows, dev), 0
    if desc.kv_shared:
        v_in = None
    else:
        if v_in is None or v_pool is None:
            raise ValueError("a K != V layer needs v_in and v_pool")
        _want(v_pool, "v_pool", pool_type, pool, dev)
        vs = _token_rows(v_in, "v_in", torch.bfloat16, rows, dev)
    if fp8:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None:
                _want(t, name, torch.float32, pool[:2], dev)
    if not _is_word(device_flags, dev):
        _refuse_bytes("device_flags", device_flags, 4)
    raw = _launch_stream(stream, dev)
    st = load_library().paged_decode_write_slots_args(_WRITE_ARGS(
        ctypes.addressof(desc), n, fp8, k_in.data_ptr(), _ptr(v_in) or 0, ks, vs, slot_map.data_ptr(),
        k_pool.data_ptr(), _ptr(v_pool) or 0, _ptr(k_scale) or 0, _ptr(v_scale) or 0, device_flags.data_ptr(),
        raw))
    if st != PD_OK:
        raise PagedDecodeError(st, "paged_decode_write_slots_fp8" if fp8 else "paged_decode_write_slots")


def paged_decode_write_slots(desc: LayerDesc, k_in, v_in, slot_map, k_pool, v_pool, device_flags, stream=None) -> None:
    """Write k_in / v_in [tokens, Hkv, d] (any token stride) into the pools' rows
    slot_map names; -1 skips a token."""
    _write_slots(False, desc, k_in, v_in, slot_map, k_pool, v_pool, None, None, device_flags, stream)


def paged_decode_write_slots_fp8(desc: LayerDesc, k_in, v_in, slot_map, k_pool, v_pool, k_scale, v_scale,
                                 device_flags, stream=None) -> None:
    """The same into e4m3 pools (uint8), each row divided by its (page, head)'s scale."""
    _write_slots(True, desc, k_in, v_in, slot_map, k_pool, v_pool, k_scale, v_scale, device_flags, stream)


# pd_slot_rows_args
_ROWS_ARGS = struct.Struct("P4i2P2q7P").pack


def _slot_rows(what: str, kv: int, desc, k_rows, v_rows, slot_map, k_pool, v_pool, k_scale, v_scale, k_exp, v_exp,
               device_flags, stream) -> None:
    """paged_decode_write_slots_fp4 (rows in) and the reads (rows out)."""
    torch = _torch()
    (n,), dev, heads, d = slot_map.shape, slot_map.get_device(), desc.num_kv_heads, desc.head_dim
    if desc.kv_dtype != kv:
        raise ValueError(f"{what}: the layer's kv_dtype is {desc.kv_dtype}, not {kv}")
    _want(slot_map, "slot_map", torch.int32, (n,), dev)
    pages, rows, scale_type = (desc.num_pages, heads, desc.page_size), (n, heads, d), None
    if kv == PD_KV_FP4_E2M1:
        pool_type = scale_type = torch.uint8
        pool, scales = pages + (d // 2,), pages + (d // 16,)
    elif kv == PD_KV_FP8_E4M3:
        pool_type, scale_type = torch.uint8, torch.float32
        pool, scales = pages + (d,), pages[:2]
    else:
        pool_type, pool = torch.bfloat16, pages + (d,)
    if k_rows is None or k_pool is None or (scale_type and k_scale is None):
        raise ValueError(f"{what}: k's rows, pool and (a quantised cache's) scales are wanted")
    _want(k_pool, "k_pool", pool_type, pool, dev)
    k_stride, v_stride = _token_rows(k_rows, "k rows", torch.bfloat16, rows, dev), 0
    k_at, v_at, v_pool_at, k_scale_at, v_scale_at = k_rows.data_ptr(), 0, 0, 0, 0
    if scale_type:
        _want(k_scale, "k_scale", scale_type, scales, dev)
        k_scale_at = k_scale.data_ptr()
    if not desc.kv_shared:
        if v_rows is None or v_pool is None or (scale_type and v_scale is None):
            raise ValueError(f"{what}: v's rows, pool and (a quantised cache's) scales are wanted")
        _want(v_pool, "v_pool", pool_type, pool, dev)
        v_stride = _token_rows(v_rows, "v rows", torch.bfloat16, rows, dev)
        v_at, v_pool_at = v_rows.data_ptr(), v_pool.data_ptr()
        if scale_type:
            _want(v_scale, "v_scale", scale_type, scales, dev)
            v_scale_at = v_scale.data_ptr()
    if not _is_word(device_flags, dev):
        _refuse_bytes("device_flags", device_flags, 4)
    raw = _launch_stream(stream, dev)
    args = _ROWS_ARGS(
        ctypes.addressof(desc), n, k_exp, v_exp, 0, k_at, v_at, k_stride, v_stride, slot_map.data_ptr(),
        k_pool.data_ptr(), v_pool_at, k_scale_at, v_scale_at, device_flags.data_ptr(), raw)
    lib = load_library()
    write = what == "paged_decode_write_slots_fp4"
    st = lib.paged_decode_write_slots_fp4_args(args) if write else lib.paged_decode_read_slots_args(args)
    if st != PD_OK:
        raise PagedDecodeError(st, what)


def paged_decode_write_slots_fp4(desc: LayerDesc, k_in, v_in, slot_map, k_pool, v_pool, k_scale, v_scale,
                                 device_flags, stream=None, *, k_exp: int = 0, v_exp: int = 0) -> None:
    """Quantise k_in / v_in [tokens, Hkv, d] (any token stride) into the rows of a 4-bit cache that slot_map names
    (codes and block scales); -1 skips a token. On a K=V layer v_exp is k_exp."""
    _slot_rows("paged_decode_write_slots_fp4", PD_KV_FP4_E2M1, desc, k_in, v_in, slot_map, k_pool, v_pool, k_scale,
               v_scale, k_exp, v_exp, device_flags, stream)


def paged_decode_read_slots(desc: LayerDesc, slot_map, k_pool, v_pool, k_out, v_out, device_flags, stream=None) -> None:
    """The cached rows that slot_map names into k_out / v_out bf16 [tokens, Hkv, d] (any token stride); -1 leaves a
    row as it is."""
    _slot_rows("paged_decode_read_slots", PD_KV_BF16, desc, k_out, v_out, slot_map, k_pool, v_pool, None, None, 0, 0,
               device_flags, stream)


def paged_decode_read_slots_fp8(desc: LayerDesc, slot_map, k_pool, v_pool, k_scale, v_scale, k_out, v_out,
                                device_flags, stream=None) -> None:
    """The same from e4m3 pools (uint8) with per-(page, KV head) scales."""
    _slot_rows("paged_decode_read_slots_fp8", PD_KV_FP8_E4M3, desc, k_out, v_out, slot_map, k_pool, v_pool, k_scale,
               v_scale, 0, 0, device_flags, stream)


def paged_decode_read_slots_fp4(desc: LayerDesc, slot_map, k_pool, v_pool, k_scale, v_scale, k_out, v_out,
                                device_flags, stream=None, *, k_exp: int = 0, v_exp: int = 0) -> None:
    """The same from a 4-bit cache."""
    _slot_rows("paged_decode_read_slots_fp4", PD_KV_FP4_E2M1, desc, k_out, v_out, slot_map, k_pool, v_pool, k_scale,
               v_scale, k_exp, v_exp, device_flags, stream)


def paged_decode_plan_shared(desc: LayerDesc, query_tokens: int, seq_lens_host: Sequence[int],
                             group_starts_host: Sequence[int], prefix_lens_host: Sequence[int], max_prefix_pages: int,
                             sm_count: int) -> SharedPlan:
    """Plan of a shared-prefix decode: group n is requests
    [group_starts[n], group_starts[n + 1]), its prefix prefix_lens[n] tokens;
    seq_lens count each request's own tokens."""
    def arr(v):
        return ctypes.cast((ctypes.c_int32 * max(1, len(v)))(*[int(x) for x in v]), ctypes.c_void_p)

    if len(group_starts_host) != len(prefix_lens_host) + 1:
        raise ValueError("group_starts has one entry more than prefix_lens")
    plan = SharedPlan()
    st = load_library().paged_decode_plan_shared(
        ctypes.byref(desc), len(seq_lens_host), int(query_tokens), arr(seq_lens_host), len(prefix_lens_host),
        arr(group_starts_host), arr(prefix_lens_host), int(max_prefix_pages), int(sm_count), ctypes.byref(plan))
    _check(st, "paged_decode_plan_shared")
    return plan


class _SharedShapes:
    """What the tensors of a shared-prefix decode have to look like, by its plan."""

    def __init__(self, plan: SharedPlan):
        ly, B, T = plan.own.layer, plan.own.batch, plan.own.query_tokens
        self.fp8 = ly.kv_dtype == PD_KV_FP8_E4M3
        self.q = (B, T, ly.num_q_heads, ly.head_dim)
        self.q_one = (B, ly.num_q_heads, ly.head_dim) if T == 1 else self.q
        self.pool = (ly.num_pages, ly.num_kv_heads, ly.page_size, ly.head_dim)
        self.prefix = (plan.num_groups, plan.max_prefix_pages)
        self.tables = (B, ly.max_pages_per_seq)

    def check(self, want, device, q, k_pool, v_pool, k_scale, v_scale, prefix_tables, prefix_lens, group_starts,
              block_tables, seq_lens, out) -> None:
        torch = _torch()
        i32, bf16 = torch.int32, torch.bfloat16
        pool_type = torch.uint8 if self.fp8 else bf16
        shape = self.q if len(getattr(q, "shape", ())) == 4 else self.q_one
        want(q, "q", bf16, shape, device)
        want(out, "out", bf16, shape, device)
        want(k_pool, "k_pool", pool_type, self.pool, device)
        if v_pool is not None:
            want(v_pool, "v_pool", pool_type, self.pool, device)
        if self.fp8:
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if t is not None:
                    want(t, name, torch.float32, self.pool[:2], device)
        want(prefix_tables, "prefix_tables", i32, self.prefix, device)
        want(prefix_lens, "prefix_lens", i32, self.prefix[:1], device)
        want(group_starts, "group_starts", i32, (self.prefix[0] + 1,), device)
        want(block_tables, "block_tables", i32, self.tables, device)
        want(seq_lens, "seq_lens", i32, self.tables[:1], device)


def _want_or_address(t, name: str, dtype, shape, device: int) -> None:
    """As _want; a raw address is the caller's word, and the library refuses what is missing."""
    if t is not None and not isinstance(t, int):
        _want(t, name, dtype, shape, device)


def _global_shared(fp8: bool, plan, q, k_pool, v_pool, k_scale, v_scale, prefix_tables, prefix_lens, group_starts,
                   block_tables, seq_lens, scale, workspace, out, stream, workspace_bytes) -> None:
    dev, nbytes = workspace.get_device(), workspace.nbytes if workspace_bytes is None else int(workspace_bytes)
    if workspace.nbytes < nbytes or not workspace.is_contiguous():
        _refuse_bytes("workspace", workspace, nbytes)
    _SharedShapes(plan).check(_want_or_address, dev, q, k_pool, v_pool, k_scale, v_scale, prefix_tables, prefix_lens,
                              group_starts, block_tables, seq_lens, out)
    st = _shared_status(fp8, plan, k_scale, v_scale, scale, workspace, nbytes, _launch_stream(stream, dev),
                        *(_ptr(t) or 0 for t in (q, k_pool, v_pool, prefix_tables, prefix_lens, group_starts,
                                                 block_tables, seq_lens, out)))
    _check(st, "paged_decode_global_shared_fp8" if fp8 else "paged_decode_global_shared")


def _shared_status(fp8: bool, plan, k_scale, v_scale, scale, workspace, workspace_bytes, stream, q, k_pool, v_pool,
                   *rest) -> int:
    """The call on addresses (rest: the prefix tables' to the lengths', then out's); 0 for what is not there."""
    *tables, out = rest
    return load_library().paged_decode_global_shared_args(_SHARED_ARGS(
        ctypes.addressof(plan), q, k_pool, v_pool, _ptr(k_scale) or 0, _ptr(v_scale) or 0, *tables, scale, fp8,
        workspace.data_ptr(), workspace.nbytes if workspace_bytes is None else int(workspace_bytes), out,
        _stream_ptr(stream) or 0))


def paged_decode_global_shared(plan: SharedPlan, q, k_pool, v_pool, prefix_tables, prefix_lens, group_starts,
                               block_tables, seq_lens, scale: float, workspace, out, stream=None,
                               workspace_bytes: Optional[int] = None) -> None:
    """Decode of a batch whose groups share prefixes, merge included. Tensors are checked against the plan; addresses
    (int) are taken as they are."""
    _global_shared(False, plan, q, k_pool, v_pool, None, None, prefix_tables, prefix_lens, group_starts, block_tables,
                   seq_lens, scale, workspace, out, stream, workspace_bytes)


def paged_decode_global_shared_fp8(plan: SharedPlan, q, k_pool, v_pool, k_scale, v_scale, prefix_tables, prefix_lens,
                                   group_starts, block_tables, seq_lens, scale: float, workspace, out, stream=None,
                                   workspace_bytes: Optional[int] = None) -> None:
    """The same over an e4m3 cache with per-(page, KV head) scales."""
    _global_shared(True, plan, q, k_pool, v_pool, k_scale, v_scale, prefix_tables, prefix_lens, group_starts,
                   block_tables, seq_lens, scale, workspace, out, stream, workspace_bytes)


class SharedPrefixStep:
    """Plan + workspace of a shared-prefix decode of one layer, reusable across
    steps whose groups are cut alike and whose lengths are no longer than the
    planned ones."""

    def __init__(self, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq, seq_lens_host,
                 *, group_starts, prefix_lens, max_prefix_pages, kv_shared=False, kv_dtype=PD_KV_BF16,
                 query_tokens=1, sm_count=None, device=None):
        import torch
        device = torch.device("cuda") if device is None else torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"a decode runs on a GPU, not on {device}")
        if sm_count is None:
            sm_count = torch.cuda.get_device_properties(device).multi_processor_count
        self.desc = layer_desc(num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq, 0,
                               kv_shared, kv_dtype)
        self.fp8 = kv_dtype == PD_KV_FP8_E4M3
        self.query_tokens = int(query_tokens)
        self.plan = paged_decode_plan_shared(self.desc, self.query_tokens, list(seq_lens_host), list(group_starts),
                                             list(prefix_lens), max_prefix_pages, sm_count)
        # zeroed once: the first word is the device error flag
        nbytes = int(self.plan.workspace_bytes)
        self.workspace = torch.zeros((nbytes + 255) // 256 * 256, dtype=torch.uint8, device=device)
        self._shapes = _SharedShapes(self.plan)

    def __call__(self, q, k_pool, v_pool, prefix_tables, prefix_lens, group_starts, block_tables, seq_lens, scale, out,
                 stream=None, k_scale=None, v_scale=None):
        dev = self.workspace.get_device()
        self._shapes.check(_want, dev, q, k_pool, v_pool, k_scale, v_scale, prefix_tables, prefix_lens, group_starts,
                           block_tables, seq_lens, out)
        raw = _launch_stream(stream, dev)
        st = _shared_status(self.fp8, self.plan, k_scale, v_scale, scale, self.workspace, None, raw, q.data_ptr(),
                            k_pool.data_ptr(), 0 if v_pool is None else v_pool.data_ptr(), prefix_tables.data_ptr(),
                            prefix_lens.data_ptr(), group_starts.data_ptr(), block_tables.data_ptr(),
                            seq_lens.data_ptr(), out.data_ptr())
        if st != PD_OK:
            raise PagedDecodeError(st, "paged_decode_global_shared_fp8" if self.fp8 else "paged_decode_global_shared")
        return out

    def check(self, stream=None) -> int:
        return paged_decode_check_device_error(self.plan.own, self.workspace, stream)
