"""Python binding of libmoe.so -- the routed sparse-MoE layer with expert
streaming on one GB300 (sm_103a).

Argument marshalling only (ctypes, and the small C module _call for the
operators without a context): every step of the layer runs in the library's
CUDA kernels.  The names mirror the C ABI in ``include/moe.h``.  Device buffers are
passed as CUDA torch tensors (fp32 / int32, contiguous) or raw integer device
addresses; streams as ``torch.cuda.Stream`` or raw ``cudaStream_t`` integers.

Importing the package does not need a GPU; loading the library does need the
built ``libmoe.so`` and raises if it is missing -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib
import os
import threading

import numpy as np

from ._build import LIB as _LIB_PATH, build  # noqa: F401

MOE_OK, MOE_EINVAL, MOE_ENOMEM, MOE_ECUDA, MOE_EPOOL, MOE_ETIMEOUT, MOE_ESTATE, MOE_EIO = 0, -1, -2, -3, -4, -5, -6, -7
MOE_STORE_DIRECT = 0x1
MOE_F32, MOE_BF16 = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_MX_E8M0, MOE_MX_E4M3 = 0, 1
MOE_ACT_NONE, MOE_ACT_SWIGLU, MOE_ACT_SILU = 0, 1, 2
MOE_NORM_NONE, MOE_NORM_RMS, MOE_NORM_L2 = 0, 1, 2
MOE_ROT_HALVES, MOE_ROT_ADJACENT = 0, 1
MOE_EVICT_LFU_RECENCY, MOE_EVICT_LRU, MOE_EVICT_LFU_PERSIST, MOE_EVICT_LFU_AGED = 0, 1, 2, 3
MOE_FAULT_PINNED_ALLOC, MOE_FAULT_MISS_COPY, MOE_FAULT_WAIT_TIMEOUT, MOE_FAULT_DEVICE_WAIT = 0x1, 0x2, 0x4, 0x8
_ERRNAMES = {MOE_EINVAL: "MOE_EINVAL", MOE_ENOMEM: "MOE_ENOMEM", MOE_ECUDA: "MOE_ECUDA", MOE_EPOOL: "MOE_EPOOL",
             MOE_ETIMEOUT: "MOE_ETIMEOUT", MOE_ESTATE: "MOE_ESTATE", MOE_EIO: "MOE_EIO"}

# every symbol include/moe.h declares
EXPORTS = (
    "moe_blob_bytes", "moe_blob_stride", "moe_pack_expert", "moe_create", "moe_destroy", "moe_load_experts",
    "moe_set_router_bias", "moe_set_router_bias_all", "moe_forward_decode", "moe_forward_decode_stack", "moe_forward_prefill",
    "moe_pool_stats", "moe_pool_reset", "moe_pool_trace", "moe_launch_count", "moe_prefill_profile", "moe_prefill_kernel_ms", "moe_route_noalloc", "moe_last_error", "moe_slotpool_create", "moe_slotpool_destroy",
    "moe_route", "moe_dispatch_workspace", "moe_dispatch", "moe_mx_bytes", "moe_mx_quantise", "moe_mx_dequantise",
    "moe_mx_product", "moe_mx_timeouts", "moe_mx_set_fault", "moe_combine", "moe_mx_quantise_rows", "moe_combine_rows",
    "moe_conv", "moe_head_norm", "moe_delta_workspace", "moe_delta",
    "moe_slotpool_request", "moe_store_create", "moe_store_write_layer", "moe_store_info", "moe_store_read",
)


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_ERRNAMES.get(code, code)}: {msg}")
        self.code = code


class moe_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_layers", "hidden", "n_experts", "top_k", "inter", "shared_inter", "bits", "group_size", "pool_slots",
        "norm_topk", "policy", "device", "max_batch", "max_tokens")] + [
        ("fault_flags", ctypes.c_uint32), ("fault_arg", ctypes.c_int32), ("timeout_ms", ctypes.c_int32),
        ("aging_period", ctypes.c_int32), ("store_flags", ctypes.c_uint32), ("store_path", ctypes.c_char_p),
        ("layer_bits", ctypes.POINTER(ctypes.c_int32))]


class moe_pool_stats_t(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_uint64), ("misses", ctypes.c_uint64), ("evictions", ctypes.c_uint64),
                ("h2d_bytes", ctypes.c_uint64), ("h2d_ms", ctypes.c_double), ("resident", ctypes.c_int32),
                ("calls", ctypes.c_int32)]


class moe_route_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_experts", "top_k", "n_groups", "top_groups", "group_best", "score",
                                              "renorm")] + [("scale", ctypes.c_float)]


class moe_mx(ctypes.Structure):
    device = -1  # ordinal of the GPU that holds the data; -1: not known, and not checked
    _fields_ = [("data_dev", ctypes.c_void_p), ("rows", ctypes.c_int64)] + [
        (n, ctypes.c_int32) for n in ("cols", "groups", "format", "ragged")]


class moe_seqs(ctypes.Structure):
    device = -1  # ordinal of the GPU that holds the lists; -1: not known, and not checked
    _fields_ = [(n, ctypes.c_void_p) for n in ("offsets_dev", "slot_dev", "carry_dev")] + [
        ("n", ctypes.c_int32), ("max_len", ctypes.c_int32)]


class moe_head_norm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dim", "norm", "rot_dim", "pairs")] + [
        ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)]


class moe_heads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x_dev", "y_dev", "gate_dev", "weight_dev")] + [
        (n, ctypes.c_int64) for n in ("x_ld", "x_head", "y_ld", "y_head", "gate_ld", "gate_head")] + [
        ("heads", ctypes.c_int32), ("type", ctypes.c_int32)]


class moe_delta_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("k_heads", "v_heads", "k_dim", "v_dim")] + [("scale", ctypes.c_float)]


_lock = threading.Lock()
_lib = None


def load_library(path: str | None = None):
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or _LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with int4_expert_streaming_gb300.build() "
                               "(this package has no CPU fallback)")
        lib = ctypes.CDLL(p)
        c, vp, i32, sz = ctypes, ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        lib.moe_blob_bytes.argtypes = [i32, i32, i32]
        lib.moe_blob_bytes.restype = sz
        lib.moe_blob_stride.argtypes = [i32, i32, i32]
        lib.moe_blob_stride.restype = sz
        lib.moe_pack_expert.argtypes = [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz]
        lib.moe_create.argtypes = [c.POINTER(moe_config), c.POINTER(vp)]
        lib.moe_destroy.argtypes = [vp]
        lib.moe_destroy.restype = None
        lib.moe_load_experts.argtypes = [vp, i32, vp, sz, vp, vp, vp, vp]
        lib.moe_set_router_bias.argtypes = [vp, i32, vp, vp]
        lib.moe_set_router_bias_all.argtypes = [vp, vp, vp]
        lib.moe_forward_decode.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp]
        lib.moe_forward_decode_stack.argtypes = [vp, i32, i32, vp, i32, vp, c.c_float, vp, vp, vp, vp]
        lib.moe_forward_prefill.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp]
        lib.moe_pool_stats.argtypes = [vp, i32, c.POINTER(moe_pool_stats_t)]
        lib.moe_pool_reset.argtypes = [vp, i32, i32, i32, vp]
        lib.moe_pool_trace.argtypes = [vp, vp, sz, c.POINTER(sz)]
        lib.moe_launch_count.argtypes = [vp, c.POINTER(c.c_uint64)]
        lib.moe_prefill_profile.argtypes = [vp, i32]
        lib.moe_route_noalloc.argtypes = [vp, i32, vp, i32, vp, vp, vp]
        lib.moe_prefill_kernel_ms.argtypes = [vp, c.POINTER(c.c_double), c.POINTER(c.c_int64)]
        lib.moe_last_error.argtypes = [vp]
        lib.moe_last_error.restype = c.c_char_p
        lib.moe_slotpool_create.argtypes = [i32, i32, i32, i32, c.POINTER(vp)]
        lib.moe_slotpool_destroy.argtypes = [vp]
        lib.moe_slotpool_destroy.restype = None
        lib.moe_slotpool_request.argtypes = [vp, vp, i32, vp]
        lib.moe_store_create.argtypes = [c.c_char_p, i32, i32, i32, i32, i32]
        lib.moe_store_write_layer.argtypes = [c.c_char_p, i32, vp, sz]
        lib.moe_store_info.argtypes = [c.c_char_p, c.POINTER(c.c_int32), c.POINTER(c.c_uint64)]
        lib.moe_store_read.argtypes = [c.c_char_p, i32, i32, vp, sz]
        i64, mx = c.c_int64, c.POINTER(moe_mx)
        lib.moe_route.argtypes = [c.POINTER(moe_route_config), vp, i32, i64, vp, i64, vp, vp, vp]
        lib.moe_dispatch_workspace.argtypes = [i64, i32, i32]
        lib.moe_dispatch_workspace.restype = sz
        lib.moe_dispatch.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        lib.moe_mx_bytes.argtypes = [mx]
        lib.moe_mx_bytes.restype = sz
        lib.moe_mx_quantise.argtypes = [mx, vp, i32, i64, i32, vp, vp, vp, vp, vp]
        lib.moe_mx_dequantise.argtypes = [mx, vp, vp, vp, vp, i32, i64, vp]
        lib.moe_mx_product.argtypes = [mx, mx, vp, vp, vp, i32, i64, vp]
        lib.moe_mx_quantise_rows.argtypes = [mx, vp, i64, i32, i64, i32, vp, vp, vp, vp, vp]
        lib.moe_combine_rows.argtypes = [vp, i64, i32, i64, vp, vp, i64, i32, i32, vp, i32, i64, vp]
        lib.moe_mx_timeouts.argtypes = [c.POINTER(c.c_uint64)]
        lib.moe_mx_set_fault.argtypes = [c.c_uint32]
        lib.moe_combine.argtypes = [vp, i32, i64, vp, vp, i64, i32, i32, vp, i32, i64, vp]
        seqs, heads = c.POINTER(moe_seqs), c.POINTER(moe_heads)
        lib.moe_conv.argtypes = [seqs, vp, i32, i64, i64, i32, vp, i32, i32, vp, i32, vp, i64, vp, i64, vp]
        lib.moe_head_norm.argtypes = [c.POINTER(moe_head_norm_config), heads, heads, vp, vp, i64, vp]
        lib.moe_delta_workspace.argtypes = [c.POINTER(moe_delta_config), i64, i32, i32]
        lib.moe_delta_workspace.restype = sz
        lib.moe_delta.argtypes = [c.POINTER(moe_delta_config), seqs, vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64,
                                  i64, vp, sz, vp]
        for name in EXPORTS:
            if name not in ("moe_delta_workspace", "moe_destroy", "moe_slotpool_destroy", "moe_blob_bytes", "moe_blob_stride",
                            "moe_last_error", "moe_dispatch_workspace", "moe_mx_bytes"):
                getattr(lib, name).restype = c.c_int
        _lib = lib
        return lib


def _check(rc: int, ctx=None) -> int:
    if rc < 0:
        msg = load_library().moe_last_error(ctx)
        raise MoeError(rc, msg.decode() if msg else "")
    return rc


def _ptr(t):
    """Device/host address of a torch tensor, numpy array, int or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        if not t.flags["C_CONTIGUOUS"]:
            raise ValueError("numpy array must be C-contiguous")
        return t.ctypes.data
    if hasattr(t, "data_ptr"):
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return t.data_ptr()
    raise TypeError(f"cannot take the address of {type(t)}")


def _dev(t, dtype_name: str):
    if t is None or isinstance(t, int):
        return _ptr(t)
    if not getattr(t, "is_cuda", False):
        raise ValueError("expected a CUDA tensor")
    if str(t.dtype) != "torch." + dtype_name:
        raise ValueError(f"expected torch.{dtype_name}, got {t.dtype}")
    return _ptr(t)


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


# --------------------------------------------------------------------------
# the C ABI, name for name
# --------------------------------------------------------------------------

def moe_blob_bytes(hidden: int, inter: int, bits: int) -> int:
    return int(load_library().moe_blob_bytes(hidden, inter, bits))


def moe_blob_stride(hidden: int, inter: int, bits: int) -> int:
    return int(load_library().moe_blob_stride(hidden, inter, bits))


def moe_pack_expert(hidden: int, inter: int, bits: int, expert: dict, out: np.ndarray | None = None) -> np.ndarray:
    """Pack one expert's quantised arrays (dict q_gate, sb_gate, q_up, sb_up,
    q_down, sb_down as produced by the input generator) into its blob."""
    stride = moe_blob_stride(hidden, inter, bits)
    if out is None:
        out = np.empty(stride, np.uint8)
    arrs = [np.ascontiguousarray(expert[k]) for k in ("q_gate", "sb_gate", "q_up", "sb_up", "q_down", "sb_down")]
    _check(load_library().moe_pack_expert(hidden, inter, bits, *[a.ctypes.data for a in arrs], _ptr(out),
                                          out.nbytes))
    return out


def moe_create(cfg: moe_config):
    h = ctypes.c_void_p()
    _check(load_library().moe_create(ctypes.byref(cfg), ctypes.byref(h)))
    return h.value


def moe_destroy(ctx) -> None:
    if ctx:
        load_library().moe_destroy(ctx)


def moe_load_experts(ctx, layer: int, blobs, stride: int, shared_blob, router_w, shared_gate_w, router_bias=None):
    """blobs: host uint8 [n_experts * stride]; shared_blob: host uint8; router_w,
    shared_gate_w: host uint16 bf16 bits; router_bias: host fp32 or None."""
    _check(load_library().moe_load_experts(ctx, layer, _ptr(blobs), stride, _ptr(shared_blob), _ptr(router_w),
                                           _ptr(shared_gate_w), _ptr(router_bias)), ctx)


def moe_set_router_bias(ctx, layer: int, bias_host, stream=None):
    _check(load_library().moe_set_router_bias(ctx, layer, _ptr(bias_host), _stream(stream)), ctx)


def moe_set_router_bias_all(ctx, bias_host, stream=None):
    """bias_host: contiguous fp32 host array [n_layers, n_experts]."""
    _check(load_library().moe_set_router_bias_all(ctx, _ptr(bias_host), _stream(stream)), ctx)


def moe_forward_decode(ctx, layer: int, x, B: int, y, topk_idx=None, topk_w=None, stream=None):
    _check(load_library().moe_forward_decode(ctx, layer, _dev(x, "float32"), B, _dev(y, "float32"),
                                             _dev(topk_idx, "int32"), _dev(topk_w, "float32"), _stream(stream)), ctx)


def moe_forward_decode_stack(ctx, layer0: int, n_layers: int, x, B: int, y, renorm_eps: float = 1e-6,
                             x_trace=None, idx_trace=None, y_trace=None, stream=None):
    _check(load_library().moe_forward_decode_stack(ctx, layer0, n_layers, _dev(x, "float32"), B,
                                                   _dev(y, "float32"), renorm_eps, _dev(x_trace, "float32"),
                                                   _dev(idx_trace, "int32"), _dev(y_trace, "float32"),
                                                   _stream(stream)), ctx)


def moe_forward_prefill(ctx, layer: int, x, T: int, y, topk_idx=None, topk_w=None, stream=None):
    _check(load_library().moe_forward_prefill(ctx, layer, _dev(x, "float32"), T, _dev(y, "float32"),
                                              _dev(topk_idx, "int32"), _dev(topk_w, "float32"), _stream(stream)),
           ctx)


def moe_route_noalloc(ctx, layer: int, x, B: int, topk_idx, topk_w, stream=None):
    _check(load_library().moe_route_noalloc(ctx, layer, _dev(x, "float32"), B, _dev(topk_idx, "int32"),
                                            _dev(topk_w, "float32"), _stream(stream)), ctx)


def moe_pool_reset(ctx, slots: int, policy: int = MOE_EVICT_LFU_RECENCY, aging_period: int = 0, stream=None) -> None:
    """Empty every layer's pool, use `slots` of the reserved slots and evict by `policy` (streaming contexts)."""
    _check(load_library().moe_pool_reset(ctx, slots, policy, aging_period, _stream(stream)), ctx)


def moe_pool_stats(ctx, layer: int = -1) -> dict:
    s = moe_pool_stats_t()
    _check(load_library().moe_pool_stats(ctx, layer, ctypes.byref(s)), ctx)
    return {f: getattr(s, f) for f, _ in s._fields_}


def moe_pool_trace(ctx) -> np.ndarray:
    n = ctypes.c_size_t()
    lib = load_library()
    _check(lib.moe_pool_trace(ctx, None, 0, ctypes.byref(n)), ctx)
    buf = np.empty((n.value, 6), np.int32)
    _check(lib.moe_pool_trace(ctx, _ptr(buf) if n.value else None, n.value, ctypes.byref(n)), ctx)
    return buf


PREFILL_KERNELS = ("router_logits", "select", "histogram", "scan", "scatter", "gather_x", "gateup_gemm", "down_gemm")


def moe_prefill_profile(ctx, enable: bool = True) -> None:
    _check(load_library().moe_prefill_profile(ctx, int(bool(enable))), ctx)


def moe_prefill_kernel_ms(ctx) -> tuple:
    """-> ({kernel name: accumulated device ms}, recorded calls)"""
    ms = (ctypes.c_double * len(PREFILL_KERNELS))()
    n = ctypes.c_int64()
    _check(load_library().moe_prefill_kernel_ms(ctx, ms, ctypes.byref(n)), ctx)
    return dict(zip(PREFILL_KERNELS, list(ms))), n.value


def moe_launch_count(ctx) -> int:
    n = ctypes.c_uint64()
    _check(load_library().moe_launch_count(ctx, ctypes.byref(n)), ctx)
    return int(n.value)


def moe_last_error(ctx=None) -> str:
    m = load_library().moe_last_error(ctx)
    return m.decode() if m else ""


def moe_slotpool_create(slots: int, n_experts: int, policy: int = MOE_EVICT_LFU_RECENCY, aging_period: int = 0):
    h = ctypes.c_void_p()
    _check(load_library().moe_slotpool_create(slots, n_experts, policy, aging_period, ctypes.byref(h)))
    return h.value


def moe_slotpool_destroy(pool) -> None:
    if pool:
        load_library().moe_slotpool_destroy(pool)


def moe_slotpool_request(pool, req) -> list:
    """req: distinct ascending expert ids -> [(expert, kind, slot, evicted)]."""
    r = np.ascontiguousarray(req, np.int32)
    ev = np.empty((max(len(r), 1), 4), np.int32)
    n = _check(load_library().moe_slotpool_request(pool, _ptr(r) if len(r) else None, len(r), _ptr(ev)))
    return [tuple(int(v) for v in ev[i]) for i in range(n)]


def make_config(n_layers, hidden, n_experts, top_k, inter, shared_inter, bits=4, pool_slots=None, norm_topk=True,
                policy=MOE_EVICT_LFU_RECENCY, device=0, max_batch=1, max_tokens=0, fault_flags=0, fault_arg=0,
                timeout_ms=0, aging_period=0, store_path=None, store_flags=0, layer_bits=None) -> moe_config:
    """store_path: an expert container (moe_store_create) for a streaming context;
    layer_bits: 4 or 8 per layer (a mixed store).  The library copies both at
    moe_create; until then the struct keeps the Python-side buffers alive."""
    lb = None
    if layer_bits is not None:
        lb = (ctypes.c_int32 * len(layer_bits))(*[int(b) for b in layer_bits])
    cfg = moe_config(n_layers, hidden, n_experts, top_k, inter, shared_inter, bits, 64,
                     n_experts if pool_slots is None else pool_slots, int(norm_topk), policy, device, max_batch,
                     max_tokens, fault_flags, fault_arg, timeout_ms, aging_period, store_flags,
                     os.fsencode(store_path) if store_path is not None else None,
                     ctypes.cast(lb, ctypes.POINTER(ctypes.c_int32)) if lb is not None else None)
    cfg._layer_bits = lb  # keeps the array alive with the struct
    return cfg


# --------------------------------------------------------------------------
# operators without a context: CUDA tensors in, shapes and strides taken from
# them; outputs are the caller's tensors.  _call (csrc/binding.c) takes the
# tensors apart; one that does not fit, or is on another GPU than the current
# one, raises ValueError.  stream=None is the legacy default stream, as in the
# calls above, not torch's current one: within torch.cuda.stream(s) pass s.
# --------------------------------------------------------------------------

_ops = None


def _binding():
    global _ops
    if _ops is None:
        load_library()
        import torch

        from . import _build

        mod = importlib.import_module("._call", __name__)  # built beside libmoe.so
        if mod.built_for() != _build.built_for(torch.__version__):
            raise RuntimeError(f"_call.so was built for {mod.built_for()}, not for {_build.built_for(torch.__version__)}: "
                               "build it again with int4_expert_streaming_gb300.build()")
        mod.dtypes(torch.float32, torch.bfloat16, torch.int32, torch.uint8)
        mod.on_failure(_check)
        _ops = mod
    return _ops


def make_route_config(n_experts, top_k, n_groups=1, top_groups=1, group_best=1, score=MOE_SCORE_SOFTMAX, renorm=True,
                      scale=1.0) -> moe_route_config:
    return moe_route_config(n_experts, top_k, n_groups, top_groups, group_best, score, int(bool(renorm)), scale)


def moe_route(cfg: moe_route_config, logits, bias, idx, w, stream=None) -> None:
    """logits [T, n_experts] fp32 or bf16 (rows may be strided), bias [n_experts] fp32 or None; fills idx [T, top_k]
    int32 and w [T, top_k] fp32."""
    rc = (_ops or _binding()).route(cfg, logits, bias, idx, w, stream)
    if rc:
        _check(rc)


def moe_dispatch_workspace(T: int, top_k: int, n_experts: int) -> int:
    return int(load_library().moe_dispatch_workspace(T, top_k, n_experts))


def moe_dispatch(idx, n_experts: int, offsets, row_of_pair, token_of_row, group_of_row, workspace=None,
                 stream=None) -> None:
    """idx [T, top_k] int32 -> offsets [n_experts + 1], row_of_pair [T, top_k], token_of_row and group_of_row
    [T * top_k], all int32; workspace: uint8, moe_dispatch_workspace() bytes."""
    rc = (_ops or _binding()).dispatch(idx, n_experts, offsets, row_of_pair, token_of_row, group_of_row, workspace, stream)
    if rc:
        _check(rc)


def moe_mx_bytes(m: moe_mx) -> int:
    return int(load_library().moe_mx_bytes(m))


def make_mx(fmt: int, rows: int, cols: int, groups: int = 1, ragged: bool = False, data=None) -> moe_mx:
    """Descriptor of a microscaled 4-bit matrix (see moe_mx in moe.h) over `data`, a contiguous CUDA uint8 tensor of at
    least moe_mx_bytes() bytes (kept alive by the descriptor; allocated on the current device if None)."""
    import torch

    m = moe_mx(None, rows, cols, groups, fmt, int(bool(ragged)))
    need = moe_mx_bytes(m)
    if need == 0 and rows != 0:
        raise ValueError(f"bad matrix shape: format {fmt}, {groups} groups, {rows} rows, {cols} columns")
    if data is None:
        data = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    if not data.is_cuda or data.dtype is not torch.uint8 or not data.is_contiguous() or data.numel() < need:
        raise ValueError(f"data: expected a contiguous CUDA tensor of at least {need} uint8, got {tuple(data.shape)} "
                         f"{data.dtype} on {data.device}")
    m.data_dev = data.data_ptr()
    m._data = data
    m.device = data.get_device()
    return m


def moe_mx_quantise(m: moe_mx, src, act: int = MOE_ACT_NONE, src_row=None, group_of_row=None, offsets=None,
                    tensor_scale=None, stream=None) -> None:
    """Rows of src (fp32 or bf16, [source rows, cols] or [.., 2 cols] for MOE_ACT_SWIGLU) into m; a src_row that is none
    of them leaves its row unwritten."""
    rc = (_ops or _binding()).quantise(m, src, act, src_row, group_of_row, offsets, tensor_scale, stream)
    if rc:
        _check(rc)


def moe_mx_dequantise(m: moe_mx, dst, group_of_row=None, offsets=None, tensor_scale=None, stream=None) -> None:
    """The numbers of m into dst [rows, cols], fp32 or bf16."""
    rc = (_ops or _binding()).dequantise(m, dst, group_of_row, offsets, tensor_scale, stream)
    if rc:
        _check(rc)


def moe_mx_product(x: moe_mx, w: moe_mx, y, offsets=None, alpha=None, stream=None) -> None:
    """y [x.rows, w.rows] (fp32 or bf16) = alpha[group] * X W[group]^T."""
    rc = (_ops or _binding()).product(x, w, y, offsets, alpha, stream)
    if rc:
        _check(rc)


def moe_mx_timeouts() -> int:
    """Grows when a wait inside a product on the current device has run out and left its y incomplete; read it after a
    synchronise and compare."""
    n = ctypes.c_uint64()
    _check(load_library().moe_mx_timeouts(n))
    return n.value


def moe_mx_set_fault(fault_flags: int) -> None:
    """Tests only: this thread's products get a wait that nothing ends (MOE_FAULT_DEVICE_WAIT), or none (0)."""
    _check(load_library().moe_mx_set_fault(fault_flags))


def moe_combine(rows, row_of_pair, w, y, stream=None) -> None:
    """y [T, cols] = sum_j w[T, k] * rows[row_of_pair[T, k]]; rows and y fp32 or bf16.  Pairs whose row is none of rows
    are skipped."""
    rc = (_ops or _binding()).combine(rows, row_of_pair, w, y, stream)
    if rc:
        _check(rc)


def make_seqs(n: int, offsets=None, slot=None, carry=None, max_len: int = 0) -> moe_seqs:
    """Descriptor of a batch of n sequences (see moe_seqs in moe.h): offsets [n + 1] (None: each row is a sequence), slot
    [n] and carry [n], contiguous int32 CUDA tensors, kept alive by the descriptor."""
    import torch

    q = moe_seqs(None, None, None, n, max_len)
    for name, t, need in (("offsets", offsets, n + 1), ("slot", slot, n), ("carry", carry, n)):
        if t is None:
            continue
        if not t.is_cuda or t.dtype is not torch.int32 or not t.is_contiguous() or t.numel() < need:
            raise ValueError(f"{name}: expected a contiguous CUDA tensor of at least {need} int32, got {tuple(t.shape)} "
                             f"{t.dtype} on {t.device}")
        if q.device >= 0 and t.get_device() != q.device:
            raise ValueError(f"{name}: is on GPU {t.get_device()}, another list on GPU {q.device}")
        q.device = t.get_device()
        setattr(q, name + "_dev", t.data_ptr())
    q._lists = (offsets, slot, carry)
    return q


def make_head_norm_config(norm: int = MOE_NORM_RMS, eps: float = 1e-6, weight_offset: float = 0.0, rot_dim: int = 0,
                          pairs: int = MOE_ROT_HALVES) -> moe_head_norm_config:
    """Without the heads' dimension, which a call takes from its tensors."""
    return moe_head_norm_config(0, norm, rot_dim, pairs, eps, weight_offset)


def moe_delta_workspace(T: int, n: int, k_heads: int, v_heads: int, k_dim: int, v_dim: int, max_len: int = 0) -> int:
    return int(load_library().moe_delta_workspace(moe_delta_config(k_heads, v_heads, k_dim, v_dim, 1.0), T, n, max_len))


def __getattr__(name):
    """moe_conv, moe_head_norm and moe_delta are _call's own functions, found when first asked for."""
    if name in ("moe_conv", "moe_head_norm", "moe_delta"):
        globals()[name] = f = getattr(_binding(), name)
        return f
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


# --------------------------------------------------------------------------
# expert container (routed blobs on disk; host only)
# --------------------------------------------------------------------------

def moe_store_create(path, n_layers: int, n_experts: int, hidden: int, inter: int, bits: int) -> None:
    _check(load_library().moe_store_create(os.fsencode(path), n_layers, n_experts, hidden, inter, bits))


def moe_store_write_layer(path, layer: int, blobs, stride: int) -> None:
    """blobs: host uint8 [n_experts * stride] (the layer's packed routed blobs)."""
    b = np.ascontiguousarray(blobs, np.uint8)
    _check(load_library().moe_store_write_layer(os.fsencode(path), layer, _ptr(b), stride))


def moe_store_info(path) -> dict:
    shape = (ctypes.c_int32 * 5)()
    stride = ctypes.c_uint64()
    _check(load_library().moe_store_info(os.fsencode(path), shape, ctypes.byref(stride)))
    return dict(zip(("n_layers", "n_experts", "hidden", "inter", "bits"), list(shape)), stride=stride.value)


def moe_store_read(path, layer: int, expert: int, stride: int) -> np.ndarray:
    out = np.empty(stride, np.uint8)
    _check(load_library().moe_store_read(os.fsencode(path), layer, expert, _ptr(out), stride))
    return out
