"""Python binding of the CLO C ABI (``include/clo.h``): argument marshalling only.

The functions carry the C names; every step of the decode path runs in the CUDA
library ``_lib/libclo.so``.  The calls on a paged cache, made once per layer and step, are
marshalled by a compiled module beside it.  There is no fallback: if the library is missing or
fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libclo.so")

CLO_OK, CLO_ERR_INVALID, CLO_ERR_OOM, CLO_ERR_CUDA, CLO_ERR_TIMEOUT, CLO_ERR_STATE, CLO_ERR_CAPACITY, \
    CLO_ERR_DEVICE = range(8)
CLO_DEC_HIT, CLO_DEC_MISS, CLO_DEC_PERSIST = 0, 1, 2
(CLO_DBG_KEY_CODES, CLO_DBG_QUERY_CODES, CLO_DBG_IDX, CLO_DBG_DECISION, CLO_DBG_SLOT_ROWS, CLO_DBG_TAU,
 CLO_DBG_PERSIST, CLO_DBG_SHAT, CLO_DBG_COS, CLO_DBG_TIMELINE, CLO_DBG_TOPK, CLO_DBG_POOL_NODE,
 CLO_DBG_STEP_BYTES) = range(1, 14)
STEP_HIST = 4096
CLO_SET_DROP_FLAG_LAYER, CLO_SET_WAIT_TIMEOUT_NS = 1, 2
CLO_ROPE_SCALING = {"none": 0, "linear": 1, "bands": 2, "yarn": 3}
CLO_ROPE_ORDER = {"sections": 0, "cycled": 1}
CLO_ROPE_MAX_PAIRS = 64
CLO_ROPE_MAX_AXES = 4

_STATUS_NAMES = {0: "CLO_OK", 1: "CLO_ERR_INVALID", 2: "CLO_ERR_OOM", 3: "CLO_ERR_CUDA", 4: "CLO_ERR_TIMEOUT",
                 5: "CLO_ERR_STATE", 6: "CLO_ERR_CAPACITY", 7: "CLO_ERR_DEVICE"}

EXPORTED = ["clo_config_default", "clo_init", "clo_destroy", "clo_append_kv", "clo_append_step", "clo_decode_step",
            "clo_decode_layer",
            "clo_sync", "clo_stats", "clo_last_error", "clo_debug_get", "clo_set", "clo_sparse_attention_noalloc",
            "clo_rope_config_default", "clo_rope_plan_init", "clo_rope", "clo_paged_append", "clo_paged_read",
            "clo_paged_attention", "clo_paged_attention_workspace"]


class CLOError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {_STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class clo_config(ctypes.Structure):
    _fields_ = [
        ("n_layers", ctypes.c_int32),
        ("batch", ctypes.c_int32),
        ("n_q_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("max_tokens", ctypes.c_int64),
        ("topk", ctypes.c_int64),
        ("topk_ratio", ctypes.c_double),
        ("hash_R", ctypes.c_void_p),
        ("tau", ctypes.c_void_p),
        ("persist_mask", ctypes.c_void_p),
        ("warmup_steps", ctypes.c_int32),
        ("tau_offset", ctypes.c_float),
        ("n_persist", ctypes.c_int32),
        ("wait_timeout_ns", ctypes.c_int64),
        ("timing", ctypes.c_int32),
        ("debug_drop_flag_layer", ctypes.c_int32),
        ("stream", ctypes.c_void_p),
        ("adaptive_tau", ctypes.c_int32),
        ("tau_ema", ctypes.c_double),
        ("kv_bits", ctypes.c_int32),
    ]


class clo_stats_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "steps", "units_hit", "units_miss", "units_persist", "host_bytes", "hbm_bytes_alg", "timeouts",
        "last_hit", "last_miss", "last_persist", "last_host_bytes", "last_hbm_bytes_alg")] + \
        [("warmup_done", ctypes.c_int32), ("timed_steps", ctypes.c_int32)] + \
        [(n, ctypes.c_float) for n in ("last_ms_decide", "last_ms_fused", "last_ms_total")] + \
        [(n, ctypes.c_double) for n in ("sum_ms_decide", "sum_ms_fused", "sum_ms_total")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class clo_rope_config(ctypes.Structure):
    _fields_ = [
        ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("theta", ctypes.c_double),
        ("scaling", ctypes.c_int32),
        ("factor", ctypes.c_double),
        ("low_freq", ctypes.c_double),
        ("high_freq", ctypes.c_double),
        ("beta_fast", ctypes.c_double),
        ("beta_slow", ctypes.c_double),
        ("original_max", ctypes.c_int64),
        ("magnitude", ctypes.c_double),
        ("n_axes", ctypes.c_int32),
        ("axis_pairs", ctypes.c_int32 * CLO_ROPE_MAX_AXES),
        ("axis_order", ctypes.c_int32),
        ("axis_own_freqs", ctypes.c_int32),
    ]


class clo_rope_plan(ctypes.Structure):
    _fields_ = [
        ("turn", ctypes.c_uint64 * CLO_ROPE_MAX_PAIRS),
        ("magnitude", ctypes.c_float),
        ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("ready", ctypes.c_int32),
        ("axis", ctypes.c_uint8 * CLO_ROPE_MAX_PAIRS),
        ("n_axes", ctypes.c_int32),
    ]


class clo_rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_token", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


class clo_paged_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages", "k_scales", "v_scales")] + \
        [(n, ctypes.c_int64) for n in ("n_pages", "k_stride_page", "k_stride_head", "k_stride_token", "v_stride_page",
                                       "v_stride_head", "v_stride_token")] + \
        [(n, ctypes.c_int32) for n in ("n_kv_heads", "head_dim", "page_size", "kv_bits")] + \
        [(n, ctypes.c_void_p) for n in ("k_group_scales", "v_group_scales")]


class clo_paged_batch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q_starts", "kv_lens", "block_table")] + \
        [("table_stride", ctypes.c_int64)] + \
        [(n, ctypes.c_int32) for n in ("max_pages", "batch", "total_q", "max_q")]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libclo.so (raises if it is missing: the package has no CPU path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library {path} is missing; build it with __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.clo_config_default.restype = None
    lib.clo_config_default.argtypes = [ctypes.POINTER(clo_config)]
    lib.clo_init.restype = ctypes.c_int
    lib.clo_init.argtypes = [ctypes.POINTER(clo_config), ctypes.POINTER(vp)]
    lib.clo_destroy.restype = ctypes.c_int
    lib.clo_destroy.argtypes = [vp]
    lib.clo_append_kv.restype = ctypes.c_int
    lib.clo_append_kv.argtypes = [vp, i32, i32, vp, vp, i64, i32]
    lib.clo_decode_step.restype = ctypes.c_int
    lib.clo_decode_step.argtypes = [vp, vp, vp, i32]
    lib.clo_append_step.restype = ctypes.c_int
    lib.clo_append_step.argtypes = [vp, vp, vp, i32]
    lib.clo_decode_layer.restype = ctypes.c_int
    lib.clo_decode_layer.argtypes = [vp, i32, vp, vp, i32]
    lib.clo_sync.restype = ctypes.c_int
    lib.clo_sync.argtypes = [vp]
    lib.clo_stats.restype = ctypes.c_int
    lib.clo_stats.argtypes = [vp, ctypes.POINTER(clo_stats_t)]
    lib.clo_last_error.restype = ctypes.c_char_p
    lib.clo_last_error.argtypes = []
    lib.clo_debug_get.restype = ctypes.c_int
    lib.clo_debug_get.argtypes = [vp, i32, i32, i32, i32, vp, i64]
    lib.clo_set.restype = ctypes.c_int
    lib.clo_set.argtypes = [vp, i32, i64]
    lib.clo_sparse_attention_noalloc.restype = ctypes.c_int
    lib.clo_sparse_attention_noalloc.argtypes = [vp, vp, vp, i32, i32, i32, i64, vp]
    lib.clo_rope_config_default.restype = None
    lib.clo_rope_config_default.argtypes = [vp]
    lib.clo_rope_plan_init.restype = ctypes.c_int
    lib.clo_rope_plan_init.argtypes = [vp, vp]
    lib.clo_rope.restype = ctypes.c_int
    lib.clo_rope.argtypes = [vp, vp, vp, vp, i64, i32, i32, i32, vp]
    lib.clo_paged_append.restype = ctypes.c_int
    lib.clo_paged_append.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, vp]
    lib.clo_paged_read.restype = ctypes.c_int
    lib.clo_paged_read.argtypes = [vp, vp, vp, vp, vp]
    lib.clo_paged_attention.restype = ctypes.c_int
    lib.clo_paged_attention.argtypes = [vp, vp, vp, vp, i32, ctypes.c_float, i32, i32, vp, i64, vp]
    lib.clo_paged_attention_workspace.restype = ctypes.c_int
    lib.clo_paged_attention_workspace.argtypes = [vp, vp, i32, i32, i32, ctypes.POINTER(i64)]
    _lib = lib
    return lib


def clo_last_error() -> str:
    return load_library().clo_last_error().decode(errors="replace")


def _check(status: int, where: str):
    if status != CLO_OK:
        raise CLOError(status, where, clo_last_error())


def _ptr(x):
    """(pointer, on_device) of a numpy array or torch tensor (must be contiguous)."""
    if isinstance(x, np.ndarray):
        if not x.flags["C_CONTIGUOUS"]:
            raise ValueError("array must be C-contiguous")
        return x.ctypes.data, False
    if hasattr(x, "data_ptr"):
        if not x.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return x.data_ptr(), x.device.type == "cuda"
    if isinstance(x, int):
        return x, None
    raise TypeError(f"unsupported buffer type {type(x)}")


# ----------------------------------------------------------------------------- C names
def clo_config_default() -> clo_config:
    cfg = clo_config()
    load_library().clo_config_default(ctypes.byref(cfg))
    return cfg


def clo_init(cfg: clo_config) -> ctypes.c_void_p:
    ctx = ctypes.c_void_p()
    _check(load_library().clo_init(ctypes.byref(cfg), ctypes.byref(ctx)), "clo_init")
    return ctx


def clo_destroy(ctx) -> None:
    _check(load_library().clo_destroy(ctx), "clo_destroy")


def clo_append_kv(ctx, layer: int, seq: int, k, v, n_tokens: int, src_is_device: bool | None = None) -> None:
    kp, kdev = _ptr(k)
    vp_, vdev = _ptr(v)
    dev = kdev if src_is_device is None else bool(src_is_device)
    _check(load_library().clo_append_kv(ctx, layer, seq, kp, vp_, int(n_tokens), int(bool(dev))), "clo_append_kv")


def clo_append_step(ctx, k, v, src_is_device: bool | None = None) -> None:
    kp, kdev = _ptr(k)
    vp_, vdev = _ptr(v)
    dev = kdev if src_is_device is None else bool(src_is_device)
    _check(load_library().clo_append_step(ctx, kp, vp_, int(bool(dev))), "clo_append_step")


def clo_decode_step(ctx, q, out, io_on_device: bool | None = None) -> None:
    qp, qdev = _ptr(q)
    op, odev = _ptr(out)
    dev = qdev if io_on_device is None else bool(io_on_device)
    _check(load_library().clo_decode_step(ctx, qp, op, int(bool(dev))), "clo_decode_step")


def clo_decode_layer(ctx, layer: int, q, out, io_on_device: bool | None = None) -> None:
    qp, qdev = _ptr(q)
    op, odev = _ptr(out)
    dev = qdev if io_on_device is None else bool(io_on_device)
    _check(load_library().clo_decode_layer(ctx, int(layer), qp, op, int(bool(dev))), "clo_decode_layer")


def clo_sync(ctx) -> None:
    _check(load_library().clo_sync(ctx), "clo_sync")


def clo_stats(ctx) -> dict:
    st = clo_stats_t()
    _check(load_library().clo_stats(ctx, ctypes.byref(st)), "clo_stats")
    return st.as_dict()


def clo_debug_get(ctx, what: int, layer: int, seq: int, kvh: int, dst: np.ndarray) -> np.ndarray:
    p, _ = _ptr(dst)
    _check(load_library().clo_debug_get(ctx, what, layer, seq, kvh, p, dst.nbytes), "clo_debug_get")
    return dst


def clo_set(ctx, key: int, value: int) -> None:
    _check(load_library().clo_set(ctx, key, int(value)), "clo_set")


def clo_sparse_attention_noalloc(q, rows, out, n_groups: int, group_size: int, head_dim: int, k: int,
                                 stream=None) -> None:
    """Allocation-free sparse attention (device buffers; see include/clo.h).

    q: bf16 (int16/uint16 bit patterns) [n_groups][group_size][head_dim], rows: bf16
    [n_groups][>= k][2][head_dim], out: fp32 [n_groups][group_size][head_dim]; all
    three CUDA tensors on the current device.  Plain integers are passed through as raw
    device addresses (the caller vouches for them)."""
    import torch

    G, D, n = int(group_size), int(head_dim), int(n_groups)
    want = {"q": (q, n * G * D, (torch.int16, torch.uint16, torch.bfloat16)),
            "rows": (rows, n * int(k) * 2 * D, (torch.int16, torch.uint16, torch.bfloat16)),
            "out": (out, n * G * D, (torch.float32,))}
    for name, (t, numel, dtypes) in want.items():
        if isinstance(t, int):
            continue
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, not on the current device")
        if t.dtype not in dtypes:
            raise ValueError(f"{name} has dtype {t.dtype}; expected one of {dtypes}")
        if (t.numel() < numel) if name == "rows" else (t.numel() != numel):
            raise ValueError(f"{name} holds {t.numel()} elements; expected {numel}")
    qp, _ = _ptr(q)
    rp, _ = _ptr(rows)
    op, _ = _ptr(out)
    _check(load_library().clo_sparse_attention_noalloc(qp, rp, op, int(n_groups), int(group_size), int(head_dim),
                                                       int(k), stream), "clo_sparse_attention_noalloc")


# ----------------------------------------------------------------------------- rotary positions, paged cache
def clo_rope_config_default() -> clo_rope_config:
    cfg = clo_rope_config()
    load_library().clo_rope_config_default(ctypes.byref(cfg))
    return cfg


def clo_rope_plan_init(cfg: clo_rope_config | None = None, **fields) -> clo_rope_plan:
    """Plan of a rotation: from a config, or from its fields (scaling by name: "none", "linear",
    "bands", "yarn").  The plan holds plain values and may serve any number of calls.

    axis_pairs: the pairs of each axis where tokens have positions on several, for example (16, 24, 24) for time,
    height and width; axis_order by name: "sections", "cycled".  Such a plan takes positions [n_axes][n_tokens]."""
    if cfg is not None and fields:
        raise TypeError("a config and its fields exclude each other")
    if cfg is not None and not isinstance(cfg, clo_rope_config):
        raise TypeError(f"cfg must be a clo_rope_config, not {type(cfg).__name__}")
    if cfg is None:
        cfg = clo_rope_config_default()
        for name, value in fields.items():
            if name not in _ROPE_FIELDS:
                raise TypeError(f"clo_rope_config has no field {name!r}")
            if name == "scaling" and isinstance(value, str):
                if value not in CLO_ROPE_SCALING:
                    raise ValueError(f"unknown scaling {value!r}; known: {sorted(CLO_ROPE_SCALING)}")
                value = CLO_ROPE_SCALING[value]
            if name == "axis_order" and isinstance(value, str):
                if value not in CLO_ROPE_ORDER:
                    raise ValueError(f"unknown axis_order {value!r}; known: {sorted(CLO_ROPE_ORDER)}")
                value = CLO_ROPE_ORDER[value]
            if name == "axis_pairs":
                value = tuple(value)
                if not 1 <= len(value) <= CLO_ROPE_MAX_AXES:
                    raise ValueError(f"axis_pairs has {len(value)} axes; 1 .. {CLO_ROPE_MAX_AXES} are possible")
                if fields.get("n_axes", len(value)) != len(value):
                    raise ValueError("n_axes is not the length of axis_pairs")
                cfg.n_axes = len(value)
                value = (ctypes.c_int32 * CLO_ROPE_MAX_AXES)(*value)
            setattr(cfg, name, int(value) if name in ("interleaved", "axis_own_freqs") else value)
    plan = clo_rope_plan()
    _check(load_library().clo_rope_plan_init(ctypes.byref(cfg), ctypes.byref(plan)), "clo_rope_plan_init")
    return plan


_ROPE_FIELDS = {n for n, _ in clo_rope_config._fields_}


def _plan_address(plan) -> int:
    if not isinstance(plan, clo_rope_plan):
        raise TypeError(f"the plan of a rotation must be a clo_rope_plan, not {type(plan).__name__}")
    return ctypes.addressof(plan)


_torch_binding = None


def _fast():
    """The compiled binding for torch tensors (csrc/clo_torch.cpp): checks, new outputs, marshalling."""
    global _torch_binding
    if _torch_binding is None:
        import importlib.machinery
        import importlib.util

        import torch

        from ._build import torch_lib

        load_library()
        path = torch_lib(torch.__version__)
        if not os.path.exists(path):
            raise RuntimeError(f"binding {path} is missing; build it with __graft_entry__.build()")
        loader = importlib.machinery.ExtensionFileLoader("_clo_torch", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_clo_torch", loader))
        loader.exec_module(module)
        _torch_binding = module
    return _torch_binding


def clo_rope(plan: clo_rope_plan, x, positions, out=None, transpose: bool = False, stream=None):
    """Rotates bf16 rows [n_tokens][n_heads][head_dim] by int64 positions [n_tokens] (see include/clo.h), or
    [n_axes][n_tokens] where the plan has several axes.

    out: rows of the same shape, x itself for in place, or None for new ones.  transpose applies the
    transposed rotation, which takes the gradient of the output to that of x: the call itself is not recorded by autograd,
    and refuses an x that requires a gradient while gradients are recorded.  Returns out."""
    r = (_torch_binding or _fast()).rope(_plan_address(plan), x, positions, out, transpose, stream)
    if type(r) is int:
        _check(r, "clo_rope")
    return r


class PagedCache:
    """K/V pages in HBM (see include/clo.h): the caller's tensors, and the calls on them.

    k_pages, v_pages: [n_pages][n_kv_heads][page_size][head_dim], bf16 or float8_e4m3fn, any strides that are
    multiples of 16 bytes with head_dim contiguous (pages laid out token by token: pass
    ``pages.transpose(1, 2)``).  8-bit pages come with contiguous fp32 scales [n_pages][n_kv_heads].

    4-bit pages: uint8 [n_pages][n_kv_heads][page_size][head_dim / 2], two codes to a byte, with the same scales and contiguous
    float8_e4m3fn group scales [n_pages][n_kv_heads][page_size][head_dim / 16], one per 16 elements of a row.

    The calls take the batch as q_starts int32 [batch + 1], kv_lens int32 [batch] (the call's tokens included)
    and block_table int32 [batch][max_pages]; max_q is the most rows that a sequence has (default: all
    rows of the call, which is right for one sequence; a step of single tokens passes 1).

    stream None is torch's current stream; otherwise a torch stream or a handle.  New outputs belong to the stream of the
    call, as under ``torch.cuda.stream``: another stream that uses them waits for it first.

    Autograd records none of the calls; rows that require a gradient are refused while it records."""

    def __init__(self, k_pages, v_pages, k_scales=None, v_scales=None, k_group_scales=None, v_group_scales=None):
        import torch

        for name, t in (("k_pages", k_pages), ("v_pages", v_pages), ("k_scales", k_scales), ("v_scales", v_scales),
                        ("k_group_scales", k_group_scales), ("v_group_scales", v_group_scales)):
            if name.endswith("scales") and t is None:
                continue
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.get_device() != torch.cuda.current_device():
                raise ValueError(f"{name} is on {t.device}, not on the current device")
            if t.requires_grad:
                raise ValueError(f"{name} requires a gradient, which the calls do not record")
        _fast()
        self.device = k_pages.get_device()
        if k_pages.dtype not in (torch.bfloat16, torch.float8_e4m3fn, torch.uint8) or v_pages.dtype is not k_pages.dtype:
            raise ValueError(f"pages have dtypes {k_pages.dtype}, {v_pages.dtype}; expected bfloat16, float8_e4m3fn or uint8 (4-bit codes) for both")
        if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
            raise ValueError(f"pages have shapes {tuple(k_pages.shape)}, {tuple(v_pages.shape)}; expected "
                             "[n_pages][n_kv_heads][page_size][head_dim] for both (4-bit pages: head_dim / 2)")
        if k_pages.stride(3) != 1 or v_pages.stride(3) != 1:
            raise ValueError("pages must be contiguous along head_dim")
        n, h, s, d = k_pages.shape
        bits = 16 if k_pages.dtype is torch.bfloat16 else 8 if k_pages.dtype is torch.float8_e4m3fn else 4
        per = 2 if bits == 4 else 1  # elements to one of the tensor's
        d *= per
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if (t is None) != (bits == 16):
                raise ValueError("8-bit and 4-bit pages come with k_scales and v_scales, bf16 pages without")
            if t is not None:
                if t.dtype is not torch.float32 or tuple(t.shape) != (n, h) or not t.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {(n, h)}")
        for name, t in (("k_group_scales", k_group_scales), ("v_group_scales", v_group_scales)):
            if (t is None) != (bits != 4):
                raise ValueError("4-bit pages come with k_group_scales and v_group_scales, others without")
            if t is not None:
                if t.dtype is not torch.float8_e4m3fn or tuple(t.shape) != (n, h, s, d // 16) or not t.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous float8_e4m3fn tensor of shape {(n, h, s, d // 16)}")
        self.k_pages, self.v_pages, self.k_scales, self.v_scales, self.k_group_scales, self.v_group_scales = self._tensors = (
            k_pages, v_pages, k_scales, v_scales, k_group_scales, v_group_scales)
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim, self.kv_bits = n, h, s, d, bits
        self._c = clo_paged_cache(k_pages.data_ptr(), v_pages.data_ptr(), None if k_scales is None else k_scales.data_ptr(),
                                  None if v_scales is None else v_scales.data_ptr(), n, *(per * x for x in k_pages.stride()[:3]),
                                  *(per * x for x in v_pages.stride()[:3]), h, d, s, bits,
                                  None if k_group_scales is None else k_group_scales.data_ptr(),
                                  None if v_group_scales is None else v_group_scales.data_ptr())
        self._ref = ctypes.byref(self._c)
        self._address = ctypes.addressof(self._c)

    @classmethod
    def create(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, kv_bits: int = 16, device=None, group=None):
        """A cache of new pages (their contents are undefined until they are appended to).

        group: the elements that share a scale, to be stated with kv_bits 4 (16 is what the calls read and write; a caller
        who means groups of another size, or codes without them, is refused)."""
        if kv_bits not in (16, 8, 4):
            raise ValueError("kv_bits must be 16, 8 or 4")
        if (group != 16) if kv_bits == 4 else (group is not None):
            raise ValueError("kv_bits 4 comes with group=16, the elements that share a scale; other kv_bits without a group")
        import torch

        device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        if kv_bits == 16:
            return cls(*(torch.empty(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
        scales = [torch.ones((n_pages, n_kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
        if kv_bits == 8:
            return cls(*(torch.empty(shape, dtype=torch.float8_e4m3fn, device=device) for _ in range(2)), *scales)
        return cls(*(torch.empty((*shape[:3], head_dim // 2), dtype=torch.uint8, device=device) for _ in range(2)), *scales,
                   *(torch.empty((*shape[:3], head_dim // 16), dtype=torch.float8_e4m3fn, device=device) for _ in range(2)))

    def append(self, k, v, q_starts, kv_lens, block_table, rope: clo_rope_plan | None = None, positions=None, q=None,
               q_out=None, max_q=None, stream=None):
        """clo_paged_append: k, v bf16 [total][n_kv_heads][head_dim] into the pages, k rotated by rope; with
        q, returns the rotated queries (q_out, or new rows)."""
        r = _torch_binding.append(self._address, self.device, k, v, q_starts, kv_lens, block_table,
                                  0 if rope is None else _plan_address(rope), positions, q, q_out, max_q, stream, self._tensors)
        if type(r) is int:
            _check(r, "clo_paged_append")
        return r

    def read(self, q_starts, kv_lens, block_table, total: int, k_out=None, v_out=None, max_q=None, stream=None):
        """clo_paged_read: the batch's last tokens as bf16 (k, v), each [total][n_kv_heads][head_dim]."""
        r = _torch_binding.read(self._address, self.device, q_starts, kv_lens, block_table, total, k_out, v_out, max_q, stream)
        if type(r) is int:
            _check(r, "clo_paged_read")
        return r

    def attention_workspace(self, n_q_heads: int, batch: int, total: int, max_pages: int, max_q=None, window: int = 0,
                            sinks: int = 0) -> int:
        """Bytes of workspace that attention of these sizes uses (0: none)."""
        b = clo_paged_batch(1 << 20, 1 << 20, 1 << 20, max_pages, max_pages, batch, total, total if max_q is None else max_q)
        size = ctypes.c_int64()
        _check(_lib.clo_paged_attention_workspace(self._ref, ctypes.byref(b), n_q_heads, window, sinks, ctypes.byref(size)),
               "clo_paged_attention_workspace")
        return size.value

    def attention(self, q, q_starts, kv_lens, block_table, out=None, max_q=None, softmax_scale: float = 0.0, window: int = 0,
                  sinks: int = 0, workspace=None, stream=None):
        """clo_paged_attention: q bf16 [total][n_q_heads][head_dim] over the pages; returns out (or new rows).

        workspace: uint8 tensor of attention_workspace() bytes, or None: allocated where the sizes ask for one."""
        r = _torch_binding.attention(self._address, self.device, q, q_starts, kv_lens, block_table, out, max_q, softmax_scale,
                                     window, sinks, workspace, stream)
        if type(r) is int:
            _check(r, "clo_paged_attention")
        return r


def clo_paged_attention_workspace(cache: PagedCache, *args, **kwargs) -> int:
    """PagedCache.attention_workspace under the C name."""
    return cache.attention_workspace(*args, **kwargs)


def clo_paged_append(cache: PagedCache, *args, **kwargs):
    """PagedCache.append under the C name."""
    return cache.append(*args, **kwargs)


def clo_paged_read(cache: PagedCache, *args, **kwargs):
    """PagedCache.read under the C name."""
    return cache.read(*args, **kwargs)


def clo_paged_attention(cache: PagedCache, *args, **kwargs):
    """PagedCache.attention under the C name."""
    return cache.attention(*args, **kwargs)


# ----------------------------------------------------------------------------- convenience
class CLOContext:
    """Owns one library context; keeps the shapes needed to size debug read-backs."""

    def __init__(self, *, n_layers, batch, n_q_heads, n_kv_heads, head_dim, max_tokens, hash_R, topk=0,
                 topk_ratio=0.1, tau=None, persist_mask=None, warmup_steps=16, tau_offset=0.05, n_persist=0,
                 wait_timeout_ns=2_000_000_000, timing=False, stream=None, adaptive_tau=False, tau_ema=0.0625,
                 kv_bits=16):
        self.L, self.B, self.Hq, self.Hkv, self.d = n_layers, batch, n_q_heads, n_kv_heads, head_dim
        self.G = n_q_heads // n_kv_heads
        self.topk, self.topk_ratio = int(topk), float(topk_ratio)
        self._R = np.ascontiguousarray(hash_R, dtype=np.uint16)
        self._tau = None if tau is None else np.ascontiguousarray(tau, dtype=np.float32)
        self._pm = None if persist_mask is None else np.ascontiguousarray(persist_mask, dtype=np.uint8)
        cfg = clo_config_default()
        cfg.n_layers, cfg.batch, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim = (
            n_layers, batch, n_q_heads, n_kv_heads, head_dim)
        cfg.max_tokens = int(max_tokens)
        cfg.topk = int(topk)
        cfg.topk_ratio = float(topk_ratio)
        cfg.hash_R = self._R.ctypes.data
        cfg.tau = None if self._tau is None else self._tau.ctypes.data
        cfg.persist_mask = None if self._pm is None else self._pm.ctypes.data
        cfg.warmup_steps = int(warmup_steps)
        cfg.tau_offset = float(tau_offset)
        cfg.n_persist = int(n_persist)
        cfg.wait_timeout_ns = int(wait_timeout_ns)
        cfg.timing = int(bool(timing))
        cfg.debug_drop_flag_layer = -1
        cfg.stream = stream
        cfg.adaptive_tau = int(bool(adaptive_tau))
        cfg.tau_ema = float(tau_ema)
        cfg.kv_bits = int(kv_bits)
        self.kv_bits = int(kv_bits)
        self.cfg = cfg
        self.ctx = clo_init(cfg)
        self.ntok = np.zeros((n_layers, batch), dtype=np.int64)

    def close(self):
        if self.ctx is not None:
            clo_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def step_bytes(self, first: int, last: int) -> np.ndarray:
        """Host-link and algorithmic HBM bytes of each step in [first, last) (timing mode):
        int64 [last - first][2], from the library's cumulative per-step history."""
        if last - first + 1 > STEP_HIST or first < 1:
            raise ValueError("the history keeps the last 4096 steps and needs the step before the first")
        h = clo_debug_get(self.ctx, CLO_DBG_STEP_BYTES, 0, 0, 0, np.empty((STEP_HIST, 2), dtype=np.uint64))
        cum = np.array([h[s % STEP_HIST] for s in range(first - 1, last)], dtype=np.int64)
        return np.diff(cum, axis=0)

    def pool_node(self) -> int:
        """NUMA node of the pinned pool's pages, or -1 when the pool was not placed."""
        return int(clo_debug_get(self.ctx, CLO_DBG_POOL_NODE, 0, 0, 0, np.empty(1, dtype=np.int32))[0])

    def k_of(self, b: int, layer: int = 0) -> int:
        """The library's top-k count of (layer, sequence b) at its current length."""
        k = clo_debug_get(self.ctx, CLO_DBG_TOPK, 0, 0, 0, np.empty((self.L, self.B), dtype=np.int32))
        return int(k[layer, b])

    def append_kv(self, layer, seq, k, v, src_is_device=None):
        n = k.shape[0]
        clo_append_kv(self.ctx, layer, seq, k, v, n, src_is_device)
        self.ntok[layer, seq] += n

    def append_step(self, k, v, src_is_device=None):
        """One new token for every (layer, sequence): k, v bf16 [L][B][Hkv][d]."""
        clo_append_step(self.ctx, k, v, src_is_device)
        self.ntok += 1

    def decode_step(self, q, out, io_on_device=None):
        clo_decode_step(self.ctx, q, out, io_on_device)

    def decode_layer(self, layer, q, out, io_on_device=None):
        """One layer of a step: q bf16 [B][Hq][d], out fp32 [B][Hq][d]; layers in order."""
        clo_decode_layer(self.ctx, layer, q, out, io_on_device)

    def sync(self):
        clo_sync(self.ctx)

    def stats(self):
        return clo_stats(self.ctx)

    def set(self, key, value):
        clo_set(self.ctx, key, value)

    # debug read-backs ----------------------------------------------------------
    def key_codes(self, l, b, h):
        return clo_debug_get(self.ctx, CLO_DBG_KEY_CODES, l, b, h,
                             np.empty((int(self.ntok[l, b]), 2), dtype=np.uint64))

    def query_codes(self, l, b, h):
        return clo_debug_get(self.ctx, CLO_DBG_QUERY_CODES, l, b, h, np.empty((self.G, 2), dtype=np.uint64))

    def idx(self, l, b, h):
        return clo_debug_get(self.ctx, CLO_DBG_IDX, l, b, h, np.empty(self.k_of(b, l), dtype=np.int32))

    def slot_rows(self, l, b, h):
        return clo_debug_get(self.ctx, CLO_DBG_SLOT_ROWS, l, b, h,
                             np.empty((self.k_of(b, l), 2, self.d), dtype=np.uint16))

    def decisions(self):
        return clo_debug_get(self.ctx, CLO_DBG_DECISION, 0, 0, 0,
                             np.empty((self.L, self.B, self.Hkv), dtype=np.uint8))

    def cosines(self):
        return clo_debug_get(self.ctx, CLO_DBG_COS, 0, 0, 0, np.empty((self.L, self.B, self.Hkv), dtype=np.float32))

    def tau(self):
        return clo_debug_get(self.ctx, CLO_DBG_TAU, 0, 0, 0, np.empty((self.L, self.Hkv), dtype=np.float32))

    def persist(self):
        return clo_debug_get(self.ctx, CLO_DBG_PERSIST, 0, 0, 0, np.empty((self.L, self.Hkv), dtype=np.uint8))

    def shat(self):
        return clo_debug_get(self.ctx, CLO_DBG_SHAT, 0, 0, 0, np.empty((self.L, self.Hkv), dtype=np.float64))

    def timeline(self):
        """Stamps of the last step's fused kernel (timing mode), in us from its start."""
        t = clo_debug_get(self.ctx, CLO_DBG_TIMELINE, 0, 0, 0, np.empty(16, dtype=np.uint64)).astype(np.int64)
        if t[0] == 0:
            return None
        rel = lambda v: None if v == 0 else round((int(v) - int(t[0])) / 1e3, 1)  # noqa: E731
        return {"sel_missed_done_us": rel(t[1]), "sel_persistent_done_us": rel(t[2]),
                "first_fetch_us": rel(t[3]), "fetch_done_us": rel(t[4]), "first_attention_us": rel(t[5]),
                "attention_done_us": rel(t[6]), "fetch_wait_sum_us": round(int(t[7]) / 1e3, 1),
                "attention_wait_sum_us": round(int(t[8]) / 1e3, 1),
                "selection_chunk_mean_us": round(int(t[9]) / 1e3 / max(1, int(t[10])), 2),
                "selection_chunks": int(t[10]),
                "attention_split_mean_us": round(int(t[11]) / 1e3 / max(1, int(t[12])), 2),
                "attention_splits": int(t[12]), "decide_start_us": rel(t[13]), "decide_end_us": rel(t[14]),
                "attention_split_run_mean_us": round(int(t[15]) / 1e3 / max(1, int(t[12])), 2)}
