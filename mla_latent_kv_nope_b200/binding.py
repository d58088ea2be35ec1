"""Thin Python binding of the C ABI in ``include/mla.h`` (ctypes).

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of ``libmla_b200.so``.  Tensors are torch CUDA tensors (device memory
and streams only); each call enqueues on the current torch stream.  A missing
library raises immediately -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import importlib.util
import os
from dataclasses import dataclass

import torch

from .build import calls_name

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla_b200.so")

MLA_BF16, MLA_F32 = 0, 1
STATUS = {
    0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED",
    3: "MLA_ERR_ALIGNMENT", 4: "MLA_ERR_WORKSPACE", 5: "MLA_ERR_CUDA",
    6: "MLA_ERR_DEVICE_TIMEOUT", 7: "MLA_ERR_BOUNDS",
}
EXPORTED = (
    "mla_cache_row_elems", "mla_cache_append_workspace_bytes", "mla_cache_append",
    "mla_absorb_q", "mla_decode_default_splits", "mla_decode_workspace_bytes",
    "mla_decode", "mla_combine", "mla_out_proj", "mla_get_device_status",
    "mla_status_string", "mla_decode_noalloc", "mla_decode_paged", "mla_cache_append_paged",
    "mla_merge_partials", "mla_debug_inject_wait", "mla_cache_fp8_row_bytes",
    "mla_cache_append_fp8", "mla_decode_fp8", "mla_fold_output_weights",
    "mla_out_proj_folded_workspace_bytes", "mla_out_proj_folded", "mla_prefill_workspace_bytes",
    "mla_prefill", "mla_rope_init", "mla_rope", "mla_plan_pages_workspace_bytes",
    "mla_plan_pages", "mla_plan_pages_capped", "mla_release_pages", "mla_cache_write_paged", "mla_cache_write_paged_step",
    "mla_cache_write_fp8_paged", "mla_decode_fp8_paged",
)

PAGE_ROWS = 64   # rows per page of a paged latent cache (one decode work tile)


class MLAError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({msg})")
        self.status = status


class CDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("d_c", ctypes.c_int32),
                ("d_r", ctypes.c_int32), ("d_nope", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("cache_capacity", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class CRopeParams(ctypes.Structure):
    _fields_ = [("d_r", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("base", ctypes.c_float), ("factor", ctypes.c_float),
                ("original_len", ctypes.c_float), ("beta_fast", ctypes.c_float),
                ("beta_slow", ctypes.c_float), ("attention_factor", ctypes.c_float)]


class RopeTable(ctypes.Structure):
    """mla_rope_table: host-side angles of a rotation (see rope_table)."""
    _fields_ = [("d_r", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("amplitude", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("turn", ctypes.c_uint64 * 128)]

    @property
    def address(self) -> int:
        return ctypes.addressof(self)


@dataclass(frozen=True)
class Dims:
    """Problem shape (names as in the header: H heads, d_c latent width,
    d_r decoupled-RoPE width, d_nope / d_v per-head content / value widths)."""
    B: int
    H: int
    d_c: int
    d_r: int
    d_nope: int
    d_v: int
    cache_capacity: int
    dtype: str = "bf16"  # "bf16" | "f32"

    def c(self) -> CDims:
        return CDims(self.B, self.H, self.d_c, self.d_r, self.d_nope, self.d_v,
                     self.cache_capacity, MLA_BF16 if self.dtype == "bf16" else MLA_F32)

    @functools.cached_property
    def _struct(self):
        return self.c()      # made once: the fields are frozen

    @functools.cached_property
    def ref(self):
        """A reference to the C struct."""
        return ctypes.byref(self._struct)

    @functools.cached_property
    def address(self) -> int:
        return ctypes.addressof(self._struct)

    def __getstate__(self):
        return {f.name: getattr(self, f.name) for f in dataclasses.fields(self)}

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == "bf16" else torch.float32

    @property
    def R(self) -> int:
        return self.d_c + self.d_r


_lib = None
_calls = None     # the checks and calls of the short operators in C++ (csrc/py_calls.cpp)


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the sm_100a library.  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with mla_latent_kv_nope_b200.build.build(); "
            "there is no non-CUDA implementation")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ, F = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                          ctypes.c_float)
    D = ctypes.POINTER(CDims)
    sig = {
        "mla_cache_row_elems": (I64, [I32, I32]),
        "mla_cache_append_workspace_bytes": (SZ, [D, I32]),
        "mla_cache_append": (ctypes.c_int, [D, I32, P, P, P, F, F, P, P, P, SZ, P]),
        "mla_absorb_q": (ctypes.c_int, [D, P, P, P, P, F, P, P]),
        "mla_decode_default_splits": (ctypes.c_int, [D]),
        "mla_decode_workspace_bytes": (SZ, [D, ctypes.c_int]),
        "mla_decode": (ctypes.c_int, [D, P, P, P, F, ctypes.c_int, P, SZ,
                                      ctypes.POINTER(ctypes.c_int), P]),
        "mla_combine": (ctypes.c_int, [D, P, P, SZ, ctypes.c_int, P, P, P]),
        "mla_out_proj": (ctypes.c_int, [D, P, P, P, P]),
        "mla_get_device_status": (ctypes.c_int, [P]),
        "mla_decode_noalloc": (ctypes.c_int, [D, P, P, P, F, P, P, P]),
        "mla_decode_paged": (ctypes.c_int, [D, P, P, I64, P, I32, P, F, ctypes.c_int, P, SZ,
                                            ctypes.POINTER(ctypes.c_int), P]),
        "mla_cache_append_paged": (ctypes.c_int, [D, I32, P, P, P, F, F, P, I64, P, I32, P, P,
                                                  SZ, P]),
        "mla_merge_partials": (ctypes.c_int, [D, ctypes.c_int, P, P, P, P, P]),
        "mla_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "mla_debug_inject_wait": (ctypes.c_int, [ctypes.c_uint64]),
        "mla_cache_fp8_row_bytes": (I64, [I32, I32]),
        "mla_fold_output_weights": (ctypes.c_int, [D, I32, P, P, P, P]),
        "mla_prefill_workspace_bytes": (SZ, [D, I32, I64]),
        "mla_prefill": (ctypes.c_int, [D, I32, I64, P, P, P, P, P, P, F, F, P, P, P, SZ, P]),
        "mla_out_proj_folded_workspace_bytes": (SZ, [D, I32]),
        "mla_out_proj_folded": (ctypes.c_int, [D, I32, P, P, P, P, SZ, P]),
        "mla_cache_append_fp8": (ctypes.c_int, [D, I32, P, P, P, F, F, P, P, P, P, SZ, P]),
        "mla_decode_fp8": (ctypes.c_int, [D, P, P, P, P, F, ctypes.c_int, P, SZ,
                                          ctypes.POINTER(ctypes.c_int), P]),
        "mla_rope_init": (ctypes.c_int, [ctypes.POINTER(CRopeParams), ctypes.POINTER(RopeTable)]),
        "mla_rope": (ctypes.c_int, [I32, P, I64, I32, P, I64, I64, P, P, I64, I64, I32, P]),
        "mla_plan_pages_workspace_bytes": (SZ, []),
        "mla_plan_pages": (ctypes.c_int, [I32, P, P, P, I32, P, I32, P, I64, I32, P, P, P, P, P,
                                          P, P, SZ, P]),
        "mla_plan_pages_capped": (ctypes.c_int, [I32, P, P, P, I32, I64, P, I32, P, I64, I32, P, P,
                                                 P, P, P, P, P, SZ, P]),
        "mla_release_pages": (ctypes.c_int, [I32, P, P, P, I32, P, I32, P, I64, P]),
        "mla_cache_write_paged": (ctypes.c_int, [D, I32, P, I64, P, F, P, P, P, P, I64, P]),
        "mla_cache_write_paged_step": (ctypes.c_int, [D, I32, P, I64, P, F, P, P, P, P, P, I64, P]),
        "mla_cache_write_fp8_paged": (ctypes.c_int, [D, I32, P, I64, P, F, P, P, P, P, I32, P, P,
                                                     I64, P]),
        "mla_decode_fp8_paged": (ctypes.c_int, [D, P, P, P, I64, P, I32, P, F, ctypes.c_int, P,
                                                SZ, ctypes.POINTER(ctypes.c_int), P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _load_calls(lib)
    _lib = lib           # once both are there
    return lib


def _load_calls(lib) -> None:
    global _calls
    at = os.path.join(_HERE, calls_name())
    if not os.path.exists(at):
        raise RuntimeError(f"{at} is missing: build it with mla_latent_kv_nope_b200.build.build()")
    spec = importlib.util.spec_from_file_location("_calls", at)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.init(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in (
        "mla_rope", "mla_plan_pages_capped", "mla_cache_write_paged_step", "mla_cache_write_fp8_paged",
        "mla_decode_fp8_paged")))
    _calls = mod


def _check(fn: str, status: int):
    if status != 0:
        msg = load_library().mla_status_string(status).decode()
        raise MLAError(fn, status, msg)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream=None):
    """Raw handle of the given stream, or of the current one of the current device."""
    if stream is None:
        torch.cuda.init()       # a host without a GPU raises here
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _need(t, dtype, shape, name):
    if t.dtype != dtype or t.shape != shape or not t.is_cuda:
        raise ValueError(f"{name}: expected CUDA {dtype} {tuple(shape)}, got "
                         f"{t.device} {t.dtype} {tuple(t.shape)}")


def _need_ws(t, name="workspace"):
    """A scratch buffer: any dtype, but device memory and contiguous (the
    library writes it from kernels, so a host tensor must never reach it)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        got = t.device if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: expected a contiguous CUDA tensor, got {got}")


# ---------------------------------------------------------------------------
def cache_row_elems(d_c: int, d_r: int) -> int:
    """Elements of one latent cache row, d_c + d_r (mla_cache_row_elems)."""
    return int(load_library().mla_cache_row_elems(d_c, d_r))


def cache_append_workspace_bytes(dims: Dims, hidden: int) -> int:
    """Bytes of fp32 workspace mla_cache_append needs for this hidden size."""
    return int(load_library().mla_cache_append_workspace_bytes(dims.ref, hidden))


def cache_append(dims: Dims, h, W_DKV, gamma, cache, seqlens, workspace, eps=1e-6,
                 rope_base=10000.0, stream=None):
    """mla_cache_append: write row L_b = [RMSNorm(W^DKV h) * gamma || RoPE(W^KR h, L_b)]
    of every sequence and increment L_b (cache [B, capacity, R])."""
    dt = dims.torch_dtype
    hidden = h.shape[-1]
    _need(h, dt, (dims.B, hidden), "h")
    _need(W_DKV, dt, (dims.R, hidden), "W_DKV")
    _need(cache, dt, (dims.B, dims.cache_capacity, dims.R), "cache")
    _need(seqlens, torch.int32, (dims.B,), "seqlens")
    if gamma is not None:
        _need(gamma, torch.float32, (dims.d_c,), "gamma")
    _need_ws(workspace)
    st = load_library().mla_cache_append(
        dims.ref, hidden, _ptr(h), _ptr(W_DKV), _ptr(gamma), eps, rope_base,
        _ptr(cache), _ptr(seqlens), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check("mla_cache_append", st)


def _need_pages(dims: Dims, pool, block_table):
    if pool.dim() != 3 or pool.shape[1:] != (PAGE_ROWS, dims.R):
        raise ValueError(f"cache_pool must be [num_pages, {PAGE_ROWS}, {dims.R}]")
    _need(pool, dims.torch_dtype, tuple(pool.shape), "cache_pool")
    if block_table.dim() != 2 or block_table.shape[0] != dims.B:
        raise ValueError("block_table must be [B, max_blocks]")
    _need(block_table, torch.int32, tuple(block_table.shape), "block_table")


def cache_append_paged(dims: Dims, h, W_DKV, gamma, cache_pool, block_table, seqlens,
                       workspace, eps=1e-6, rope_base=10000.0, stream=None):
    """mla_cache_append on a paged cache: cache_pool [num_pages, 64, R], block_table
    [B, max_blocks] int32 page ids."""
    dt = dims.torch_dtype
    hidden = h.shape[-1]
    _need(h, dt, (dims.B, hidden), "h")
    _need(W_DKV, dt, (dims.R, hidden), "W_DKV")
    _need_pages(dims, cache_pool, block_table)
    _need(seqlens, torch.int32, (dims.B,), "seqlens")
    if gamma is not None:
        _need(gamma, torch.float32, (dims.d_c,), "gamma")
    _need_ws(workspace)
    st = load_library().mla_cache_append_paged(
        dims.ref, hidden, _ptr(h), _ptr(W_DKV), _ptr(gamma), eps, rope_base,
        _ptr(cache_pool), cache_pool.shape[0], _ptr(block_table), block_table.shape[1],
        _ptr(seqlens), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check("mla_cache_append_paged", st)


def decode_paged(dims: Dims, q_cat, cache_pool, block_table, seqlens, softmax_scale, workspace,
                 num_splits=0, stream=None) -> int:
    """mla_decode on a paged cache (see cache_append_paged)."""
    _need(q_cat, dims.torch_dtype, (dims.B, dims.H, dims.R), "q_cat")
    _need_pages(dims, cache_pool, block_table)
    _need(seqlens, torch.int32, (dims.B,), "seqlens")
    _need_ws(workspace)
    used = ctypes.c_int(0)
    st = load_library().mla_decode_paged(
        dims.ref, _ptr(q_cat), _ptr(cache_pool), cache_pool.shape[0],
        _ptr(block_table), block_table.shape[1], _ptr(seqlens), float(softmax_scale), num_splits,
        _ptr(workspace), workspace.numel() * workspace.element_size(), ctypes.byref(used),
        _stream(stream))
    _check("mla_decode_paged", st)
    return used.value


def cache_fp8_row_bytes(d_c: int, d_r: int) -> int:
    """Bytes of one FP8 latent cache row: d_c E4M3 codes + d_r bf16 RoPE keys."""
    return int(load_library().mla_cache_fp8_row_bytes(d_c, d_r))


def _need_fp8_cache(dims: Dims, cache, scales):
    rb = dims.d_c + 2 * dims.d_r
    _need(cache, torch.uint8, (dims.B, dims.cache_capacity, rb), "cache_fp8")
    _need(scales, torch.float32, (dims.B, dims.cache_capacity), "scales")


def cache_append_fp8(dims: Dims, h, W_DKV, gamma, cache, scales, seqlens, workspace, eps=1e-6,
                     rope_base=10000.0, stream=None):
    """mla_cache_append_fp8: as cache_append, into an FP8 latent cache
    (cache [B, capacity, d_c + 2 d_r] uint8, scales [B, capacity] fp32)."""
    dt = dims.torch_dtype
    hidden = h.shape[-1]
    _need(h, dt, (dims.B, hidden), "h")
    _need(W_DKV, dt, (dims.R, hidden), "W_DKV")
    _need_fp8_cache(dims, cache, scales)
    _need(seqlens, torch.int32, (dims.B,), "seqlens")
    if gamma is not None:
        _need(gamma, torch.float32, (dims.d_c,), "gamma")
    _need_ws(workspace)
    st = load_library().mla_cache_append_fp8(
        dims.ref, hidden, _ptr(h), _ptr(W_DKV), _ptr(gamma), eps, rope_base,
        _ptr(cache), _ptr(scales), _ptr(seqlens), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check("mla_cache_append_fp8", st)


def decode_fp8(dims: Dims, q_cat, cache, scales, seqlens, softmax_scale, workspace,
               num_splits=0, stream=None) -> int:
    """mla_decode_fp8: mla_decode over an FP8 latent cache; returns the splits used."""
    _need(q_cat, dims.torch_dtype, (dims.B, dims.H, dims.R), "q_cat")
    _need_fp8_cache(dims, cache, scales)
    _need(seqlens, torch.int32, (dims.B,), "seqlens")
    _need_ws(workspace)
    used = ctypes.c_int(0)
    st = load_library().mla_decode_fp8(dims.ref, _ptr(q_cat), _ptr(cache),
                                       _ptr(scales), _ptr(seqlens), float(softmax_scale),
                                       num_splits, _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       ctypes.byref(used), _stream(stream))
    _check("mla_decode_fp8", st)
    return used.value


def absorb_q(dims: Dims, q_nope, q_pe, W_UK, q_pos, q_cat, rope_base=10000.0, stream=None):
    """mla_absorb_q: q_cat[b,i] = [W^UK_i^T q_nope[b,i] ; RoPE(q_pe[b,i], q_pos[b])]
    (no rotation when q_pos is None)."""
    dt = dims.torch_dtype
    _need(q_nope, dt, (dims.B, dims.H, dims.d_nope), "q_nope")
    _need(q_pe, dt, (dims.B, dims.H, dims.d_r), "q_pe")
    _need(W_UK, dt, (dims.H, dims.d_nope, dims.d_c), "W_UK")
    _need(q_cat, dt, (dims.B, dims.H, dims.R), "q_cat")
    if q_pos is not None:
        _need(q_pos, torch.int32, (dims.B,), "q_pos")
    st = load_library().mla_absorb_q(dims.ref, _ptr(q_nope), _ptr(q_pe),
                                     _ptr(W_UK), _ptr(q_pos), rope_base, _ptr(q_cat),
                                     _stream(stream))
    _check("mla_absorb_q", st)


def decode_default_splits(dims: Dims) -> int:
    """The split count mla_decode uses on the current device when asked for 0."""
    return int(load_library().mla_decode_default_splits(dims.ref))


def decode_workspace_bytes(dims: Dims, num_splits: int = 0) -> int:
    """Bytes of workspace mla_decode needs for this many splits (0 = default)."""
    return int(load_library().mla_decode_workspace_bytes(dims.ref, num_splits))


def decode(dims: Dims, q_cat, cache, seqlens, softmax_scale, workspace, num_splits=0,
           stream=None) -> int:
    """mla_decode: split-KV latent attention of q_cat over the cache; writes the
    partials into ``workspace`` and returns the number of splits used."""
    dt = dims.torch_dtype
    _need(q_cat, dt, (dims.B, dims.H, dims.R), "q_cat")
    _need(cache, dt, (dims.B, dims.cache_capacity, dims.R), "cache")
    _need(seqlens, torch.int32, (dims.B,), "seqlens")
    _need_ws(workspace)
    used = ctypes.c_int(0)
    st = load_library().mla_decode(dims.ref, _ptr(q_cat), _ptr(cache),
                                   _ptr(seqlens), float(softmax_scale), num_splits,
                                   _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   ctypes.byref(used), _stream(stream))
    _check("mla_decode", st)
    return used.value


def combine(dims: Dims, seqlens, workspace, splits_used, o_lat, lse=None, stream=None):
    """mla_combine: log-sum-exp merge of the partials into o_lat [B,H,d_c] fp32 (and
    lse [B,H] fp32 when given)."""
    _need(seqlens, torch.int32, (dims.B,), "seqlens")
    _need_ws(workspace)
    _need(o_lat, torch.float32, (dims.B, dims.H, dims.d_c), "o_lat")
    if lse is not None:
        _need(lse, torch.float32, (dims.B, dims.H), "lse")
    st = load_library().mla_combine(dims.ref, _ptr(seqlens), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), splits_used,
                                    _ptr(o_lat), _ptr(lse), _stream(stream))
    _check("mla_combine", st)


def merge_partials(dims: Dims, o_parts, lse_parts, o_lat, lse=None, stream=None):
    """mla_merge_partials: log-sum-exp merge of n per-token-range results,
    o_parts [n,B,H,d_c] fp32 and lse_parts [n,B,H] fp32 (stacked combine
    outputs), into o_lat [B,H,d_c] (and lse [B,H] when given)."""
    n = o_parts.shape[0]
    _need(o_parts, torch.float32, (n, dims.B, dims.H, dims.d_c), "o_parts")
    _need(lse_parts, torch.float32, (n, dims.B, dims.H), "lse_parts")
    _need(o_lat, torch.float32, (dims.B, dims.H, dims.d_c), "o_lat")
    if lse is not None:
        _need(lse, torch.float32, (dims.B, dims.H), "lse")
    st = load_library().mla_merge_partials(dims.ref, n, _ptr(o_parts),
                                           _ptr(lse_parts), _ptr(o_lat), _ptr(lse),
                                           _stream(stream))
    _check("mla_merge_partials", st)


def out_proj(dims: Dims, o_lat, W_UV, out, stream=None):
    """mla_out_proj: out[b,i] = W^UV_i o_lat[b,i]."""
    dt = dims.torch_dtype
    _need(o_lat, torch.float32, (dims.B, dims.H, dims.d_c), "o_lat")
    _need(W_UV, dt, (dims.H, dims.d_v, dims.d_c), "W_UV")
    _need(out, dt, (dims.B, dims.H, dims.d_v), "out")
    st = load_library().mla_out_proj(dims.ref, _ptr(o_lat), _ptr(W_UV), _ptr(out),
                                     _stream(stream))
    _check("mla_out_proj", st)


def debug_inject_wait(cycles: int) -> None:
    """mla_debug_inject_wait: test hook that makes later bf16 decode launches
    wait ``cycles`` SM cycles on a barrier nothing arrives on and give up
    (MLA_ERR_DEVICE_TIMEOUT in the status word); 0 turns it off."""
    _check("mla_debug_inject_wait", load_library().mla_debug_inject_wait(int(cycles)))


def prefill_workspace_bytes(dims: Dims, T: int, L: int) -> int:
    return int(load_library().mla_prefill_workspace_bytes(dims.ref, T, L))


def prefill(dims: Dims, q_nope, q_pe, q_pos, W_UK, W_UV, rows, out, workspace, lse=None,
            softmax_scale: float = 0.0, rope_base: float = 10000.0, stream=None):
    """mla_prefill: materialised causal attention of one sequence's T query
    tokens over its L latent rows [L, d_c + d_r]; out [T, H, d_v] (+ lse [T, H])."""
    T, L = q_nope.shape[0], rows.shape[0]
    dt = dims.torch_dtype
    _need(q_nope, dt, (T, dims.H, dims.d_nope), "q_nope")
    if dims.d_r:
        _need(q_pe, dt, (T, dims.H, dims.d_r), "q_pe")
    _need(q_pos, torch.int32, (T,), "q_pos")
    _need(W_UK, dt, (dims.H, dims.d_nope, dims.d_c), "W_UK")
    _need(W_UV, dt, (dims.H, dims.d_v, dims.d_c), "W_UV")
    _need(rows, dt, (L, dims.R), "rows")
    _need(out, dt, (T, dims.H, dims.d_v), "out")
    if lse is not None:
        _need(lse, torch.float32, (T, dims.H), "lse")
    _need_ws(workspace)
    st = load_library().mla_prefill(
        dims.ref, T, L, _ptr(q_nope), _ptr(q_pe) if dims.d_r else None,
        _ptr(q_pos), _ptr(W_UK), _ptr(W_UV), _ptr(rows), softmax_scale, rope_base, _ptr(out),
        _ptr(lse) if lse is not None else None, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check("mla_prefill", st)


def fold_output_weights(dims: Dims, W_O, W_UV, W_fold, stream=None):
    """mla_fold_output_weights: W_fold [d_model, H*d_c] with
    W_fold[m, i*d_c + c] = (W^O_i W^UV_i)[m, c]; W_O [d_model, H*d_v]."""
    d_model = W_O.shape[0]
    _need(W_O, dims.torch_dtype, (d_model, dims.H * dims.d_v), "W_O")
    _need(W_UV, dims.torch_dtype, (dims.H, dims.d_v, dims.d_c), "W_UV")
    _need(W_fold, dims.torch_dtype, (d_model, dims.H * dims.d_c), "W_fold")
    st = load_library().mla_fold_output_weights(dims.ref, d_model, _ptr(W_O),
                                                _ptr(W_UV), _ptr(W_fold), _stream(stream))
    _check("mla_fold_output_weights", st)


def out_proj_folded_workspace_bytes(dims: Dims, d_model: int) -> int:
    return int(load_library().mla_out_proj_folded_workspace_bytes(dims.ref,
                                                                  d_model))


def out_proj_folded(dims: Dims, o_lat, W_fold, u, workspace, stream=None):
    """mla_out_proj_folded: u [B, d_model] = sum_i B_i o_lat[:, i] (bf16)."""
    d_model = W_fold.shape[0]
    _need(o_lat, torch.float32, (dims.B, dims.H, dims.d_c), "o_lat")
    _need(W_fold, dims.torch_dtype, (d_model, dims.H * dims.d_c), "W_fold")
    _need(u, dims.torch_dtype, (dims.B, d_model), "u")
    _need_ws(workspace)
    st = load_library().mla_out_proj_folded(
        dims.ref, d_model, _ptr(o_lat), _ptr(W_fold), _ptr(u), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check("mla_out_proj_folded", st)


# ---------------------------------------------------------------------------
# Paged serving: rotary positions, page plans, writes of many tokens, 8-bit pages.
# Their kernels take a few microseconds, so the host's part is short too: a call on
# the current device and stream goes to _calls, which checks the tensors in C++ and
# makes it, or answers None where something is amiss (or on another device or stream);
# then the checks here say what, or make the call through ctypes.
_ROPE_LAYOUT = {"half": 0, "interleaved": 1}
_ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_I32, _I64, _F32, _BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16


def _arg(t, dtype, shape, name, dev):
    """Device address of a contiguous CUDA tensor of this dtype and shape on device `dev`."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _need(t, dtype, shape, name)
        raise ValueError(f"tensors on different devices: {name} is on {t.device}, not cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous")
    return t.data_ptr()


def _device(t, name):
    """Device index of a CUDA tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        got = t.device if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: expected a CUDA tensor, got {got}")
    return t.get_device()


def _ws_arg(t, dev):
    """Address and bytes of a scratch buffer on device `dev`."""
    _need_ws(t)
    if t.get_device() != dev:
        raise ValueError(f"tensors on different devices: workspace is on {t.device}, not cuda:{dev}")
    return t.data_ptr(), t.nbytes


def _launch(fn, dev, stream, *args, name=None):
    """Call the library's `fn`(*args, stream) with `dev` current, on its current
    stream unless one is given, and raise on a bad status (as `name`, if given)."""
    f = getattr(_lib or load_library(), fn)
    if torch._C._cuda_getDevice() == dev:
        st = f(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None
               else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None
                   else stream.cuda_stream)
    if st:
        _check(name or fn, st)


def _table_ptr(table):
    if table is None:
        return None
    if not isinstance(table, RopeTable):
        raise TypeError("table must come from rope_table()")
    return table.address


def _rows(x, dtype, width, dev):
    """Address, rows and row stride of [T, width] rows with unit inner stride (rows of a
    wider matrix are fine)."""
    if (x.dtype is not dtype or x.dim() != 2 or x.shape[1] != width
            or (width > 1 and x.stride(1) != 1)):
        raise ValueError(f"x: expected CUDA {dtype} rows [T, {width}] with unit inner stride, "
                         f"got {x.device} {x.dtype} {tuple(x.shape)} strides {x.stride()}")
    T = x.shape[0]
    return x.data_ptr(), T, x.stride(0) if T > 1 else width


def rope_table(d_r: int, base: float = 10000.0, layout: str = "half", scaling: str = "none",
               factor: float = 1.0, original_len: float = 4096.0, beta_fast: float = 32.0,
               beta_slow: float = 1.0, attention_factor: float = 0.0) -> RopeTable:
    """mla_rope_init: the angles of a rotation of d_r values.  layout "half" pairs
    (x[k], x[k + d_r/2]), "interleaved" (x[2k], x[2k+1]); scaling "none",
    "linear", "ntk" or "yarn" stretches it by ``factor`` for long contexts."""
    if layout not in _ROPE_LAYOUT:
        raise ValueError(f"layout must be one of {sorted(_ROPE_LAYOUT)}, got {layout!r}")
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALING)}, got {scaling!r}")
    p = CRopeParams(d_r, _ROPE_LAYOUT[layout], _ROPE_SCALING[scaling], base, factor, original_len,
                    beta_fast, beta_slow, attention_factor)
    t = RopeTable()
    _check("mla_rope_init", load_library().mla_rope_init(ctypes.byref(p), ctypes.byref(t)))
    return t


def rope(table: RopeTable, x, pos, out=None, transpose=False, stream=None):
    """mla_rope: rotate the rows of x [T, H, d_r] (or [T, d_r]; any token and head
    strides, e.g. the last d_r of each head of a [T, H, d_nope + d_r] query) by
    pos [T] int32 into ``out`` (x itself rotates in place; a new contiguous
    tensor if None).  ``transpose`` applies the transposed rotation (the
    gradient of the rotation's output taken back to its input)."""
    if not isinstance(table, RopeTable):
        raise TypeError("table must come from rope_table()")
    if _calls is not None and out is not None and stream is None:
        st = _calls.rope(table, x, pos, out, transpose)
        if st is not None:
            return out if st == 0 else _check("mla_rope", st)
    dev = _device(x, "x")
    shape, st, dt = x.shape, x.stride(), x.dtype
    n = len(shape)
    if (n != 3 and n != 2) or shape[-1] != table.d_r or st[-1] != 1 or (dt is not _BF16
                                                                        and dt is not _F32):
        raise ValueError(f"x: expected CUDA bf16 or fp32 [T, (H,) {table.d_r}] with unit inner "
                         f"stride, got {x.device} {dt} {tuple(shape)} strides {st}")
    if out is None:
        out = torch.empty(shape, dtype=dt, device=x.device)
    elif (out.shape != shape or out.dtype is not dt or out.get_device() != dev
          or out.stride(-1) != 1):
        raise ValueError("out must match x's shape, dtype and device, with unit inner stride")
    so = out.stride()
    T = shape[0]
    p = _arg(pos, _I32, (T,), "pos", dev)
    H, xh, oh = (shape[1], st[1], so[1]) if n == 3 else (1, 0, 0)
    if H:
        _launch("mla_rope", dev, stream, MLA_BF16 if dt is _BF16 else MLA_F32, table.address, T, H,
                x.data_ptr(), st[0], xh, p, out.data_ptr(), so[0], oh, 1 if transpose else 0)
    return out


def plan_pages_workspace_bytes() -> int:
    """Bytes of zeroed workspace plan_pages needs."""
    return int(load_library().mla_plan_pages_workspace_bytes())


def plan_pages(seqlens, new_lens, block_table, free_pages, free_count, num_pages, query_start,
               positions, slots, seqlens_out, free_count_out, workspace, token_request=None,
               stream=None, capacity=None):
    """mla_plan_pages: take the pages this step's new tokens need off the free
    list into block_table [B, max_blocks], and fill query_start [B+1],
    positions [T] (int32) and slots [T] (int64); seqlens_out and
    free_count_out may be seqlens and free_count.  ``capacity`` is the longest sequence
    (None: 64 * max_blocks)."""
    if _calls is not None and stream is None:
        st = _calls.plan_pages(seqlens, new_lens, block_table, free_pages, free_count, num_pages,
                               query_start, positions, slots, seqlens_out, free_count_out,
                               workspace, token_request, capacity)
        if st is not None:
            return _check("mla_plan_pages", st) if st else None
    dev = _device(seqlens, "seqlens")
    B, T, F = seqlens.shape[0], positions.shape[0], free_pages.numel()
    mb = block_table.shape[-1]
    b, one, t = (B,), (1,), (T,)
    ws, nws = _ws_arg(workspace, dev)
    _launch("mla_plan_pages_capped", dev, stream, B, _arg(seqlens, _I32, b, "seqlens", dev),
            _arg(new_lens, _I32, b, "new_lens", dev),
            _arg(block_table, _I32, (B, mb), "block_table", dev), mb,
            mb * PAGE_ROWS if capacity is None else capacity,
            _arg(free_pages, _I32, (F,), "free_pages", dev), F,
            _arg(free_count, _I32, one, "free_count", dev), num_pages, T,
            _arg(query_start, _I32, (B + 1,), "query_start", dev),
            _arg(positions, _I32, t, "positions", dev), _arg(slots, _I64, t, "slots", dev),
            None if token_request is None else _arg(token_request, _I32, t, "token_request", dev),
            _arg(seqlens_out, _I32, b, "seqlens_out", dev),
            _arg(free_count_out, _I32, one, "free_count_out", dev), ws, nws, name="mla_plan_pages")


def release_pages(seqlens, release, block_table, free_pages, free_count, num_pages, stream=None):
    """mla_release_pages: return the pages of every request with release[b] != 0 to
    the free list (seqlens, block_table, free_pages and free_count in place)."""
    dev = _device(seqlens, "seqlens")
    B, F, mb = seqlens.shape[0], free_pages.numel(), block_table.shape[-1]
    _launch("mla_release_pages", dev, stream, B, _arg(seqlens, _I32, (B,), "seqlens", dev),
            _arg(release, _I32, (B,), "release", dev),
            _arg(block_table, _I32, (B, mb), "block_table", dev), mb,
            _arg(free_pages, _I32, (F,), "free_pages", dev), F,
            _arg(free_count, _I32, (1,), "free_count", dev), num_pages)


def cache_write_paged(dims: Dims, x, gamma, positions, slots, cache_pool, table=None, eps=1e-6,
                      stream=None, planned=None):
    """mla_cache_write_paged: the rows [RMSNorm(x_c) * gamma || RoPE(x_r, position)] of
    projected tokens x [T, d_c + d_r] to rows ``slots`` (int64, -1: none) of
    cache_pool [num_pages, 64, d_c + d_r].  Without a table x_r is stored as it is.
    ``planned`` (int32 [1], query_start's last entry) is the number of the step's tokens: a
    T of less is recorded as MLA_ERR_BOUNDS."""
    if (_calls is not None and stream is None
            and (table is None or isinstance(table, RopeTable))):
        st = _calls.cache_write_paged(dims.address, x, gamma, positions, slots, cache_pool, table,
                                      eps, planned)
        if st is not None:
            return _check("mla_cache_write_paged", st) if st else None
    dev = _device(x, "x")
    dt, R, n = dims.torch_dtype, dims.R, cache_pool.shape[0]
    px, T, sx = _rows(x, dt, R, dev)
    _launch("mla_cache_write_paged_step", dev, stream, dims.ref, T, px, sx,
            None if gamma is None else _arg(gamma, _F32, (dims.d_c,), "gamma", dev), eps,
            _table_ptr(table),
            None if positions is None else _arg(positions, _I32, (T,), "positions", dev),
            _arg(slots, _I64, (T,), "slots", dev),
            None if planned is None else _arg(planned, _I32, (1,), "planned", dev),
            _arg(cache_pool, dt, (n, PAGE_ROWS, R), "cache_pool", dev), n,
            name="mla_cache_write_paged")


def cache_write_fp8_paged(dims: Dims, x, gamma, query_start, seqlens, block_table, cache_pool,
                          page_scales, table=None, eps=1e-6, stream=None):
    """mla_cache_write_fp8_paged: the rows of cache_write_paged into an 8-bit pool
    [num_pages, 64, d_c + 2 d_r] uint8 with one scale per page [num_pages];
    request b's rows are x[query_start[b]:query_start[b+1]], the last of its
    seqlens[b] tokens (the lengths after the step)."""
    if (_calls is not None and stream is None
            and (table is None or isinstance(table, RopeTable))):
        st = _calls.cache_write_fp8_paged(dims.address, x, gamma, query_start, seqlens, block_table,
                                          cache_pool, page_scales, table, eps)
        if st is not None:
            return _check("mla_cache_write_fp8_paged", st) if st else None
    dev = _device(x, "x")
    B, n, mb = dims.B, cache_pool.shape[0], block_table.shape[-1]
    px, T, sx = _rows(x, dims.torch_dtype, dims.R, dev)
    _launch("mla_cache_write_fp8_paged", dev, stream, dims.ref, T, px, sx,
            None if gamma is None else _arg(gamma, _F32, (dims.d_c,), "gamma", dev), eps,
            _table_ptr(table), _arg(query_start, _I32, (B + 1,), "query_start", dev),
            _arg(seqlens, _I32, (B,), "seqlens", dev),
            _arg(block_table, _I32, (B, mb), "block_table", dev), mb,
            _arg(cache_pool, torch.uint8, (n, PAGE_ROWS, dims.d_c + 2 * dims.d_r), "cache_pool", dev),
            _arg(page_scales, _F32, (n,), "page_scales", dev), n)


def decode_fp8_paged(dims: Dims, q_cat, cache_pool, page_scales, block_table, seqlens,
                     softmax_scale, workspace, num_splits=0, stream=None) -> int:
    """mla_decode_fp8_paged: mla_decode over an 8-bit paged cache (see
    cache_write_fp8_paged); returns the splits used, for combine."""
    if _calls is not None and stream is None:
        got = _calls.decode_fp8_paged(dims.address, q_cat, cache_pool, page_scales, block_table,
                                      seqlens, softmax_scale, workspace, num_splits)
        if got is not None:
            return got if got > 0 else _check("mla_decode_fp8_paged", -got)
    dev = _device(q_cat, "q_cat")
    B, n, mb = dims.B, cache_pool.shape[0], block_table.shape[-1]
    ws, nws = _ws_arg(workspace, dev)
    used = ctypes.c_int(0)
    _launch("mla_decode_fp8_paged", dev, stream, dims.ref,
            _arg(q_cat, dims.torch_dtype, (B, dims.H, dims.R), "q_cat", dev),
            _arg(cache_pool, torch.uint8, (n, PAGE_ROWS, dims.d_c + 2 * dims.d_r), "cache_pool", dev),
            _arg(page_scales, _F32, (n,), "page_scales", dev), n,
            _arg(block_table, _I32, (B, mb), "block_table", dev), mb,
            _arg(seqlens, _I32, (B,), "seqlens", dev), float(softmax_scale), num_splits, ws, nws,
            ctypes.byref(used))
    return used.value


def get_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(load_library().mla_get_device_status(_stream(stream)))


# ---------------------------------------------------------------------------
class DecodeStep:
    """One MLA decode layer on the device: owns its workspaces (allocated once
    by the caller side through torch) and runs append -> absorb_q -> decode ->
    combine -> out_proj.  All arithmetic is in the CUDA kernels; this class
    only keeps buffers, pointers and the stream order.

    absorb_q does not depend on the cache append, so with ``overlap`` it runs
    on a second stream forked from the current one and joined before decode.
    ``capture`` records one step (plus any caller work) into a CUDA graph so a
    step is replayed with one launch from the host."""

    def __init__(self, dims: Dims, W_UK, W_UV, W_DKV=None, gamma=None, softmax_scale=None,
                 rope_base=10000.0, eps=1e-6, num_splits=0, device="cuda", overlap=True,
                 rope_table=None):
        self.dims = dims
        self.W_UK, self.W_UV, self.W_DKV, self.gamma = W_UK, W_UV, W_DKV, gamma
        # 0 asks the library for the pages' scale 1/sqrt(d_nope + d_r).
        self.scale = 0.0 if softmax_scale is None else float(softmax_scale)
        self.rope_base, self.eps = rope_base, eps
        self._splits_arg = num_splits     # 8-bit pages have a default of their own
        self.num_splits = num_splits or decode_default_splits(dims)
        ws = decode_workspace_bytes(dims, self.num_splits)
        self.ws = torch.empty(ws // 4, dtype=torch.float32, device=device)
        hidden = W_DKV.shape[1] if W_DKV is not None else 1
        self.ws_append = torch.empty(max(cache_append_workspace_bytes(dims, hidden) // 4, 1),
                                     dtype=torch.float32, device=device)
        dt = dims.torch_dtype
        self.q_cat = torch.empty(dims.B, dims.H, dims.R, dtype=dt, device=device)
        self.o_lat = torch.empty(dims.B, dims.H, dims.d_c, dtype=torch.float32, device=device)
        self.lse = torch.empty(dims.B, dims.H, dtype=torch.float32, device=device)
        self.out = torch.empty(dims.B, dims.H, dims.d_v, dtype=dt, device=device)
        self.splits_used = self.num_splits
        # A rope table (see rope_table) rotates the queries in its layout and
        # scaling instead of absorb_q's half-split, unscaled rotation.
        self.rope_table = rope_table
        if rope_table is not None and rope_table.d_r != dims.d_r:
            raise ValueError(f"rope_table is for d_r = {rope_table.d_r}, not {dims.d_r}")
        self.q_rot = (torch.empty(dims.B, dims.H, dims.d_r, dtype=dt, device=device)
                      if rope_table is not None else None)
        self._side = torch.cuda.Stream(device=device) if overlap else None

    def _no_append(self, page_scales):
        if page_scales is not None or self.rope_table is not None:
            raise ValueError("8-bit pages and rope tables take their rows from "
                             "cache_write_fp8_paged / cache_write_paged, before the step (h=None)")

    def append(self, h, cache, seqlens, block_table=None, scales=None, page_scales=None):
        self._no_append(page_scales)
        if scales is not None:
            cache_append_fp8(self.dims, h, self.W_DKV, self.gamma, cache, scales, seqlens,
                             self.ws_append, self.eps, self.rope_base)
        elif block_table is None:
            cache_append(self.dims, h, self.W_DKV, self.gamma, cache, seqlens, self.ws_append,
                         self.eps, self.rope_base)
        else:
            cache_append_paged(self.dims, h, self.W_DKV, self.gamma, cache, block_table,
                               seqlens, self.ws_append, self.eps, self.rope_base)

    def absorb(self, q_nope, q_pe, q_pos):
        """absorb_q into the step's q_cat buffer."""
        if self.rope_table is not None and q_pos is not None:
            q_pe, q_pos = rope(self.rope_table, q_pe, q_pos, self.q_rot), None
        absorb_q(self.dims, q_nope, q_pe, self.W_UK, q_pos, self.q_cat, self.rope_base)

    def _attend_latent(self, cache, seqlens, block_table=None, scales=None, page_scales=None):
        if page_scales is not None:
            self.splits_used = decode_fp8_paged(self.dims, self.q_cat, cache, page_scales,
                                                block_table, seqlens, self.scale, self.ws,
                                                self._splits_arg)
        elif scales is not None:
            self.splits_used = decode_fp8(self.dims, self.q_cat, cache, scales, seqlens,
                                          self.scale, self.ws, self.num_splits)
        elif block_table is None:
            self.splits_used = decode(self.dims, self.q_cat, cache, seqlens, self.scale, self.ws,
                                      self.num_splits)
        else:
            self.splits_used = decode_paged(self.dims, self.q_cat, cache, block_table, seqlens,
                                            self.scale, self.ws, self.num_splits)
        combine(self.dims, seqlens, self.ws, self.splits_used, self.o_lat, self.lse)
        out_proj(self.dims, self.o_lat, self.W_UV, self.out)
        return self.out

    def attend(self, q_nope, q_pe, q_pos, cache, seqlens, block_table=None, scales=None,
               page_scales=None):
        self.absorb(q_nope, q_pe, q_pos)
        return self._attend_latent(cache, seqlens, block_table, scales, page_scales)

    def __call__(self, q_nope, q_pe, q_pos, cache, seqlens, h=None, block_table=None,
                 scales=None, page_scales=None):
        """One step.  With ``block_table`` the cache is a paged pool
        [num_pages, 64, R] (see decode_paged); with ``scales`` it is an FP8
        latent cache [B, capacity, d_c + 2 d_r] uint8 with its scale plane
        [B, capacity] (see decode_fp8); with ``block_table`` and
        ``page_scales`` [num_pages] an 8-bit paged pool (see decode_fp8_paged),
        whose rows are written before the step."""
        if page_scales is not None and block_table is None:
            raise ValueError("page_scales needs a block_table")
        if h is not None:
            self._no_append(page_scales)     # before the fork: a capture must be joined
        if self._side is None:
            if h is not None:
                self.append(h, cache, seqlens, block_table, scales, page_scales)
            return self.attend(q_nope, q_pe, q_pos, cache, seqlens, block_table, scales,
                               page_scales)
        main = torch.cuda.current_stream()
        # Fork: the side stream starts after everything issued so far (the
        # previous step's decode has finished reading q_cat).  absorb_q is
        # launched first: measured in a graph on B200 the pair takes 14.9 us
        # this way and 20.6 us with the append launched first (each alone
        # about 12.3 us).
        self._side.wait_stream(main)
        with torch.cuda.stream(self._side):
            self.absorb(q_nope, q_pe, q_pos)
        if h is not None:
            self.append(h, cache, seqlens, block_table, scales, page_scales)
        main.wait_stream(self._side)
        return self._attend_latent(cache, seqlens, block_table, scales, page_scales)

    def host_pipeline(self, host_inputs, host_out, cache, seqlens, after=None,
                      block_table=None, scales=None, page_scales=None):
        """Steps fed from pinned host memory with the copies overlapped.

        ``host_inputs`` = (q_nope, q_pe, q_pos[, h]) pinned host tensors,
        ``host_out`` a pinned host tensor shaped like ``self.out``.  Two device
        input sets and two output stages alternate; each is served by one CUDA
        graph that runs a step on set c while a forked copy stream brings the
        next step's inputs into set 1 - c and takes the previous step's
        output from stage 1 - c to ``host_out``.  So every step still copies
        its own inputs in and its result out, but one graph launch per step
        does it.  ``run(n)`` performs n steps, with the first step's inputs
        copied in before and the last result copied out after; ``host_out``
        holds the last step's result once the stream has finished."""
        return _HostPipeline(self, host_inputs, host_out, cache, seqlens, after, block_table,
                             scales, page_scales)

    def capture(self, q_nope, q_pe, q_pos, cache, seqlens, h=None, before=None, after=None,
                block_table=None, scales=None, page_scales=None):
        """Record one step into a CUDA graph; ``before``/``after`` are optional
        callables whose device work is recorded around it.  Replay with
        ``graph.replay()``; inputs are read from the same tensors each time."""
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if before is not None:
                before()
            self(q_nope, q_pe, q_pos, cache, seqlens, h=h, block_table=block_table,
                 scales=scales, page_scales=page_scales)
            if after is not None:
                after()
        return g


class _HostPipeline:
    """See DecodeStep.host_pipeline."""

    def __init__(self, step, host_inputs, host_out, cache, seqlens, after, block_table, scales,
                 page_scales=None):
        for t in (*host_inputs, host_out):
            if t.is_cuda or not t.is_pinned():
                raise ValueError("host_pipeline needs pinned host tensors")
        self.step, self.host_in, self.host_out = step, tuple(host_inputs), host_out
        dev = step.out.device
        self.sets = [[torch.empty_like(t, device=dev) for t in self.host_in] for _ in range(2)]
        self.stages = [torch.empty_like(step.out) for _ in range(2)]
        # Host->device and device->host copies on separate streams, so the two
        # directions overlap each other as well as the step.
        self.in_stream = torch.cuda.Stream(device=dev)
        self.out_stream = torch.cuda.Stream(device=dev)
        self.graphs = []
        # Each graph's step writes its output straight into its own stage (the
        # step's output buffer is pointed at the stage while the graph is
        # recorded), so no device copy sits between the step and the next
        # device->host copy.
        out = step.out
        try:
            for c in range(2):
                step.out = self.stages[c]
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    main = torch.cuda.current_stream()
                    self.in_stream.wait_stream(main)
                    self.out_stream.wait_stream(main)
                    with torch.cuda.stream(self.in_stream):
                        for d_t, h_t in zip(self.sets[1 - c], self.host_in):
                            d_t.copy_(h_t, non_blocking=True)
                    with torch.cuda.stream(self.out_stream):
                        self.host_out.copy_(self.stages[1 - c], non_blocking=True)
                    x = self.sets[c]
                    step(x[0], x[1], x[2], cache, seqlens, h=x[3] if len(x) > 3 else None,
                         block_table=block_table, scales=scales, page_scales=page_scales)
                    if after is not None:
                        after()
                    main.wait_stream(self.in_stream)
                    main.wait_stream(self.out_stream)
                self.graphs.append(g)
        finally:
            step.out = out

    def run(self, n: int):
        for d_t, h_t in zip(self.sets[0], self.host_in):
            d_t.copy_(h_t, non_blocking=True)
        for k in range(n):
            self.graphs[k % 2].replay()
        if n:
            self.host_out.copy_(self.stages[(n - 1) % 2], non_blocking=True)

    def bytes_per_step(self):
        """(host->device, device->host) bytes each step copies."""
        return (sum(t.numel() * t.element_size() for t in self.host_in),
                self.host_out.numel() * self.host_out.element_size())
