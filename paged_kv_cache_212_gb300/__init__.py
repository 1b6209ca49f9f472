"""GB300-native paged KV cache: page write (bf16 / int8), gather, in-place paged
decode attention with split-KV, and chunked paged prefill, as hand-written
sm_103a CUDA kernels behind the C ABI of ``libpagedkv.so`` (``include/pagedkv.h``).

This module is argument marshalling only: it checks tensor shapes, dtypes and
devices, passes raw device pointers and the current CUDA stream to the
library, and turns a non-zero status into an exception.  (The rotary, windowed
and ragged-batch calls are marshalled in native code, binding/native.cpp, as
long as they pass its checks; the ones here then say what is wrong.)  Every step of the
computation runs in the library's kernels; there is no CPU or PyTorch
fallback, and using any call without the built library raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import sysconfig
import typing
import warnings

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpagedkv.so")
# binding/native.cpp, built against this torch for this Python (build.native_lib)
NATIVE_PATH = os.path.join(HERE, f"_native-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")

PKV_KV_BF16, PKV_KV_INT8 = 0, 1
DEV_BAD_BLOCK_ID, DEV_BAD_POSITION, DEV_BAD_LENGTH = 1, 2, 4
DEV_WORKSPACE_OVERFLOW, DEV_TIMEOUT, DEV_OUT_OF_BLOCKS = 8, 16, 32

EXPORTS = ("pkv_status_string", "pkv_last_cuda_error", "pkv_set_pipeline_wait_ns", "paged_kv_write",
           "paged_kv_write_int8",
           "paged_kv_gather", "pkv_decode_workspace_bytes", "paged_decode_attention",
           "paged_prefill_attention", "paged_decode_attention_noalloc", "paged_decode_step",
           "paged_kv_copy_blocks",
           # host-side block manager (include/pagedkv_blocks.h)
           "pkv_bm_create", "pkv_bm_destroy", "pkv_bm_alloc", "pkv_bm_free", "pkv_bm_num_free",
           "pkv_bm_peak_used", "pkv_bm_refcount", "pkv_bm_can_admit", "pkv_bm_admit", "pkv_bm_release",
           "pkv_bm_fork", "pkv_bm_reserve_step", "pkv_bm_begin_step", "pkv_bm_end_step", "pkv_bm_export",
           # decode streamed from a host tier (include/pagedkv_stream.h)
           "pkv_sp_create", "pkv_sp_destroy", "pkv_sp_lookup", "pkv_sp_invalidate", "pkv_sp_plan_tile",
           "paged_kv_stage_blocks", "pkv_streamed_workspace_bytes", "paged_decode_streamed",
           # rotary positions written into the pages (include/pagedkv_rope.h)
           "pkv_rope_phases", "paged_kv_write_rope",
           # sliding window with first tokens (include/pagedkv_window.h)
           "paged_decode_attention_window", "paged_decode_step_window", "paged_prefill_attention_window",
           # batches of requests of any lengths (include/pagedkv_batch.h)
           "paged_step_maps", "paged_kv_write_slots", "pkv_rows_workspace_bytes", "paged_cross_attention",
           "paged_decode_attention_shared")
NOALLOC_DECODE_SCRATCH_BYTES = 16 * 1024 * 1024


class PagedKVError(RuntimeError):
    """A library call returned a non-zero PKV_* status (``status``; for
    PKV_ERR_CUDA the CUDA error code is in the message)."""

    def __init__(self, fn, status, name, cuda_error=0):
        msg = f"{fn} returned {name} ({status})"
        if cuda_error:
            msg += f", cudaError {cuda_error}"
        super().__init__(msg)
        self.status = status


class Dims(ctypes.Structure):
    """pkv_dims: pool geometry (n_blocks physical blocks, the pool tensors have
    n_blocks + 1 with the scratch block last)."""
    _fields_ = [("n_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _RopeC(ctypes.Structure):
    """pkv_rope."""
    _fields_ = [("phases", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("magnitude", ctypes.c_double)]


_lib = None
_native = None          # the native marshalling, once the library is loaded


def _load_native(lib):
    """binding/native.cpp with the library's entry points (None: not built, or it does
    not load, and the calls go through Python)."""
    if not os.path.exists(NATIVE_PATH):
        return None
    try:
        spec = importlib.util.spec_from_file_location("_native", NATIVE_PATH)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    except (ImportError, OSError) as e:
        warnings.warn(f"the native part of the binding was not loaded, its calls go through Python: {e!r}", RuntimeWarning)
        return None
    mod.set_functions(*(ctypes.cast(getattr(lib, fn), ctypes.c_void_p).value for fn in (
        "paged_kv_write_rope", "paged_decode_attention_window", "paged_decode_step_window",
        "paged_prefill_attention_window")))
    mod.set_batch_functions(*(ctypes.cast(getattr(lib, fn), ctypes.c_void_p).value for fn in (
        "paged_step_maps", "paged_kv_write_slots", "pkv_rows_workspace_bytes", "paged_cross_attention",
        "paged_decode_attention_shared")))
    return mod


def load_library(path: str = LIB_PATH):
    """Load libpagedkv.so (raises if it has not been built)."""
    global _lib, _native
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with paged_kv_cache_212_gb300.build.build() "
                           "(nvcc, sm_103a); there is no fallback path")
    lib = ctypes.CDLL(path)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.pkv_status_string.argtypes = [ctypes.c_int]
    lib.pkv_status_string.restype = ctypes.c_char_p
    lib.pkv_last_cuda_error.argtypes = []
    lib.pkv_last_cuda_error.restype = ctypes.c_int
    lib.pkv_set_pipeline_wait_ns.argtypes = [ctypes.c_uint64]
    lib.pkv_set_pipeline_wait_ns.restype = ctypes.c_uint64
    lib.paged_kv_write.argtypes = [P, P, P, P, Dims, P, i32, P, i32, i32, P, P]
    lib.paged_kv_write_int8.argtypes = [P, P, P, P, P, P, Dims, P, i32, P, i32, i32, P, P]
    lib.paged_kv_gather.argtypes = [P, P, Dims, P, i32, P, i32, i32, P, P, P, P]
    lib.pkv_decode_workspace_bytes.argtypes = [i32, i32, i32, i64, i32]
    lib.pkv_decode_workspace_bytes.restype = sz
    lib.paged_decode_attention.argtypes = [P, i32, P, P, P, P, i32, Dims, P, i32, P, i32, ctypes.c_float,
                                           i32, P, P, P, sz, P, P]
    lib.paged_prefill_attention.argtypes = [P, i32, P, P, Dims, P, i32, P, i32, i32, ctypes.c_float, P, P,
                                            P, P]
    lib.paged_decode_attention_noalloc.argtypes = [P, i32, P, P, P, P, i32, Dims, P, i32, P, i32,
                                                   ctypes.c_float, i32, i64, P, P, P, P]
    lib.paged_decode_step.argtypes = [P, P, P, i32, P, i32, P, P, P, P, i32, Dims, P, i32, P, i32,
                                      ctypes.c_float, i32, P, P, P, sz, P, P]
    lib.paged_kv_copy_blocks.argtypes = [P, i32, P, P, P, P, i32, Dims, P, P]
    for fn in ("paged_kv_write", "paged_kv_write_int8", "paged_kv_gather", "paged_decode_attention",
               "paged_prefill_attention", "paged_decode_attention_noalloc", "paged_decode_step",
               "paged_kv_copy_blocks"):
        getattr(lib, fn).restype = ctypes.c_int
    PP = ctypes.POINTER(ctypes.c_void_p)
    lib.pkv_bm_create.argtypes = [i32, i32, i32, i32, PP]
    lib.pkv_bm_destroy.argtypes = [P]
    lib.pkv_bm_destroy.restype = None
    lib.pkv_bm_alloc.argtypes = [P, P]
    lib.pkv_bm_free.argtypes = [P, P, i32]
    lib.pkv_bm_num_free.argtypes = [P]
    lib.pkv_bm_peak_used.argtypes = [P]
    lib.pkv_bm_refcount.argtypes = [P, i32]
    lib.pkv_bm_can_admit.argtypes = [P, P, i32, P]
    lib.pkv_bm_admit.argtypes = [P, i32, i32]
    lib.pkv_bm_release.argtypes = [P, i32]
    lib.pkv_bm_fork.argtypes = [P, i32, i32]
    lib.pkv_bm_reserve_step.argtypes = [P, P, P]
    lib.pkv_bm_begin_step.argtypes = [P, P, P]
    lib.pkv_bm_end_step.argtypes = [P]
    lib.pkv_bm_export.argtypes = [P, P, P, P]
    for fn in EXPORTS:
        if fn.startswith("pkv_bm_") and fn != "pkv_bm_destroy":
            getattr(lib, fn).restype = ctypes.c_int
    lib.pkv_sp_create.argtypes = [i32, i32, PP]
    lib.pkv_sp_destroy.argtypes = [P]
    lib.pkv_sp_destroy.restype = None
    lib.pkv_sp_lookup.argtypes = [P, i32]
    lib.pkv_sp_invalidate.argtypes = [P, i32]
    lib.pkv_sp_plan_tile.argtypes = [P, P, i32, P, i32, i32, i32, P, P, P, P, P, P]
    lib.paged_kv_stage_blocks.argtypes = [P, i32, P, P, i32, P, P, Dims, P, P]
    lib.pkv_streamed_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.pkv_streamed_workspace_bytes.restype = sz
    lib.paged_decode_streamed.argtypes = [P, i32, P, P, i32, P, P, Dims, P, P, i32, P, i32, ctypes.c_float, P, P,
                                          P, sz, P, P]
    for fn in ("pkv_sp_create", "pkv_sp_lookup", "pkv_sp_invalidate", "pkv_sp_plan_tile", "paged_kv_stage_blocks",
               "paged_decode_streamed"):
        getattr(lib, fn).restype = ctypes.c_int
    f32, f64, RP = ctypes.c_float, ctypes.c_double, ctypes.POINTER(_RopeC)
    lib.pkv_rope_phases.argtypes = [i32, f64, i32, f64, f64, f64, f64, P, ctypes.POINTER(f64)]
    lib.paged_kv_write_rope.argtypes = [P, i64, i32, P, i64, P, i64, RP, P, P, P, P, P, i32, Dims, P, i32, P, i32, i32,
                                        P, P]
    lib.paged_decode_attention_window.argtypes = [P, i32, P, P, P, P, i32, Dims, P, i32, P, i32, f32, i32, i32, P, P,
                                                  P, P]
    lib.paged_decode_step_window.argtypes = [P, i64, P, i64, P, P, i64, i32, RP, P, P, P, P, i32, Dims, P, i32, P, i32,
                                             f32, i32, i32, P, P, P, P]
    lib.paged_prefill_attention_window.argtypes = [P, i32, P, P, Dims, P, i32, P, i32, i32, f32, i32, i32, P, P, P, P]
    for fn in ("pkv_rope_phases", "paged_kv_write_rope", "paged_decode_attention_window", "paged_decode_step_window",
               "paged_prefill_attention_window"):
        getattr(lib, fn).restype = ctypes.c_int
    lib.paged_step_maps.argtypes = [P, P, i32, P, i32, P, i32, i32, P, i32, i32, P, P, P, P, P, P, P, P]
    lib.paged_kv_write_slots.argtypes = [P, i64, P, i64, P, P, P, P, i32, Dims, P, i32, P, P]
    lib.pkv_rows_workspace_bytes.argtypes = [i32, i32, i32]
    lib.pkv_rows_workspace_bytes.restype = sz
    lib.paged_cross_attention.argtypes = [P, i64, i32, P, i32, P, P, P, P, i32, Dims, P, i32, P, i32, f32, P, P, P, sz, P,
                                          P]
    lib.paged_decode_attention_shared.argtypes = [P, i64, i32, P, P, P, P, i32, Dims, P, i32, P, i32, P, i32, P, i32, P,
                                                  f32, P, P, P, sz, P, P]
    for fn in ("paged_step_maps", "paged_kv_write_slots", "paged_cross_attention", "paged_decode_attention_shared"):
        getattr(lib, fn).restype = ctypes.c_int
    _native = _load_native(lib)
    _lib = lib
    return lib


def _check(fn, status):
    if status != 0:
        lib = load_library()
        raise PagedKVError(fn, status, lib.pkv_status_string(status).decode(),
                           lib.pkv_last_cuda_error())


def _ptr(t):
    # ctypes turns an int into the void * argument
    return None if t is None else t.data_ptr()


try:
    from torch._C import _cuda_getCurrentRawStream as _raw_stream, _cuda_getDevice as _current_device
except ImportError:      # pragma: no cover - older PyTorch builds
    _raw_stream = _current_device = None


def _stream(stream):
    """The cudaStream_t of `stream`, or of the current stream of the current
    device (as an int)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(_current_device())
    return torch.cuda.current_stream().cuda_stream


def _device_of(t, name):
    """CUDA device index of the tensor the other arguments must share."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return d


def _need(t, name, dtype=None, ndim=None, device=None):
    """A contiguous CUDA tensor of the given dtype, rank and device index; the
    common case is one test, the messages come from _refuse."""
    if (isinstance(t, torch.Tensor) and (dtype is None or t.dtype is dtype) and (ndim is None or t.dim() == ndim)
            and t.is_contiguous() and (t.get_device() == device if device is not None else t.is_cuda)):
        return
    _refuse(t, name, dtype, ndim, device)


def _refuse(t, name, dtype, ndim, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} was refused")


def _shape(t, name, shape):
    """A tensor of the wrong shape would become an out-of-bounds device access:
    refuse it here."""
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_status(dev_status, device):
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, None, device)
        if dev_status.numel() < 1:
            raise ValueError("dev_status needs at least one int32")


def _check_pools(k_pool, v_pool, k_scales=None, v_scales=None):
    _shape(v_pool, "v_pool", k_pool.shape)
    _shape(k_scales, "k_scales", k_pool.shape[:3])
    _shape(v_scales, "v_scales", k_pool.shape[:3])


def _check_batch(n_seqs, block_tables, lens, lens_name):
    if block_tables.shape[0] != n_seqs:
        raise ValueError(f"block_tables has {block_tables.shape[0]} rows for {n_seqs} sequences")
    _shape(lens, lens_name, (n_seqs,))


def pool_dims(k_pool: torch.Tensor) -> Dims:
    """Geometry of a [n_blocks + 1, block_size, n_kv_heads, head_dim] pool (the
    last row is the scratch block)."""
    nb1, bs, hkv, d = k_pool.shape
    return Dims(nb1 - 1, bs, hkv, d)


_dims_cache = {}


def _dims(k_pool):
    """pool_dims, one shared (never modified) structure per pool shape."""
    d = _dims_cache.get(k_pool.shape)
    if d is None:
        if len(_dims_cache) > 64:
            _dims_cache.clear()
        d = _dims_cache[k_pool.shape] = pool_dims(k_pool)
    return d


def paged_kv_write(k_new, v_new, k_pool, v_pool, block_tables, start_pos, dev_status=None, stream=None):
    """Native bf16 page write: k_new/v_new [n_seqs, n_new, Hkv, D] to positions
    start_pos[s] .. of each sequence."""
    lib = load_library()
    dev = _device_of(k_pool, "k_pool")
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_pool, "k_pool"), (v_pool, "v_pool")):
        _need(t, n, torch.bfloat16, 4, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(start_pos, "start_pos", torch.int32, 1, dev)
    _check_status(dev_status, dev)
    _check_pools(k_pool, v_pool)
    _shape(k_new, "k_new", (k_new.shape[0], k_new.shape[1]) + tuple(k_pool.shape[2:]))
    _shape(v_new, "v_new", k_new.shape)
    _check_batch(k_new.shape[0], block_tables, start_pos, "start_pos")
    st = lib.paged_kv_write(_ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool), _dims(k_pool),
                            _ptr(block_tables), block_tables.shape[1], _ptr(start_pos), k_new.shape[0],
                            k_new.shape[1], _ptr(dev_status), _stream(stream))
    _check("paged_kv_write", st)


def paged_kv_write_int8(k_new, v_new, k_pool, v_pool, k_scales, v_scales, block_tables, start_pos,
                        dev_status=None, stream=None):
    """Quantised page write: int8 pools [NB+1, bs, Hkv, D], fp32 scales [NB+1, bs, Hkv]."""
    lib = load_library()
    dev = _device_of(k_pool, "k_pool")
    _need(k_new, "k_new", torch.bfloat16, 4, dev)
    _need(v_new, "v_new", torch.bfloat16, 4, dev)
    _need(k_pool, "k_pool", torch.int8, 4, dev)
    _need(v_pool, "v_pool", torch.int8, 4, dev)
    _need(k_scales, "k_scales", torch.float32, 3, dev)
    _need(v_scales, "v_scales", torch.float32, 3, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(start_pos, "start_pos", torch.int32, 1, dev)
    _check_status(dev_status, dev)
    _check_pools(k_pool, v_pool, k_scales, v_scales)
    _shape(k_new, "k_new", (k_new.shape[0], k_new.shape[1]) + tuple(k_pool.shape[2:]))
    _shape(v_new, "v_new", k_new.shape)
    _check_batch(k_new.shape[0], block_tables, start_pos, "start_pos")
    st = lib.paged_kv_write_int8(_ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool), _ptr(k_scales),
                                 _ptr(v_scales), _dims(k_pool), _ptr(block_tables), block_tables.shape[1],
                                 _ptr(start_pos), k_new.shape[0], k_new.shape[1], _ptr(dev_status),
                                 _stream(stream))
    _check("paged_kv_write_int8", st)


def paged_kv_gather(k_pool, v_pool, block_tables, lens, out_tokens, k_out=None, v_out=None, dev_status=None,
                    stream=None):
    """Contiguous copy [n_seqs, Hkv, out_tokens, D] of every sequence's pages
    (zeros past its length).  Returns (k_out, v_out)."""
    lib = load_library()
    dev = _device_of(k_pool, "k_pool")
    _need(k_pool, "k_pool", torch.bfloat16, 4, dev)
    _need(v_pool, "v_pool", torch.bfloat16, 4, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(lens, "lens", torch.int32, 1, dev)
    n_seqs = block_tables.shape[0]
    shape = (n_seqs, k_pool.shape[2], int(out_tokens), k_pool.shape[3])
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if v_out is None:
        v_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    _need(k_out, "k_out", torch.bfloat16, 4, dev)
    _need(v_out, "v_out", torch.bfloat16, 4, dev)
    _check_status(dev_status, dev)
    _check_pools(k_pool, v_pool)
    _check_batch(n_seqs, block_tables, lens, "lens")
    _shape(k_out, "k_out", shape)
    _shape(v_out, "v_out", shape)
    st = lib.paged_kv_gather(_ptr(k_pool), _ptr(v_pool), _dims(k_pool), _ptr(block_tables),
                             block_tables.shape[1], _ptr(lens), n_seqs, int(out_tokens), _ptr(k_out), _ptr(v_out),
                             _ptr(dev_status), _stream(stream))
    _check("paged_kv_gather", st)
    return k_out, v_out


def paged_kv_copy_blocks(pairs, k_pool, v_pool, k_scales=None, v_scales=None, dev_status=None, stream=None):
    """Copy whole pool blocks: pairs int32 [n, 2] of (source, destination) ids
    on the device (the device half of copy-on-write)."""
    lib = load_library()
    dev = _device_of(k_pool, "k_pool")
    _need(pairs, "pairs", torch.int32, 2, dev)
    int8 = k_pool.dtype == torch.int8
    if int8:
        _need(k_scales, "k_scales", torch.float32, 3, dev)
        _need(v_scales, "v_scales", torch.float32, 3, dev)
    else:
        _need(k_pool, "k_pool", torch.bfloat16, 4, dev)
    _need(v_pool, "v_pool", k_pool.dtype, 4, dev)
    _check_status(dev_status, dev)
    _check_pools(k_pool, v_pool, k_scales if int8 else None, v_scales if int8 else None)
    if pairs.shape[1] != 2:
        raise ValueError(f"pairs must be [n, 2], got {tuple(pairs.shape)}")
    st = lib.paged_kv_copy_blocks(_ptr(pairs), pairs.shape[0], _ptr(k_pool), _ptr(v_pool), _ptr(k_scales),
                                  _ptr(v_scales), PKV_KV_INT8 if int8 else PKV_KV_BF16, _dims(k_pool),
                                  _ptr(dev_status), _stream(stream))
    _check("paged_kv_copy_blocks", st)


def decode_workspace_bytes(n_seqs, n_q_heads, head_dim, max_total_ctx_tokens, split_tokens=0) -> int:
    """Device workspace a decode call needs for batches of n_seqs sequences whose
    contexts sum to at most max_total_ctx_tokens (pkv_decode_workspace_bytes)."""
    n = load_library().pkv_decode_workspace_bytes(int(n_seqs), int(n_q_heads), int(head_dim),
                                                  int(max_total_ctx_tokens), int(split_tokens))
    if n == 0:
        raise ValueError("invalid arguments to pkv_decode_workspace_bytes")
    return int(n)


def _check_decode(q, k_pool, v_pool, k_scales, v_scales, block_tables, ctx_lens, out, lse_out, dev_status):
    """Shapes of a decode call's tensors against q [n_seqs, Hq, D] and the pool."""
    n_seqs, n_q_heads, D = q.shape
    _check_status(dev_status, q.get_device())
    _check_pools(k_pool, v_pool, k_scales, v_scales)
    if k_pool.shape[3] != D:
        raise ValueError(f"q has head_dim {D}, the pool {k_pool.shape[3]}")
    _check_batch(n_seqs, block_tables, ctx_lens, "ctx_lens")
    _shape(out, "out", q.shape)
    _shape(lse_out, "lse_out", (n_seqs, n_q_heads))


def paged_decode_attention(q, k_pool, v_pool, block_tables, ctx_lens, softmax_scale, k_scales=None,
                           v_scales=None, split_tokens=0, out=None, lse_out=None, workspace=None,
                           max_total_ctx_tokens=None, dev_status=None, stream=None):
    """In-place paged GQA decode attention.  q [n_seqs, Hq, D] bf16; bf16 pools,
    or int8 pools with k_scales/v_scales.  Returns out [n_seqs, Hq, D] bf16.
    ``workspace`` (uint8 CUDA tensor) is allocated when not given, sized from
    max_total_ctx_tokens (default: every table entry full)."""
    lib = load_library()
    dev = _device_of(q, "q")
    _need(q, "q", torch.bfloat16, 3, dev)
    int8 = k_pool.dtype == torch.int8
    _need(k_pool, "k_pool", torch.int8 if int8 else torch.bfloat16, 4, dev)
    _need(v_pool, "v_pool", torch.int8 if int8 else torch.bfloat16, 4, dev)
    if int8:
        _need(k_scales, "k_scales", torch.float32, 3, dev)
        _need(v_scales, "v_scales", torch.float32, 3, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(ctx_lens, "ctx_lens", torch.int32, 1, dev)
    n_seqs, n_q_heads, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 3, dev)
    if lse_out is not None:
        _need(lse_out, "lse_out", torch.float32, 2, dev)
    _check_decode(q, k_pool, v_pool, k_scales, v_scales, block_tables, ctx_lens, out, lse_out, dev_status)
    if workspace is None:
        if max_total_ctx_tokens is None:
            max_total_ctx_tokens = n_seqs * block_tables.shape[1] * k_pool.shape[1]
        nbytes = decode_workspace_bytes(n_seqs, n_q_heads, D, max_total_ctx_tokens, split_tokens)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, 1, dev)
    st = lib.paged_decode_attention(_ptr(q), n_q_heads, _ptr(k_pool), _ptr(v_pool), _ptr(k_scales),
                                    _ptr(v_scales), PKV_KV_INT8 if int8 else PKV_KV_BF16, _dims(k_pool),
                                    _ptr(block_tables), block_tables.shape[1], _ptr(ctx_lens), n_seqs,
                                    float(softmax_scale), int(split_tokens), _ptr(out), _ptr(lse_out),
                                    _ptr(workspace), workspace.numel(), _ptr(dev_status), _stream(stream))
    _check("paged_decode_attention", st)
    return out


def paged_decode_step(k_new, v_new, start_pos, q, k_pool, v_pool, block_tables, ctx_lens, softmax_scale,
                      k_scales=None, v_scales=None, split_tokens=0, out=None, lse_out=None, workspace=None,
                      max_total_ctx_tokens=None, dev_status=None, stream=None):
    """One decode step of one layer: the page write of k_new/v_new
    [n_seqs, n_new, Hkv, D] at start_pos (int8 pools: quantised) and paged
    decode attention over ctx_lens tokens (which count the new rows), in one
    call.  Returns out [n_seqs, Hq, D] bf16."""
    lib = load_library()
    dev = _device_of(q, "q")
    _need(q, "q", torch.bfloat16, 3, dev)
    _need(k_new, "k_new", torch.bfloat16, 4, dev)
    _need(v_new, "v_new", torch.bfloat16, 4, dev)
    _need(start_pos, "start_pos", torch.int32, 1, dev)
    int8 = k_pool.dtype == torch.int8
    _need(k_pool, "k_pool", torch.int8 if int8 else torch.bfloat16, 4, dev)
    _need(v_pool, "v_pool", torch.int8 if int8 else torch.bfloat16, 4, dev)
    if int8:
        _need(k_scales, "k_scales", torch.float32, 3, dev)
        _need(v_scales, "v_scales", torch.float32, 3, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(ctx_lens, "ctx_lens", torch.int32, 1, dev)
    n_seqs, n_q_heads, D = q.shape
    if k_new.shape[0] != n_seqs:
        raise ValueError("k_new and q disagree on n_seqs")
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 3, dev)
    if lse_out is not None:
        _need(lse_out, "lse_out", torch.float32, 2, dev)
    _check_decode(q, k_pool, v_pool, k_scales, v_scales, block_tables, ctx_lens, out, lse_out, dev_status)
    _shape(k_new, "k_new", (n_seqs, k_new.shape[1]) + tuple(k_pool.shape[2:]))
    _shape(v_new, "v_new", k_new.shape)
    _shape(start_pos, "start_pos", (n_seqs,))
    if workspace is None:
        if max_total_ctx_tokens is None:
            max_total_ctx_tokens = n_seqs * block_tables.shape[1] * k_pool.shape[1]
        nbytes = decode_workspace_bytes(n_seqs, n_q_heads, D, max_total_ctx_tokens, split_tokens)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, 1, dev)
    st = lib.paged_decode_step(_ptr(k_new), _ptr(v_new), _ptr(start_pos), k_new.shape[1], _ptr(q), n_q_heads,
                               _ptr(k_pool), _ptr(v_pool), _ptr(k_scales), _ptr(v_scales),
                               PKV_KV_INT8 if int8 else PKV_KV_BF16, _dims(k_pool), _ptr(block_tables),
                               block_tables.shape[1], _ptr(ctx_lens), n_seqs, float(softmax_scale),
                               int(split_tokens), _ptr(out), _ptr(lse_out), _ptr(workspace), workspace.numel(),
                               _ptr(dev_status), _stream(stream))
    _check("paged_decode_step", st)
    return out


class DecodePlan:
    """paged_decode_attention / paged_decode_step with the arguments that stay
    the same from call to call checked once: the pools (and int8 scales), the
    block tables and lengths, the workspace, out, lse_out and dev_status.
    ``run(q)`` then checks only q (and, for a step, k_new / v_new / start_pos)
    before the library call, which keeps the host's cost per call low where
    the GPU work is short (small batches, one call per layer).

    The plan keeps references to its tensors and reads their contents at every
    call (so block tables and lengths may be rewritten in place between calls);
    they must keep their shapes and storage: resizing one after planning is not
    allowed.  ``max_total_ctx_tokens`` bounds sum(ctx_lens) over every call.
    Returns ``out`` from ``run``."""

    def __init__(self, k_pool, v_pool, block_tables, ctx_lens, softmax_scale, n_q_heads, k_scales=None,
                 v_scales=None, split_tokens=0, out=None, lse_out=None, workspace=None, max_total_ctx_tokens=None,
                 dev_status=None):
        dev = _device_of(k_pool, "k_pool")
        self._lib = load_library()
        n_seqs, D = block_tables.shape[0], k_pool.shape[3]
        q_like = torch.empty((n_seqs, int(n_q_heads), D), dtype=torch.bfloat16, device=dev)
        if out is None:
            out = torch.empty_like(q_like)
        # the one-call checks against a query of the planned shape
        self.int8 = k_pool.dtype is torch.int8
        _need(k_pool, "k_pool", torch.int8 if self.int8 else torch.bfloat16, 4, dev)
        _need(v_pool, "v_pool", torch.int8 if self.int8 else torch.bfloat16, 4, dev)
        if self.int8:
            _need(k_scales, "k_scales", torch.float32, 3, dev)
            _need(v_scales, "v_scales", torch.float32, 3, dev)
        _need(block_tables, "block_tables", torch.int32, 2, dev)
        _need(ctx_lens, "ctx_lens", torch.int32, 1, dev)
        _need(out, "out", torch.bfloat16, 3, dev)
        if lse_out is not None:
            _need(lse_out, "lse_out", torch.float32, 2, dev)
        _check_decode(q_like, k_pool, v_pool, k_scales, v_scales, block_tables, ctx_lens, out, lse_out, dev_status)
        if workspace is None:
            if max_total_ctx_tokens is None:
                max_total_ctx_tokens = n_seqs * block_tables.shape[1] * k_pool.shape[1]
            workspace = torch.empty(decode_workspace_bytes(n_seqs, n_q_heads, D, max_total_ctx_tokens,
                                                           split_tokens), dtype=torch.uint8, device=dev)
        _need(workspace, "workspace", torch.uint8, 1, dev)
        self.device, self.q_shape, self.out = dev, q_like.shape, out
        self.new_shape_tail = tuple(k_pool.shape[2:])
        # held so that the pointers below stay valid
        self._tensors = (k_pool, v_pool, k_scales, v_scales, block_tables, ctx_lens, out, lse_out, workspace,
                         dev_status)
        self._pools = (_ptr(k_pool), _ptr(v_pool), _ptr(k_scales), _ptr(v_scales),
                       PKV_KV_INT8 if self.int8 else PKV_KV_BF16, pool_dims(k_pool), _ptr(block_tables),
                       block_tables.shape[1], _ptr(ctx_lens), n_seqs, float(softmax_scale), int(split_tokens),
                       _ptr(out), _ptr(lse_out), _ptr(workspace), workspace.numel(), _ptr(dev_status))
        self.n_q_heads, self.n_seqs = int(n_q_heads), n_seqs

    def run(self, q, k_new=None, v_new=None, start_pos=None, stream=None):
        """Decode attention of q [n_seqs, Hq, D] (bf16) over the planned pools;
        with k_new / v_new [n_seqs, n_new, Hkv, D] and start_pos [n_seqs] the
        step's page write runs first, in the same call (paged_decode_step)."""
        dev = self.device
        _need(q, "q", torch.bfloat16, 3, dev)
        _shape(q, "q", self.q_shape)
        if k_new is None:
            if v_new is not None or start_pos is not None:
                raise ValueError("v_new and start_pos come with k_new")
            st = self._lib.paged_decode_attention(q.data_ptr(), self.n_q_heads, *self._pools, _stream(stream))
            _check("paged_decode_attention", st)
            return self.out
        _need(k_new, "k_new", torch.bfloat16, 4, dev)
        _need(v_new, "v_new", torch.bfloat16, 4, dev)
        _need(start_pos, "start_pos", torch.int32, 1, dev)
        n_new = k_new.shape[1]
        _shape(k_new, "k_new", (self.n_seqs, n_new) + self.new_shape_tail)
        _shape(v_new, "v_new", k_new.shape)
        _shape(start_pos, "start_pos", (self.n_seqs,))
        st = self._lib.paged_decode_step(k_new.data_ptr(), v_new.data_ptr(), start_pos.data_ptr(), n_new,
                                         q.data_ptr(), self.n_q_heads, *self._pools, _stream(stream))
        _check("paged_decode_step", st)
        return self.out


def paged_decode_attention_noalloc(q, k_pool, v_pool, block_tables, ctx_lens, softmax_scale,
                                   max_total_ctx_tokens, out, k_scales=None, v_scales=None, split_tokens=0,
                                   lse_out=None, dev_status=None, stream=None):
    """paged_decode_attention for callers that cannot allocate device memory:
    the split-KV scratch is the library's own static 16 MiB device array, so
    no workspace is passed and the call allocates nothing (``out`` must be
    given).  max_total_ctx_tokens bounds sum(ctx_lens); a request whose
    scratch would not fit raises (PKV_ERR_WORKSPACE).  Calls share the one
    array: do not let two of them overlap on the GPU."""
    lib = load_library()
    dev = _device_of(q, "q")
    _need(q, "q", torch.bfloat16, 3, dev)
    int8 = k_pool.dtype == torch.int8
    _need(k_pool, "k_pool", torch.int8 if int8 else torch.bfloat16, 4, dev)
    _need(v_pool, "v_pool", torch.int8 if int8 else torch.bfloat16, 4, dev)
    if int8:
        _need(k_scales, "k_scales", torch.float32, 3, dev)
        _need(v_scales, "v_scales", torch.float32, 3, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(ctx_lens, "ctx_lens", torch.int32, 1, dev)
    _need(out, "out", torch.bfloat16, 3, dev)
    if lse_out is not None:
        _need(lse_out, "lse_out", torch.float32, 2, dev)
    _check_decode(q, k_pool, v_pool, k_scales, v_scales, block_tables, ctx_lens, out, lse_out, dev_status)
    n_seqs, n_q_heads, _ = q.shape
    st = lib.paged_decode_attention_noalloc(_ptr(q), n_q_heads, _ptr(k_pool), _ptr(v_pool), _ptr(k_scales),
                                            _ptr(v_scales), PKV_KV_INT8 if int8 else PKV_KV_BF16,
                                            _dims(k_pool), _ptr(block_tables), block_tables.shape[1],
                                            _ptr(ctx_lens), n_seqs, float(softmax_scale), int(split_tokens),
                                            int(max_total_ctx_tokens), _ptr(out), _ptr(lse_out),
                                            _ptr(dev_status), _stream(stream))
    _check("paged_decode_attention_noalloc", st)
    return out


def paged_prefill_attention(q, k_pool, v_pool, block_tables, prefix_lens, softmax_scale, out=None,
                            lse_out=None, dev_status=None, stream=None):
    """Chunked paged prefill: q [n_seqs, chunk, Hq, D] bf16 (the chunk's K/V
    already written at prefix_lens[s] ..).  Returns out, same shape as q."""
    lib = load_library()
    dev = _device_of(q, "q")
    _need(q, "q", torch.bfloat16, 4, dev)
    _need(k_pool, "k_pool", torch.bfloat16, 4, dev)
    _need(v_pool, "v_pool", torch.bfloat16, 4, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(prefix_lens, "prefix_lens", torch.int32, 1, dev)
    n_seqs, chunk, n_q_heads, _ = q.shape
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 4, dev)
    if lse_out is not None:
        _need(lse_out, "lse_out", torch.float32, 3, dev)
    _check_status(dev_status, dev)
    _check_pools(k_pool, v_pool)
    if k_pool.shape[3] != q.shape[3]:
        raise ValueError(f"q has head_dim {q.shape[3]}, the pool {k_pool.shape[3]}")
    _check_batch(n_seqs, block_tables, prefix_lens, "prefix_lens")
    _shape(out, "out", q.shape)
    _shape(lse_out, "lse_out", q.shape[:3])
    st = lib.paged_prefill_attention(_ptr(q), n_q_heads, _ptr(k_pool), _ptr(v_pool), _dims(k_pool),
                                     _ptr(block_tables), block_tables.shape[1], _ptr(prefix_lens), n_seqs,
                                     chunk, float(softmax_scale), _ptr(out), _ptr(lse_out), _ptr(dev_status),
                                     _stream(stream))
    _check("paged_prefill_attention", st)
    return out


# ---- rotary positions and sliding windows -----------------------------------

ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}
_ROPE_TURNS = {"bands": (1.0, 4.0), "yarn": (1.0, 32.0)}      # low_turns, high_turns


class Rope:
    """The rotary turn of a model: rot_dim of each head's elements, pairs in the
    half layout (i, i + rot_dim / 2) or interleaved (2 i, 2 i + 1), frequencies
    base^(-2 i / rot_dim) scaled for contexts beyond original_context by
    ``factor`` ("linear", "ntk", "bands", "yarn": include/pagedkv_rope.h gives
    the formulas; low_turns / high_turns default to 1 / 4 for bands, 1 / 32 for
    yarn).  Holds the phases on the device; made once per model."""

    def __init__(self, rot_dim, base=10000.0, interleaved=False, scaling="none", factor=1.0, original_context=None,
                 low_turns=None, high_turns=None, device="cuda"):
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
        low, high = _ROPE_TURNS.get(scaling, (1.0, 2.0))
        low, high = low if low_turns is None else low_turns, high if high_turns is None else high_turns
        if scaling in _ROPE_TURNS and original_context is None:
            raise ValueError(f"scaling {scaling!r} needs original_context")
        self.rot_dim, self.interleaved = int(rot_dim), bool(interleaved)
        host = torch.empty(max(self.rot_dim, 0) // 2, dtype=torch.int64)
        magnitude = ctypes.c_double()
        _check("pkv_rope_phases", load_library().pkv_rope_phases(
            self.rot_dim, float(base), ROPE_SCALINGS[scaling], float(factor), float(original_context or 0.0),
            float(low), float(high), host.data_ptr(), ctypes.byref(magnitude)))
        self.magnitude = magnitude.value
        self.phases = host.to(device)             # 2^64 turns per position, as int64 bits
        self._c = _RopeC(self.phases.data_ptr(), self.rot_dim, int(self.interleaved), self.magnitude)
        self._p, self._address = ctypes.pointer(self._c), ctypes.addressof(self._c)


def _rope_arg(rope, head_dim, dev):
    """The pkv_rope pointer of a Rope on the call's device (None: no turn)."""
    if rope is None:
        return None
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope")
    if rope.phases.get_device() != dev:
        raise ValueError(f"rope is on {rope.phases.device}, expected cuda:{dev}")
    if rope.rot_dim > head_dim:
        raise ValueError(f"rope turns {rope.rot_dim} elements of heads of {head_dim}")
    return rope._p


def _token_stride(t, name, ndim, dev):
    """Elements between the tokens of t [..., heads, D] (bf16): its head rows lie
    behind one another, its tokens one stride apart (so t may be a part of a
    fused projection's rows)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    shape, stride = t.shape, t.stride()
    heads, d = shape[-2], shape[-1]
    if (d > 1 and stride[-1] != 1) or (heads > 1 and stride[-2] != d):
        raise ValueError(f"{name}: the heads of a token must lie behind one another, got strides {stride}")
    step = heads * d
    if shape[0] > 1:
        step = stride[0]
    if ndim == 4 and shape[1] > 1:
        if shape[0] > 1 and stride[0] != shape[1] * stride[1]:
            raise ValueError(f"{name}: tokens must be one stride apart, got strides {stride}")
        step = stride[1]
    return step


def _count(x, name):
    """A token count as int32: no length reaches 2^31, so larger ones mean that."""
    x = int(x)
    if x < 0:
        raise ValueError(f"{name} must not be negative, got {x}")
    return min(x, 0x7fffffff)


def _elsewhere(dev):
    """Whether the tensors' device is not the current one (the call is then made
    with that device current, on its current stream)."""
    return (_current_device() if _current_device is not None else torch.cuda.current_device()) != dev


def _empty(shape, dtype, dev, stream):
    """An output that belongs to the stream the call writes it on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _check_paged(k_pool, v_pool, k_scales, v_scales, block_tables, dev):
    """Pools of bf16 or int8 (with scales) pages and their tables; True for int8."""
    int8 = _check_pool_kinds(k_pool, v_pool, k_scales, v_scales, dev)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    return int8


def _check_pool_kinds(k_pool, v_pool, k_scales, v_scales, dev):
    """Pools of bf16 or int8 (with scales) pages; True for int8."""
    int8 = k_pool.dtype is torch.int8
    kind = torch.int8 if int8 else torch.bfloat16
    _need(k_pool, "k_pool", kind, 4, dev)
    _need(v_pool, "v_pool", kind, 4, dev)
    if int8:
        _need(k_scales, "k_scales", torch.float32, 3, dev)
        _need(v_scales, "v_scales", torch.float32, 3, dev)
        _check_pools(k_pool, v_pool, k_scales, v_scales)
    else:
        _check_pools(k_pool, v_pool)
    return int8


def paged_kv_write_rope(q, k_new, v_new, rope, k_pool, v_pool, block_tables, start_pos, k_scales=None, v_scales=None,
                        q_out=None, dev_status=None, stream=None):
    """Rotary positions and the page write in one launch: the query and key heads
    of token j of sequence s are turned at position start_pos[s] + j, its key and
    value rows go into the pages (bf16, or int8 with k_scales / v_scales).
    q [n_seqs, n_new, Hq, D], k_new / v_new [n_seqs, n_new, Hkv, D] bf16; the
    three may be parts of a fused projection's rows.  Returns the turned queries
    (q_out, contiguous; q itself may be given)."""
    if stream is None and _native is not None and type(rope) is Rope:
        done = _native.write_rope(q, k_new, v_new, rope._address, rope.phases, k_pool, v_pool, block_tables, start_pos,
                                  k_scales, v_scales, q_out, dev_status)
        if done is not None:
            if type(done) is int:
                _check("paged_kv_write_rope", done)
            return done
    dev = _device_of(k_pool, "k_pool")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return paged_kv_write_rope(q, k_new, v_new, rope, k_pool, v_pool, block_tables, start_pos, k_scales,
                                       v_scales, q_out, dev_status, stream)
    lib = load_library()
    int8 = _check_paged(k_pool, v_pool, k_scales, v_scales, block_tables, dev)
    qs, ks, vs = (_token_stride(t, n, 4, dev) for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new")))
    n_seqs, n_new, n_q_heads, D = q.shape
    if rope is None:
        raise TypeError("rope must be a Rope")
    rp = _rope_arg(rope, D, dev)
    _need(start_pos, "start_pos", torch.int32, 1, dev)
    _shape(k_new, "k_new", (n_seqs, n_new) + tuple(k_pool.shape[2:]))
    _shape(v_new, "v_new", k_new.shape)
    if D != k_pool.shape[3]:
        raise ValueError(f"q has head_dim {D}, the pool {k_pool.shape[3]}")
    _check_batch(n_seqs, block_tables, start_pos, "start_pos")
    _check_status(dev_status, dev)
    if q_out is None:
        q_out = _empty(q.shape, torch.bfloat16, dev, stream)
    else:
        _need(q_out, "q_out", torch.bfloat16, 4, dev)
        _shape(q_out, "q_out", q.shape)
    st = lib.paged_kv_write_rope(_ptr(q), qs, n_q_heads, _ptr(k_new), ks, _ptr(v_new), vs, rp, _ptr(q_out),
                                 _ptr(k_pool), _ptr(v_pool), _ptr(k_scales), _ptr(v_scales),
                                 PKV_KV_INT8 if int8 else PKV_KV_BF16, _dims(k_pool), _ptr(block_tables),
                                 block_tables.shape[1], _ptr(start_pos), n_seqs, n_new, _ptr(dev_status),
                                 _stream(stream))
    _check("paged_kv_write_rope", st)
    return q_out


class WindowDecodePlan:
    """paged_decode_attention_window / paged_decode_step_window with the arguments
    that stay the same from call to call checked once, as DecodePlan does for the
    unwindowed calls (and with the same conditions on the planned tensors).  No
    workspace is needed.  ``run(q)`` attends; ``run(q, k_new, v_new, start_pos)``
    is a whole step: turn (where the plan has a rope), page write, attention."""

    def __init__(self, k_pool, v_pool, block_tables, ctx_lens, softmax_scale, n_q_heads, window, sinks=0, rope=None,
                 k_scales=None, v_scales=None, out=None, lse_out=None, dev_status=None):
        dev = _device_of(k_pool, "k_pool")
        self._lib = load_library()
        int8 = _check_paged(k_pool, v_pool, k_scales, v_scales, block_tables, dev)
        _need(ctx_lens, "ctx_lens", torch.int32, 1, dev)
        n_seqs, D = block_tables.shape[0], k_pool.shape[3]
        self.q_shape = torch.Size((n_seqs, int(n_q_heads), D))
        if out is None:
            out = torch.empty(self.q_shape, dtype=torch.bfloat16, device=dev)
        _need(out, "out", torch.bfloat16, 3, dev)
        _shape(out, "out", self.q_shape)
        if lse_out is not None:
            _need(lse_out, "lse_out", torch.float32, 2, dev)
            _shape(lse_out, "lse_out", self.q_shape[:2])
        _check_batch(n_seqs, block_tables, ctx_lens, "ctx_lens")
        _check_status(dev_status, dev)
        self.device, self.out, self.n_q_heads = dev, out, int(n_q_heads)
        self.new_shape = torch.Size((n_seqs, 1) + tuple(k_pool.shape[2:]))
        self._rope = _rope_arg(rope, D, dev)
        # held so that the pointers below stay valid
        self._tensors = (k_pool, v_pool, k_scales, v_scales, block_tables, ctx_lens, out, lse_out, dev_status, rope)
        self._args = (_ptr(k_pool), _ptr(v_pool), _ptr(k_scales), _ptr(v_scales),
                      PKV_KV_INT8 if int8 else PKV_KV_BF16, pool_dims(k_pool), _ptr(block_tables),
                      block_tables.shape[1], _ptr(ctx_lens), n_seqs, float(softmax_scale), _count(window, "window"),
                      _count(sinks, "sinks"), _ptr(out), _ptr(lse_out), _ptr(dev_status))
        self._plan = None
        if _native is not None:
            kp, vp, ks, vs, kind, dims, tab, width, ctx, n, scale, window, sinks, o, lse, st = self._args
            self._plan = _native.make_plan(dev, self.n_q_heads, 0 if rope is None else rope._address, kp, vp, ks or 0,
                                           vs or 0, kind, dims.n_blocks, dims.block_size, dims.n_kv_heads, dims.head_dim,
                                           tab, width, ctx, n, scale, window, sinks, o, lse or 0, st or 0)

    def run(self, q, k_new=None, v_new=None, start_pos=None, stream=None):
        """q [n_seqs, Hq, D] bf16 (contiguous for the attention alone); k_new /
        v_new [n_seqs, 1, Hkv, D]; start_pos [n_seqs].  In a step the three may
        be parts of a fused projection's rows.  Returns the plan's out."""
        if stream is None and self._plan is not None:
            st = _native.run_plan(self._plan, q, k_new, v_new, start_pos)
            if st is not None:
                if st:
                    _check("paged_decode_attention_window" if k_new is None else "paged_decode_step_window", st)
                return self.out
        dev = self.device
        if _elsewhere(dev):
            with torch.cuda.device(dev):
                return self.run(q, k_new, v_new, start_pos, stream)
        if k_new is None:
            if v_new is not None or start_pos is not None:
                raise ValueError("v_new and start_pos come with k_new")
            if self._rope is not None:
                raise ValueError("a plan with a rope runs steps: give k_new, v_new and start_pos")
            _need(q, "q", torch.bfloat16, 3, dev)
            _shape(q, "q", self.q_shape)
            st = self._lib.paged_decode_attention_window(q.data_ptr(), self.n_q_heads, *self._args, _stream(stream))
            _check("paged_decode_attention_window", st)
            return self.out
        qs = _token_stride(q, "q", 3, dev)
        ks, vs = _token_stride(k_new, "k_new", 4, dev), _token_stride(v_new, "v_new", 4, dev)
        _shape(q, "q", self.q_shape)
        _shape(k_new, "k_new", self.new_shape)
        _shape(v_new, "v_new", self.new_shape)
        _need(start_pos, "start_pos", torch.int32, 1, dev)
        _shape(start_pos, "start_pos", self.q_shape[:1])
        st = self._lib.paged_decode_step_window(k_new.data_ptr(), ks, v_new.data_ptr(), vs, start_pos.data_ptr(),
                                                q.data_ptr(), qs, self.n_q_heads, self._rope, *self._args,
                                                _stream(stream))
        _check("paged_decode_step_window", st)
        return self.out


def paged_decode_attention_window(q, k_pool, v_pool, block_tables, ctx_lens, softmax_scale, window, sinks=0,
                                  k_scales=None, v_scales=None, out=None, lse_out=None, dev_status=None, stream=None):
    """paged_decode_attention under a sliding window: the query of sequence s (at
    position ctx_lens[s] - 1) sees the first ``sinks`` tokens and the last
    ``window`` ones.  Blocks that hold none of them are never looked up.  Returns
    out [n_seqs, Hq, D] bf16."""
    dev = _device_of(q, "q")
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    _need(q, "q", torch.bfloat16, 3, dev)
    plan = WindowDecodePlan(k_pool, v_pool, block_tables, ctx_lens, softmax_scale, q.shape[1], window, sinks, None,
                            k_scales, v_scales, out, lse_out, dev_status)
    return plan.run(q, stream=stream)


def paged_decode_step_window(k_new, v_new, start_pos, q, k_pool, v_pool, block_tables, ctx_lens, softmax_scale, window,
                             sinks=0, rope=None, k_scales=None, v_scales=None, out=None, lse_out=None, dev_status=None,
                             stream=None):
    """One layer's step of one token per sequence in one launch: q and k_new
    [n_seqs, 1, Hkv, D] turned at start_pos (rope None: as they are), k_new and
    v_new written to the pages, then paged_decode_attention_window over ctx_lens
    tokens (which count the new one).  Returns out [n_seqs, Hq, D] bf16."""
    dev = _device_of(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q must have 3 dims, got {tuple(q.shape)}")
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    if k_new is None:
        raise TypeError("k_new must be a torch.Tensor")
    plan = WindowDecodePlan(k_pool, v_pool, block_tables, ctx_lens, softmax_scale, q.shape[1], window, sinks, rope,
                            k_scales, v_scales, out, lse_out, dev_status)
    return plan.run(q, k_new, v_new, start_pos, stream=stream)


def paged_prefill_attention_window(q, k_pool, v_pool, block_tables, prefix_lens, softmax_scale, window, sinks=0,
                                   out=None, lse_out=None, dev_status=None, stream=None):
    """paged_prefill_attention under a sliding window: query i of sequence s (at
    position prefix_lens[s] + i) sees the first ``sinks`` tokens and the last
    ``window`` ones up to itself.  Returns out, same shape as q."""
    if stream is None and _native is not None:
        done = _native.prefill_window(q, k_pool, v_pool, block_tables, prefix_lens, softmax_scale, window, sinks, out,
                                      lse_out, dev_status)
        if done is not None:
            if type(done) is int:
                _check("paged_prefill_attention_window", done)
            return done
    dev = _device_of(q, "q")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return paged_prefill_attention_window(q, k_pool, v_pool, block_tables, prefix_lens, softmax_scale, window,
                                                  sinks, out, lse_out, dev_status, stream)
    lib = load_library()
    _need(q, "q", torch.bfloat16, 4, dev)
    _need(k_pool, "k_pool", torch.bfloat16, 4, dev)
    _need(v_pool, "v_pool", torch.bfloat16, 4, dev)
    _check_pools(k_pool, v_pool)
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    _need(prefix_lens, "prefix_lens", torch.int32, 1, dev)
    n_seqs, chunk, n_q_heads, D = q.shape
    if k_pool.shape[3] != D:
        raise ValueError(f"q has head_dim {D}, the pool {k_pool.shape[3]}")
    _check_batch(n_seqs, block_tables, prefix_lens, "prefix_lens")
    _check_status(dev_status, dev)
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    else:
        _need(out, "out", torch.bfloat16, 4, dev)
        _shape(out, "out", q.shape)
    if lse_out is not None:
        _need(lse_out, "lse_out", torch.float32, 3, dev)
        _shape(lse_out, "lse_out", q.shape[:3])
    st = lib.paged_prefill_attention_window(_ptr(q), n_q_heads, _ptr(k_pool), _ptr(v_pool), _dims(k_pool),
                                            _ptr(block_tables), block_tables.shape[1], _ptr(prefix_lens), n_seqs, chunk,
                                            float(softmax_scale), _count(window, "window"), _count(sinks, "sinks"),
                                            _ptr(out), _ptr(lse_out), _ptr(dev_status), _stream(stream))
    _check("paged_prefill_attention_window", st)
    return out


# ---- batches of requests of any lengths ---------------------------------------

class StepMaps(typing.NamedTuple):
    """The maps of a step (paged_step_maps): ctx_lens [n_seqs], token_starts
    [n_seqs + 1], token_seqs and positions [n_tokens], cursor [1] int32, slots
    [n_tokens] int64."""
    ctx_lens: torch.Tensor
    token_starts: torch.Tensor
    token_seqs: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor
    cursor: torch.Tensor

    @classmethod
    def empty(cls, n_seqs, n_tokens, device, stream=None):
        """Uninitialised maps for paged_step_maps to write into."""
        dev = torch.device(device)
        return cls(*(_empty((n,), torch.int64 if i == 4 else torch.int32, dev, stream)
                     for i, n in enumerate((n_seqs, n_seqs + 1, n_tokens, n_tokens, n_tokens, 1))))


def paged_step_maps(lens, n_new, free_blocks, block_tables, block_size, n_blocks, n_tokens, cursor=None, out=None,
                    dev_status=None, stream=None):
    """The block tables and slot maps of a step, built on the device: sequence s
    holds lens[s] tokens and adds n_new[s]; the blocks that it needs for them are
    the next of free_blocks (behind the cursor[0] entries that earlier steps
    have taken) and go into its row of block_tables.  n_tokens: the rows of the
    packed batch, at least sum(n_new).  ``out`` (a StepMaps) is written into;
    lens and ctx_lens, cursor and out.cursor have to be different tensors.
    Returns the StepMaps."""
    if stream is None and _native is not None and type(out) is StepMaps:
        st = _native.step_maps(lens, n_new, free_blocks, block_tables, block_size, n_blocks, n_tokens, cursor, out,
                               dev_status)
        if st is not None:
            if st:
                _check("paged_step_maps", st)
            return out
    dev = _device_of(block_tables, "block_tables")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return paged_step_maps(lens, n_new, free_blocks, block_tables, block_size, n_blocks, n_tokens, cursor, out,
                                   dev_status, stream)
    lib = load_library()
    _need(block_tables, "block_tables", torch.int32, 2, dev)
    n_seqs = block_tables.shape[0]
    for t, name in ((lens, "lens"), (n_new, "n_new")):
        _need(t, name, torch.int32, 1, dev)
        _shape(t, name, (n_seqs,))
    _need(free_blocks, "free_blocks", torch.int32, 1, dev)
    if cursor is not None:
        _need(cursor, "cursor", torch.int32, 1, dev)
        _shape(cursor, "cursor", (1,))
    _check_status(dev_status, dev)
    n_tokens = int(n_tokens)
    if n_tokens < 0:
        raise ValueError(f"n_tokens must not be negative, got {n_tokens}")
    if out is None:
        out = StepMaps.empty(n_seqs, n_tokens, torch.device("cuda", dev), stream)
    elif not isinstance(out, StepMaps):
        raise TypeError("out must be a StepMaps")
    else:
        for name, n in zip(StepMaps._fields, (n_seqs, n_seqs + 1, n_tokens, n_tokens, n_tokens, 1)):
            t = getattr(out, name)
            _need(t, name, torch.int64 if name == "slots" else torch.int32, 1, dev)
            _shape(t, name, (n,))
    st = lib.paged_step_maps(_ptr(lens), _ptr(n_new), n_seqs, _ptr(free_blocks), free_blocks.shape[0], _ptr(cursor),
                             int(n_blocks), int(block_size), _ptr(block_tables), block_tables.shape[1], n_tokens,
                             _ptr(out.ctx_lens), _ptr(out.token_starts), _ptr(out.token_seqs), _ptr(out.positions),
                             _ptr(out.slots), _ptr(out.cursor), _ptr(dev_status), _stream(stream))
    _check("paged_step_maps", st)
    return out


def paged_kv_write_slots(k_new, v_new, k_pool, v_pool, slots, k_scales=None, v_scales=None, dev_status=None,
                         stream=None):
    """Packed rows to their pool rows: row i of k_new / v_new [n_rows, Hkv, D]
    bf16 (they may be parts of a fused projection's rows) goes to pool row
    slots[i] (int64; negative: nowhere), as it is or, into int8 pools, quantised
    with k_scales / v_scales."""
    if stream is None and _native is not None:
        st = _native.write_slots(k_new, v_new, k_pool, v_pool, slots, k_scales, v_scales, dev_status)
        if st is not None:
            if st:
                _check("paged_kv_write_slots", st)
            return
    dev = _device_of(k_pool, "k_pool")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return paged_kv_write_slots(k_new, v_new, k_pool, v_pool, slots, k_scales, v_scales, dev_status, stream)
    lib = load_library()
    int8 = _check_pool_kinds(k_pool, v_pool, k_scales, v_scales, dev)
    ks, vs = _token_stride(k_new, "k_new", 3, dev), _token_stride(v_new, "v_new", 3, dev)
    n_rows = k_new.shape[0]
    _shape(k_new, "k_new", (n_rows,) + tuple(k_pool.shape[2:]))
    _shape(v_new, "v_new", k_new.shape)
    _need(slots, "slots", torch.int64, 1, dev)
    _shape(slots, "slots", (n_rows,))
    _check_status(dev_status, dev)
    st = lib.paged_kv_write_slots(_ptr(k_new), ks, _ptr(v_new), vs, _ptr(k_pool), _ptr(v_pool), _ptr(k_scales),
                                  _ptr(v_scales), PKV_KV_INT8 if int8 else PKV_KV_BF16, _dims(k_pool), _ptr(slots),
                                  n_rows, _ptr(dev_status), _stream(stream))
    _check("paged_kv_write_slots", st)


def rows_workspace_bytes(n_rows, n_q_heads, head_dim) -> int:
    """Device workspace of paged_cross_attention for n_rows packed query rows, and of
    paged_decode_attention_shared for n_rows sequences (pkv_rows_workspace_bytes)."""
    n = load_library().pkv_rows_workspace_bytes(int(n_rows), int(n_q_heads), int(head_dim))
    if n == 0:
        raise ValueError("invalid arguments to pkv_rows_workspace_bytes")
    return int(n)


def _rows_buffers(q, out, lse_out, workspace, dev, stream):
    """out and workspace of a call over packed query rows, made where they are not given."""
    n_rows, n_q_heads, D = q.shape
    if out is None:
        out = _empty(q.shape, torch.bfloat16, dev, stream)
    else:
        _need(out, "out", torch.bfloat16, 3, dev)
        _shape(out, "out", q.shape)
    if lse_out is not None:
        _need(lse_out, "lse_out", torch.float32, 2, dev)
        _shape(lse_out, "lse_out", q.shape[:2])
    if workspace is None:
        workspace = _empty((rows_workspace_bytes(n_rows, n_q_heads, D),), torch.uint8, dev, stream)
    _need(workspace, "workspace", torch.uint8, 1, dev)
    return out, workspace


def paged_cross_attention(q, q_starts, k_pool, v_pool, block_tables, key_lens, softmax_scale, k_scales=None,
                          v_scales=None, out=None, lse_out=None, workspace=None, dev_status=None, stream=None):
    """Attention of packed queries to keys of another length, without a causal
    mask: rows q_starts[s] .. q_starts[s + 1] - 1 of q [n_rows, Hq, D] bf16 (its
    tokens may be a stride apart) see the key_lens[s] tokens of sequence s's
    pages, bf16 or int8 with k_scales / v_scales.  Rows of no sequence are left
    as they were.  ``workspace`` (uint8, rows_workspace_bytes) is allocated when
    not given.  Returns out [n_rows, Hq, D] bf16."""
    if stream is None and _native is not None:
        done = _native.cross(q, q_starts, k_pool, v_pool, block_tables, key_lens, softmax_scale, k_scales, v_scales, out,
                             lse_out, workspace, dev_status)
        if done is not None:
            if type(done) is int:
                _check("paged_cross_attention", done)
            return done
    dev = _device_of(q, "q")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return paged_cross_attention(q, q_starts, k_pool, v_pool, block_tables, key_lens, softmax_scale, k_scales,
                                         v_scales, out, lse_out, workspace, dev_status, stream)
    lib = load_library()
    int8 = _check_paged(k_pool, v_pool, k_scales, v_scales, block_tables, dev)
    qs = _token_stride(q, "q", 3, dev)
    n_rows, n_q_heads, D = q.shape
    if D != k_pool.shape[3]:
        raise ValueError(f"q has head_dim {D}, the pool {k_pool.shape[3]}")
    n_seqs = block_tables.shape[0]
    _need(key_lens, "key_lens", torch.int32, 1, dev)
    _shape(key_lens, "key_lens", (n_seqs,))
    _need(q_starts, "q_starts", torch.int32, 1, dev)
    _shape(q_starts, "q_starts", (n_seqs + 1,))
    _check_status(dev_status, dev)
    out, workspace = _rows_buffers(q, out, lse_out, workspace, dev, stream)
    st = lib.paged_cross_attention(_ptr(q), qs, n_q_heads, _ptr(q_starts), n_rows, _ptr(k_pool), _ptr(v_pool),
                                   _ptr(k_scales), _ptr(v_scales), PKV_KV_INT8 if int8 else PKV_KV_BF16, _dims(k_pool),
                                   _ptr(block_tables), block_tables.shape[1], _ptr(key_lens), n_seqs,
                                   float(softmax_scale), _ptr(out), _ptr(lse_out), _ptr(workspace), workspace.numel(),
                                   _ptr(dev_status), _stream(stream))
    _check("paged_cross_attention", st)
    return out


class SharedDecodePlan:
    """paged_decode_attention_shared with the arguments that stay the same from
    call to call checked once, as DecodePlan does for paged_decode_attention (and
    with the same conditions on the planned tensors; calls of one plan share its
    workspace, so they must not run at once)."""

    def __init__(self, k_pool, v_pool, block_tables, ctx_lens, group_starts, prefix_tables, prefix_lens, softmax_scale,
                 n_q_heads, k_scales=None, v_scales=None, out=None, lse_out=None, workspace=None, dev_status=None):
        dev = _device_of(k_pool, "k_pool")
        self._lib = load_library()
        int8 = _check_paged(k_pool, v_pool, k_scales, v_scales, block_tables, dev)
        n_seqs, D = block_tables.shape[0], k_pool.shape[3]
        _need(ctx_lens, "ctx_lens", torch.int32, 1, dev)
        _check_batch(n_seqs, block_tables, ctx_lens, "ctx_lens")
        _need(prefix_tables, "prefix_tables", torch.int32, 2, dev)
        _need(prefix_lens, "prefix_lens", torch.int32, 1, dev)
        _need(group_starts, "group_starts", torch.int32, 1, dev)
        n_groups = prefix_tables.shape[0]
        _shape(prefix_lens, "prefix_lens", (n_groups,))
        _shape(group_starts, "group_starts", (n_groups + 1,))
        self.q_shape = torch.Size((n_seqs, int(n_q_heads), D))
        if out is None:
            out = torch.empty(self.q_shape, dtype=torch.bfloat16, device=dev)
        _need(out, "out", torch.bfloat16, 3, dev)
        _shape(out, "out", self.q_shape)
        if lse_out is not None:
            _need(lse_out, "lse_out", torch.float32, 2, dev)
            _shape(lse_out, "lse_out", self.q_shape[:2])
        if workspace is None:
            workspace = torch.empty(rows_workspace_bytes(n_seqs, n_q_heads, D), dtype=torch.uint8, device=dev)
        _need(workspace, "workspace", torch.uint8, 1, dev)
        _check_status(dev_status, dev)
        self.device, self.out, self.n_q_heads = dev, out, int(n_q_heads)
        # held so that the pointers below stay valid
        self._tensors = (k_pool, v_pool, k_scales, v_scales, block_tables, ctx_lens, group_starts, prefix_tables,
                         prefix_lens, out, lse_out, workspace, dev_status)
        self._args = (_ptr(k_pool), _ptr(v_pool), _ptr(k_scales), _ptr(v_scales), PKV_KV_INT8 if int8 else PKV_KV_BF16,
                      pool_dims(k_pool), _ptr(block_tables), block_tables.shape[1], _ptr(ctx_lens), n_seqs,
                      _ptr(group_starts), n_groups, _ptr(prefix_tables), prefix_tables.shape[1], _ptr(prefix_lens),
                      float(softmax_scale), _ptr(out), _ptr(lse_out), _ptr(workspace), workspace.numel(),
                      _ptr(dev_status))
        self._plan = None
        if _native is not None:
            kp, vp, ks, vs, kind, dims, tab, width, ctx, n, gs, ng, pt, pw, pl, scale, o, lse, ws, wsb, st = self._args
            self._plan = _native.make_shared_plan(dev, self.n_q_heads, kp, vp, ks or 0, vs or 0, kind, dims.n_blocks,
                                                  dims.block_size, dims.n_kv_heads, dims.head_dim, tab, width, ctx, n, gs,
                                                  ng, pt, pw, pl, scale, o, lse or 0, ws, wsb, st or 0)

    def run(self, q, stream=None):
        """q [n_seqs, Hq, D] bf16 (its tokens may be a stride apart).  Returns the plan's out."""
        if stream is None and self._plan is not None:
            st = _native.run_shared_plan(self._plan, q)
            if st is not None:
                if st:
                    _check("paged_decode_attention_shared", st)
                return self.out
        dev = self.device
        if _elsewhere(dev):
            with torch.cuda.device(dev):
                return self.run(q, stream)
        qs = _token_stride(q, "q", 3, dev)
        _shape(q, "q", self.q_shape)
        st = self._lib.paged_decode_attention_shared(q.data_ptr(), qs, self.n_q_heads, *self._args, _stream(stream))
        _check("paged_decode_attention_shared", st)
        return self.out


def paged_decode_attention_shared(q, k_pool, v_pool, block_tables, ctx_lens, group_starts, prefix_tables, prefix_lens,
                                  softmax_scale, k_scales=None, v_scales=None, out=None, lse_out=None, workspace=None,
                                  dev_status=None, stream=None):
    """paged_decode_attention for groups of sequences that share their first tokens:
    sequences group_starts[g] .. group_starts[g + 1] - 1 see the prefix_lens[g]
    tokens of prefix_tables[g], read once for all of them, and each goes on at
    that position in its own row of block_tables (entries of blocks wholly within
    the prefix are not read).  Returns out [n_seqs, Hq, D] bf16."""
    dev = _device_of(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q must have 3 dims, got {tuple(q.shape)}")
    out, workspace = _rows_buffers(q, out, lse_out, workspace, dev, stream)
    plan = SharedDecodePlan(k_pool, v_pool, block_tables, ctx_lens, group_starts, prefix_tables, prefix_lens,
                            softmax_scale, q.shape[1], k_scales, v_scales, out, lse_out, workspace, dev_status)
    return plan.run(q, stream=stream)


class BlockManager:
    """The library's host-side block manager (include/pagedkv_blocks.h): free
    stack and reference counts of n_blocks blocks, n_slots sequence slots with
    tables of max_blocks entries.  Methods mirror the C calls; failures raise
    PagedKVError (nothing changed)."""

    def __init__(self, n_blocks, block_size, n_slots, max_blocks):
        self._lib = load_library()
        h = ctypes.c_void_p()
        _check("pkv_bm_create", self._lib.pkv_bm_create(int(n_blocks), int(block_size), int(n_slots),
                                                          int(max_blocks), ctypes.byref(h)))
        self._h = h
        self.n_blocks, self.block_size, self.n_slots, self.max_blocks = n_blocks, block_size, n_slots, max_blocks

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._lib.pkv_bm_destroy(h)
            self._h = None

    def _call(self, fn, *args):
        _check(fn, getattr(self._lib, fn)(self._h, *args))

    @staticmethod
    def _ints(values):
        arr = (ctypes.c_int32 * max(1, len(values)))(*values)
        return arr

    def alloc(self) -> int:
        b = ctypes.c_int32()
        self._call("pkv_bm_alloc", ctypes.byref(b))
        return b.value

    def free(self, blocks):
        self._call("pkv_bm_free", self._ints(list(blocks)), len(blocks))

    @property
    def num_free(self) -> int:
        return self._lib.pkv_bm_num_free(self._h)

    @property
    def peak_used(self) -> int:
        return self._lib.pkv_bm_peak_used(self._h)

    def refcount(self, block) -> int:
        return self._lib.pkv_bm_refcount(self._h, int(block))

    def can_admit(self, lengths) -> bool:
        ok = ctypes.c_int32()
        self._call("pkv_bm_can_admit", self._ints(list(lengths)), len(lengths), ctypes.byref(ok))
        return bool(ok.value)

    def admit(self, slot, n_tokens):
        self._call("pkv_bm_admit", int(slot), int(n_tokens))

    def release(self, slot):
        self._call("pkv_bm_release", int(slot))

    def fork(self, src_slot, dst_slot):
        self._call("pkv_bm_fork", int(src_slot), int(dst_slot))

    def reserve_step(self):
        victims = (ctypes.c_int32 * self.n_slots)()
        n = ctypes.c_int32()
        self._call("pkv_bm_reserve_step", victims, ctypes.byref(n))
        return list(victims[:n.value])

    def begin_step(self):
        copies = (ctypes.c_int32 * (2 * self.n_slots))()
        n = ctypes.c_int32()
        self._call("pkv_bm_begin_step", copies, ctypes.byref(n))
        return [(copies[2 * i], copies[2 * i + 1]) for i in range(n.value)]

    def end_step(self):
        self._call("pkv_bm_end_step")

    def export(self):
        """(tables [n_slots][max_blocks], lens [n_slots], active [n_slots]) as int32 CPU tensors."""
        tables = torch.empty((self.n_slots, self.max_blocks), dtype=torch.int32)
        lens = torch.empty(self.n_slots, dtype=torch.int32)
        active = torch.empty(self.n_slots, dtype=torch.int32)
        self._call("pkv_bm_export", ctypes.c_void_p(tables.data_ptr()), ctypes.c_void_p(lens.data_ptr()),
                   ctypes.c_void_p(active.data_ptr()))
        return tables, lens, active


class ScratchPool:
    """Residency of a device scratch pool of n_slots blocks for decode streamed
    from a host tier (include/pagedkv_stream.h)."""

    def __init__(self, n_slots, max_seqs):
        self._lib = load_library()
        h = ctypes.c_void_p()
        _check("pkv_sp_create", self._lib.pkv_sp_create(int(n_slots), int(max_seqs), ctypes.byref(h)))
        self._h = h
        self.n_slots, self.max_seqs = int(n_slots), int(max_seqs)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._lib.pkv_sp_destroy(h)
            self._h = None

    def lookup(self, host_block) -> int:
        return self._lib.pkv_sp_lookup(self._h, int(host_block))

    def invalidate(self, host_block):
        _check("pkv_sp_invalidate", self._lib.pkv_sp_invalidate(self._h, int(host_block)))

    def plan_tile(self, host_tables, ctx_lens, block_size, cursor, tile_blocks=0):
        """Plan the next tile of at most tile_blocks blocks (0: n_slots) from host
        int32 tensors; returns (tile_tables, tile_lens, pairs list, done) and
        advances cursor (a 2-element list)."""
        host_tables = host_tables.to(torch.int32).contiguous()
        ctx_lens = ctx_lens.to(torch.int32).contiguous()
        n_seqs = ctx_lens.shape[0]
        cap = self.n_slots if tile_blocks <= 0 or tile_blocks > self.n_slots else int(tile_blocks)
        tt = torch.empty((n_seqs, min(cap, host_tables.shape[1])), dtype=torch.int32)
        tl = torch.empty(n_seqs, dtype=torch.int32)
        pr = torch.empty((self.n_slots, 2), dtype=torch.int32)
        cur = (ctypes.c_int32 * 2)(*cursor)
        n, done = ctypes.c_int32(), ctypes.c_int32()
        _check("pkv_sp_plan_tile", self._lib.pkv_sp_plan_tile(
            self._h, ctypes.c_void_p(host_tables.data_ptr()), host_tables.shape[1],
            ctypes.c_void_p(ctx_lens.data_ptr()), n_seqs, int(block_size), int(tile_blocks), cur,
            ctypes.c_void_p(tt.data_ptr()),
            ctypes.c_void_p(tl.data_ptr()), ctypes.c_void_p(pr.data_ptr()), ctypes.byref(n), ctypes.byref(done)))
        cursor[0], cursor[1] = cur[0], cur[1]
        return tt, tl, [tuple(x) for x in pr[:n.value].tolist()], bool(done.value)


def paged_kv_stage_blocks(pairs, host_k, host_v, pool_k, pool_v, dev_status=None, stream=None):
    """Copy host-tier blocks (pinned CPU tensors [n_host_blocks, bs, Hkv, D]
    bf16) into scratch-pool slots (device [n_slots + 1, bs, Hkv, D]):
    pairs int32 [n, 2] (host block, slot) on the device."""
    lib = load_library()
    dev = _device_of(pool_k, "pool_k")
    _need(pairs, "pairs", torch.int32, 2, dev)
    for t, n in ((host_k, "host_k"), (host_v, "host_v")):
        if t.device.type != "cpu" or t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous bf16 CPU tensor [n_host_blocks, bs, Hkv, D]")
    _need(pool_k, "pool_k", torch.bfloat16, 4, dev)
    _need(pool_v, "pool_v", torch.bfloat16, 4, dev)
    _check_status(dev_status, dev)
    _check_pools(pool_k, pool_v)
    if pairs.shape[1] != 2:
        raise ValueError(f"pairs must be [n, 2], got {tuple(pairs.shape)}")
    if tuple(host_k.shape[1:]) != tuple(pool_k.shape[1:]) or host_v.shape != host_k.shape:
        raise ValueError("host_k / host_v blocks must match the scratch pool's [bs, Hkv, D]")
    st = lib.paged_kv_stage_blocks(_ptr(pairs), pairs.shape[0], ctypes.c_void_p(host_k.data_ptr()),
                                   ctypes.c_void_p(host_v.data_ptr()), host_k.shape[0], _ptr(pool_k), _ptr(pool_v),
                                   _dims(pool_k), _ptr(dev_status), _stream(stream))
    _check("paged_kv_stage_blocks", st)


def streamed_workspace_bytes(n_seqs, n_q_heads, head_dim, n_slots, block_size) -> int:
    """Device workspace paged_decode_streamed needs (pkv_streamed_workspace_bytes)."""
    n = load_library().pkv_streamed_workspace_bytes(int(n_seqs), int(n_q_heads), int(head_dim), int(n_slots),
                                                    int(block_size))
    if n == 0:
        raise ValueError("invalid arguments to pkv_streamed_workspace_bytes")
    return int(n)


def paged_decode_streamed(q, host_k, host_v, pool_k, pool_v, scratch_pool, host_tables, ctx_lens, softmax_scale,
                          out=None, lse_out=None, workspace=None, dev_status=None, stream=None):
    """Decode attention over blocks in a host tier (pinned CPU tensors), streamed
    through the device scratch pool (pool_k/pool_v [n_slots + 1, bs, Hkv, D]) one
    tile of at most n_slots blocks at a time.  host_tables / ctx_lens: int32 CPU
    tensors.  Returns out (bf16 [n_seqs, Hq, D])."""
    lib = load_library()
    dev = _device_of(q, "q")
    _need(q, "q", torch.bfloat16, 3, dev)
    _need(pool_k, "pool_k", torch.bfloat16, 4, dev)
    _need(pool_v, "pool_v", torch.bfloat16, 4, dev)
    for t, n in ((host_k, "host_k"), (host_v, "host_v")):
        if t.device.type != "cpu" or t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous bf16 CPU tensor [n_host_blocks, bs, Hkv, D]")
    host_tables = host_tables.to(torch.int32).contiguous()
    ctx_lens = ctx_lens.to(torch.int32).contiguous()
    if host_tables.device.type != "cpu" or ctx_lens.device.type != "cpu":
        raise ValueError("host_tables and ctx_lens are host (CPU) tensors")
    n_seqs, n_q_heads, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 3, dev)
    if lse_out is not None:
        _need(lse_out, "lse_out", torch.float32, 2, dev)
    _check_status(dev_status, dev)
    _check_pools(pool_k, pool_v)
    if tuple(host_k.shape[1:]) != tuple(pool_k.shape[1:]) or host_v.shape != host_k.shape:
        raise ValueError("host_k / host_v blocks must match the scratch pool's [bs, Hkv, D]")
    if pool_k.shape[3] != D:
        raise ValueError(f"q has head_dim {D}, the pool {pool_k.shape[3]}")
    _check_batch(n_seqs, host_tables, ctx_lens, "ctx_lens")
    _shape(out, "out", q.shape)
    _shape(lse_out, "lse_out", (n_seqs, n_q_heads))
    if workspace is None:
        workspace = torch.empty(streamed_workspace_bytes(n_seqs, n_q_heads, D, pool_k.shape[0] - 1,
                                                         pool_k.shape[1]), dtype=torch.uint8, device=dev)
    st = lib.paged_decode_streamed(
        _ptr(q), n_q_heads, ctypes.c_void_p(host_k.data_ptr()), ctypes.c_void_p(host_v.data_ptr()),
        host_k.shape[0], _ptr(pool_k), _ptr(pool_v), _dims(pool_k), scratch_pool._h,
        ctypes.c_void_p(host_tables.data_ptr()), host_tables.shape[1], ctypes.c_void_p(ctx_lens.data_ptr()), n_seqs,
        float(softmax_scale), _ptr(out), _ptr(lse_out), _ptr(workspace), workspace.numel(), _ptr(dev_status),
        _stream(stream))
    _check("paged_decode_streamed", st)
    return out
