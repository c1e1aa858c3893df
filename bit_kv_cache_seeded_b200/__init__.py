"""Python binding of the kvq C ABI (include/kvq.h): argument marshalling only.

Every step of the hot path -- rotation, Lloyd-Max coding, QJL sketch, packing, decode
attention, split reduce -- runs in the CUDA kernels of ``libkvq.so``. This module loads that
library (built in-tree by ``bit_kv_cache_seeded_b200.build``) and raises if it is missing or
if no CUDA device is present when a call needs one; there is no fallback path.

The C functions are exposed under their own names (``kvq_cache_bytes``, ``kvq_cache_init``,
``kvq_quantize``, ``kvq_workspace_bytes``, ``kvq_decode_attention``, ...), taking torch
tensors for device buffers. ``KvqCache`` bundles the arena, the host handle and the
workspace for convenience.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkvq.so")

KVQ_OK = 0
STATUS_NAMES = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARG", 2: "KVQ_ERR_UNSUPPORTED",
                3: "KVQ_ERR_CAPACITY", 4: "KVQ_ERR_ALIGNMENT", 5: "KVQ_ERR_WORKSPACE",
                6: "KVQ_ERR_CUDA"}
MODES = {"lm_qjl": 0, "lm": 1, "sign1": 2, "fp4": 3, "kivi": 4}
DTYPES = {torch.float32: 0, torch.bfloat16: 1}

# Every symbol include/kvq.h declares.
EXPORTS = ("kvq_status_str", "kvq_cache_bytes", "kvq_packed_bytes_per_token", "kvq_cache_init",
           "kvq_quantize", "kvq_workspace_bytes", "kvq_decode_attention", "kvq_cache_lengths",
           "kvq_cache_layout", "kvq_lloyd_max_table", "kvq_cache_destroy",
           "kvq_debug_quantize_rotated", "kvq_decode_attention_static", "kvq_kernel_launches",
           "kvq_cache_status", "kvq_debug_decode_unset_wait", "kvq_debug_decode_timed", "kvq_decode_step",
           "kvq_step_staging_bytes", "kvq_decode_step_host", "kvq_draw_rotation_signs", "kvq_draw_qjl_matrix",
           "kvq_partial_floats", "kvq_decode_partials", "kvq_combine_partials",
           "kvq_cache_bytes_paged", "kvq_cache_init_paged", "kvq_extend_block_table", "kvq_slot_map",
           "kvq_quantize_slots", "kvq_quantize_slots_rows", "kvq_cache_set_lengths", "kvq_chunk_workspace_bytes", "kvq_chunk_attention",
           "kvq_chunk_attention_held")
KVQ_STATUS_WAIT_TIMEOUT = 1


class KvqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


class kvq_cfg(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("k_mode", ctypes.c_int32),
                ("v_mode", ctypes.c_int32), ("k_bits", ctypes.c_int32),
                ("v_bits", ctypes.c_int32), ("qjl_dim", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("latent_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("rot_per_head", ctypes.c_int32),
                ("rot_seed", ctypes.c_uint64), ("qjl_seed", ctypes.c_uint64),
                ("sink_tokens", ctypes.c_int32), ("recent_tokens", ctypes.c_int32)]


_lib = None


def load() -> ctypes.CDLL:
    """Load libkvq.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise OSError(f"{LIB_PATH} not built: run `python -m bit_kv_cache_seeded_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, SZ, VP = ctypes.POINTER, ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p
    sig = {
        "kvq_status_str": ([I32], ctypes.c_char_p),
        "kvq_cache_bytes": ([P(kvq_cfg), I32, I32, P(SZ)], I32),
        "kvq_packed_bytes_per_token": ([P(kvq_cfg), P(SZ)], I32),
        "kvq_cache_init": ([P(VP), P(kvq_cfg), I32, I32, VP, SZ, VP, VP, VP], I32),
        "kvq_quantize": ([VP, VP, VP, I32, I32, VP, I32, VP], I32),
        "kvq_workspace_bytes": ([VP, P(SZ)], I32),
        "kvq_decode_attention": ([VP, VP, I32, VP, VP, SZ, VP], I32),
        "kvq_cache_lengths": ([VP, VP], I32),
        "kvq_cache_layout": ([VP, VP, I32], I32),
        "kvq_lloyd_max_table": ([I32, VP, VP], I32),
        "kvq_cache_destroy": ([VP], None),
        "kvq_debug_quantize_rotated": ([VP, VP, I32, VP, VP, VP, VP], I32),
        "kvq_decode_attention_static": ([VP, VP, I32, VP, VP], I32),
        "kvq_kernel_launches": ([], ctypes.c_uint64),
        "kvq_cache_status": ([VP, VP, VP], I32),
        "kvq_debug_decode_unset_wait": ([VP, VP, I32, VP, VP, SZ, ctypes.c_int64, VP], I32),
        "kvq_debug_decode_timed": ([VP, VP, I32, VP, VP, SZ, VP, VP], I32),
        "kvq_decode_step": ([VP, VP, VP, VP, I32, VP, VP, SZ, VP], I32),
        "kvq_step_staging_bytes": ([VP, I32, P(SZ)], I32),
        "kvq_decode_step_host": ([VP, VP, VP, VP, I32, VP, VP, SZ, VP, SZ, VP, VP], I32),
        "kvq_draw_rotation_signs": ([ctypes.c_uint64, I32, VP], I32),
        "kvq_draw_qjl_matrix": ([ctypes.c_uint64, I32, I32, VP], I32),
        "kvq_partial_floats": ([VP, P(I32)], I32),
        "kvq_cache_bytes_paged": ([P(kvq_cfg), I32, I32, P(SZ)], I32),
        "kvq_cache_init_paged": ([P(VP), P(kvq_cfg), I32, I32, I32, VP, VP, SZ, VP, VP, VP], I32),
        "kvq_decode_partials": ([VP, VP, I32, VP, VP, SZ, VP], I32),
        "kvq_combine_partials": ([VP, I32, I32, I32, I32, VP, VP], I32),
        "kvq_extend_block_table": ([VP, VP, I32, VP, I32, VP, VP, I32, VP, VP, VP, VP], I32),
        "kvq_slot_map": ([VP, VP, VP, I32, VP, I32, I32, I32, VP, VP, VP, VP], I32),
        "kvq_quantize_slots": ([VP, VP, VP, I32, VP, I32, VP], I32),
        "kvq_quantize_slots_rows": ([VP, VP, VP, I32, VP, I32, VP, VP], I32),
        "kvq_cache_set_lengths": ([VP, VP, VP], I32),
        "kvq_chunk_workspace_bytes": ([VP, I32, I32, P(SZ)], I32),
        "kvq_chunk_attention": ([VP, VP, I32, I32, VP, VP, VP, VP, SZ, VP], I32),
        "kvq_chunk_attention_held": ([VP, VP, I32, I32, VP, VP, VP, VP, VP, SZ, VP], I32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != KVQ_OK:
        raise KvqError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _on_device(fn: str, **tensors):
    """Device entry points take device pointers: a host tensor would reach a kernel as an address
    it cannot read, so refuse it here."""
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{fn}: {name} must be a CUDA tensor")


def _stream(stream=None):
    if stream is None:  # torch.cuda.current_stream().cuda_stream without the object: 0.3 us instead of 3.4
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _memory_of(stream):
    """What is allocated inside is `stream`'s memory (None: the current one's). A tensor that a call on `stream` writes
    must not come from another stream's: its memory may be in use there by work that `stream` does not wait for."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def make_cfg(head_dim=128, n_q_heads=1, n_kv_heads=1, k_mode="lm_qjl", v_mode="lm_qjl", k_bits=2,
             v_bits=2, qjl_dim=128, softmax_scale=0.0, latent_dim=0, rope_dim=0, rot_per_head=0,
             rot_seed=0, qjl_seed=0, sink_tokens=0, recent_tokens=0) -> kvq_cfg:
    return kvq_cfg(head_dim, n_q_heads, n_kv_heads, MODES[k_mode], MODES[v_mode], k_bits, v_bits,
                   qjl_dim, softmax_scale, latent_dim, rope_dim, int(rot_per_head), rot_seed, qjl_seed,
                   sink_tokens, recent_tokens)


def cfg_for_workload(w) -> kvq_cfg:
    """kvq_cfg of a kvq_inputs.Workload (its seeds included)."""
    if w.k_mode == "fp4":
        return make_cfg(head_dim=w.latent_dim, n_q_heads=w.n_q_heads, n_kv_heads=1, k_mode="fp4",
                        v_mode="fp4", k_bits=4, v_bits=4, qjl_dim=0, latent_dim=w.latent_dim,
                        rope_dim=w.rope_dim)
    return make_cfg(w.head_dim, w.n_q_heads, w.n_kv_heads, w.k_mode, w.v_mode, w.k_bits, w.v_bits,
                    w.qjl_dim, rot_per_head=int(getattr(w, "rot_per_head", False)), rot_seed=w.rot_seed,
                    qjl_seed=w.qjl_seed, sink_tokens=getattr(w, "sink_tokens", 0),
                    recent_tokens=getattr(w, "recent_tokens", 0))


def kvq_draw_rotation_signs(seed: int, n: int) -> np.ndarray:
    """The library's seeded +-1 draws (int8 [n]), as kvq_cache_init makes them from a seed."""
    out = np.zeros(n, dtype=np.int8)
    _check("kvq_draw_rotation_signs", load().kvq_draw_rotation_signs(seed, n, out.ctypes.data_as(ctypes.c_void_p)))
    return out


def kvq_draw_qjl_matrix(seed: int, m: int, d: int) -> np.ndarray:
    """The library's seeded Gaussian sketch matrix (float32 [m, d])."""
    out = np.zeros((m, d), dtype=np.float32)
    _check("kvq_draw_qjl_matrix", load().kvq_draw_qjl_matrix(seed, m, d, out.ctypes.data_as(ctypes.c_void_p)))
    return out


# ---------------------------------------------------------------- same-name wrappers

def kvq_status_str(status: int) -> str:
    return load().kvq_status_str(status).decode()


def kvq_cache_bytes(cfg: kvq_cfg, batch: int, capacity: int) -> int:
    out = ctypes.c_size_t()
    _check("kvq_cache_bytes", load().kvq_cache_bytes(ctypes.byref(cfg), batch, capacity, ctypes.byref(out)))
    return out.value


def kvq_packed_bytes_per_token(cfg: kvq_cfg) -> int:
    out = ctypes.c_size_t()
    _check("kvq_packed_bytes_per_token", load().kvq_packed_bytes_per_token(ctypes.byref(cfg), ctypes.byref(out)))
    return out.value


def kvq_cache_init(cfg: kvq_cfg, batch: int, capacity: int, arena: torch.Tensor, rot_signs=None,
                   qjl_matrix=None, stream=None) -> ctypes.c_void_p:
    _on_device("kvq_cache_init", arena=arena)
    handle = ctypes.c_void_p()
    signs = None if rot_signs is None else np.ascontiguousarray(rot_signs, dtype=np.int8)
    S = None if qjl_matrix is None else np.ascontiguousarray(qjl_matrix, dtype=np.float32)
    st = load().kvq_cache_init(ctypes.byref(handle), ctypes.byref(cfg), batch, capacity, _ptr(arena),
                               arena.numel() * arena.element_size(),
                               None if signs is None else signs.ctypes.data_as(ctypes.c_void_p),
                               None if S is None else S.ctypes.data_as(ctypes.c_void_p), _stream(stream))
    _check("kvq_cache_init", st)
    return handle


def kvq_cache_bytes_paged(cfg: kvq_cfg, batch: int, n_pages: int) -> int:
    out = ctypes.c_size_t()
    _check("kvq_cache_bytes_paged", load().kvq_cache_bytes_paged(ctypes.byref(cfg), batch, n_pages, ctypes.byref(out)))
    return out.value


def kvq_cache_init_paged(cfg: kvq_cfg, batch: int, n_pages: int, block_table: torch.Tensor, arena: torch.Tensor,
                         rot_signs=None, qjl_matrix=None, stream=None) -> ctypes.c_void_p:
    """A paged cache: block_table int32 CUDA tensor [batch, pages_per_seq] (the caller keeps it)."""
    _on_device("kvq_cache_init_paged", arena=arena, block_table=block_table)
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != batch \
            or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 [batch, pages_per_seq] tensor")
    handle = ctypes.c_void_p()
    signs = None if rot_signs is None else np.ascontiguousarray(rot_signs, dtype=np.int8)
    S = None if qjl_matrix is None else np.ascontiguousarray(qjl_matrix, dtype=np.float32)
    st = load().kvq_cache_init_paged(ctypes.byref(handle), ctypes.byref(cfg), batch, block_table.shape[1], n_pages,
                                     _ptr(block_table), _ptr(arena), arena.numel() * arena.element_size(),
                                     None if signs is None else signs.ctypes.data_as(ctypes.c_void_p),
                                     None if S is None else S.ctypes.data_as(ctypes.c_void_p), _stream(stream))
    _check("kvq_cache_init_paged", st)
    return handle


def kvq_quantize(handle, K: torch.Tensor, V: torch.Tensor, seq_ids=None, stream=None):
    _on_device("kvq_quantize", K=K, V=V)
    if K.dtype not in DTYPES or V.dtype != K.dtype:
        raise TypeError("K and V must both be float32 or bfloat16")
    if not (K.is_contiguous() and V.is_contiguous()):
        raise ValueError("K and V must be contiguous")
    n_seq = K.shape[0]
    n_new = K.shape[-2]
    ids = None
    if seq_ids is not None:
        ids = np.ascontiguousarray(seq_ids, dtype=np.int32)
        if ids.shape[0] != n_seq:
            raise ValueError("seq_ids length must match K.shape[0]")
    st = load().kvq_quantize(handle, _ptr(K), _ptr(V), DTYPES[K.dtype], n_new,
                             None if ids is None else ids.ctypes.data_as(ctypes.c_void_p), n_seq,
                             _stream(stream))
    _check("kvq_quantize", st)


def kvq_workspace_bytes(handle) -> int:
    out = ctypes.c_size_t()
    _check("kvq_workspace_bytes", load().kvq_workspace_bytes(handle, ctypes.byref(out)))
    return out.value


def kvq_decode_attention(handle, q: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                         stream=None):
    _on_device("kvq_decode_attention", q=q, out=out, workspace=workspace)
    if q.dtype not in DTYPES or out.dtype != torch.float32:
        raise TypeError("q must be float32/bfloat16 and out float32")
    if not (q.is_contiguous() and out.is_contiguous()):
        raise ValueError("q and out must be contiguous")
    st = load().kvq_decode_attention(handle, _ptr(q), DTYPES[q.dtype], _ptr(out), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream))
    _check("kvq_decode_attention", st)


def kvq_partial_floats(handle) -> int:
    n = ctypes.c_int32(0)
    _check("kvq_partial_floats", load().kvq_partial_floats(handle, ctypes.byref(n)))
    return int(n.value)


def kvq_decode_partials(handle, q: torch.Tensor, partials: torch.Tensor, workspace: torch.Tensor, stream=None):
    """Softmax state of this cache's tokens: partials [batch, n_q_heads, 2 + dv] float32 (m, l, o)."""
    _on_device("kvq_decode_partials", q=q, partials=partials, workspace=workspace)
    if q.dtype not in DTYPES or partials.dtype != torch.float32:
        raise TypeError("q must be float32/bfloat16 and partials float32")
    if not (q.is_contiguous() and partials.is_contiguous()):
        raise ValueError("q and partials must be contiguous")
    st = load().kvq_decode_partials(handle, _ptr(q), DTYPES[q.dtype], _ptr(partials), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    _check("kvq_decode_partials", st)


def kvq_combine_partials(partials: torch.Tensor, out: torch.Tensor, stream=None):
    """Merge partials [n_parts, batch, n_q_heads, 2 + dv] into out [batch, n_q_heads, dv]."""
    _on_device("kvq_combine_partials", partials=partials, out=out)
    if partials.dtype != torch.float32 or out.dtype != torch.float32:
        raise TypeError("partials and out must be float32")
    if partials.dim() != 4 or out.dim() != 3 or tuple(partials.shape[1:3]) != tuple(out.shape[:2]) \
            or partials.shape[3] != out.shape[2] + 2:
        raise ValueError("partials must be [n_parts, batch, n_q_heads, 2 + dv] for out [batch, n_q_heads, dv]")
    if not (partials.is_contiguous() and out.is_contiguous()):
        raise ValueError("partials and out must be contiguous")
    n, B, H, S = partials.shape
    _check("kvq_combine_partials", load().kvq_combine_partials(_ptr(partials), n, B, H, S - 2, _ptr(out),
                                                               _stream(stream)))


def kvq_decode_step(handle, K: torch.Tensor, V: torch.Tensor, q: torch.Tensor, out: torch.Tensor,
                    workspace: torch.Tensor, stream=None):
    """Append one token per sequence (K, V [B, Hkv, 1, d]; FP4: latent, rope) and decode with q."""
    _on_device("kvq_decode_step", K=K, V=V, q=q, out=out, workspace=workspace)
    if K.dtype != V.dtype or K.dtype != q.dtype or q.dtype not in DTYPES or out.dtype != torch.float32:
        raise TypeError("K, V and q must share float32/bfloat16; out is float32")
    if not (K.is_contiguous() and V.is_contiguous() and q.is_contiguous() and out.is_contiguous()):
        raise ValueError("K, V, q and out must be contiguous")
    if K.shape[-2] != 1 or V.shape[-2] != 1:
        raise ValueError("a decode step appends exactly one token per sequence")
    st = load().kvq_decode_step(handle, _ptr(K), _ptr(V), _ptr(q), DTYPES[q.dtype], _ptr(out), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream))
    _check("kvq_decode_step", st)


def kvq_step_staging_bytes(handle, dtype) -> int:
    n = ctypes.c_size_t(0)
    _check("kvq_step_staging_bytes", load().kvq_step_staging_bytes(handle, DTYPES[dtype], ctypes.byref(n)))
    return n.value


def kvq_decode_step_host(handle, K: torch.Tensor, V: torch.Tensor, q: torch.Tensor, dtype, out: torch.Tensor,
                         staging: torch.Tensor, workspace: torch.Tensor, stream=None, out_event=None):
    """kvq_decode_step from host memory: K, V, q and out are CPU tensors (pinned for asynchronous
    copies) holding the bytes of the layouts kvq_decode_step takes, inputs of type `dtype`. Without
    out_event, out is valid once the stream reaches the end of the call's work; with a
    torch.cuda.Event, the library records it after the output copy (on its own copy stream) and the
    stream does not wait: out is valid once the event has completed. The sizes are the caller's to
    get right (KvqCache.step_host checks them)."""
    for t in (K, V, q, out):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("kvq_decode_step_host takes contiguous host tensors")
    ev = None
    if out_event is not None:
        if out_event.cuda_event == 0:  # torch creates the event lazily, on its first record
            out_event.record()
        ev = ctypes.c_void_p(out_event.cuda_event)
    st = load().kvq_decode_step_host(handle, _ptr(K), _ptr(V), _ptr(q), DTYPES[dtype], _ptr(out), _ptr(staging),
                                     staging.numel() * staging.element_size(), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream), ev)
    _check("kvq_decode_step_host", st)
    return out


# ---- ragged serving path

def _here(fn: str, dtype=None, **tensors):
    """Contiguous CUDA tensors, of one type if dtype is given, on the current device (the calls launch there).
    A call of the ragged path takes a few microseconds on the device: one pass over its tensors."""
    here = -1
    for name, t in tensors.items():
        if t is None:
            continue
        at = t.get_device()
        if at < 0:
            raise ValueError(f"{fn}: {name} must be a CUDA tensor")
        if dtype is not None and t.dtype is not dtype:
            raise TypeError(f"{fn}: {name} must be {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be contiguous")
        if here < 0:
            here = torch.cuda.current_device()
        if at != here:
            raise ValueError(f"{fn}: {name} is on {t.device}, not on the current device")


# Counts that the library takes as int32 are compared with this (in place: a call takes a few microseconds); ctypes would
# cut larger ones down to 32 bits without a word.
INT32_MAX = 2**31 - 1


def _too_many(fn: str):
    return ValueError(f"{fn}: a count that does not fit 32 bits")


def kvq_extend_block_table(held: torch.Tensor, n_new: torch.Tensor, free_pages: torch.Tensor, block_table: torch.Tensor,
                           seq_start: torch.Tensor, ctx_lens: torch.Tensor, taken: torch.Tensor, cursor=None, stream=None):
    """Give pages to n_new [batch] new tokens of requests holding held [batch]: writes block_table [batch,
    pages_per_seq] from free_pages [n_free] (starting at cursor [1]), seq_start [batch + 1], ctx_lens [batch]
    and taken [2] (pages given, requests refused). All int32 CUDA tensors."""
    fn = "kvq_extend_block_table"
    _here(fn, torch.int32, held=held, n_new=n_new, free_pages=free_pages, block_table=block_table, seq_start=seq_start,
          ctx_lens=ctx_lens, taken=taken, cursor=cursor)
    B, shape = held.numel(), block_table.shape
    if len(shape) != 2 or shape[0] != B or n_new.numel() != B or seq_start.numel() != B + 1 \
            or ctx_lens.numel() != B or taken.numel() != 2 or (cursor is not None and cursor.numel() != 1):
        raise ValueError(f"{fn}: held, n_new, ctx_lens [batch], seq_start [batch + 1], block_table [batch, pages_per_seq], "
                         "taken [2], cursor [1]")
    n_free = free_pages.numel()
    if B > INT32_MAX or n_free > INT32_MAX or shape[1] > INT32_MAX:
        raise _too_many(fn)
    _check(fn, load().kvq_extend_block_table(held.data_ptr(), n_new.data_ptr(), B, free_pages.data_ptr(), n_free,
                                             None if cursor is None else cursor.data_ptr(), block_table.data_ptr(), shape[1],
                                             seq_start.data_ptr(), ctx_lens.data_ptr(), taken.data_ptr(), _stream(stream)))


def kvq_slot_map(held: torch.Tensor, seq_start: torch.Tensor, ctx_lens: torch.Tensor, block_table: torch.Tensor, n_pages: int,
                 seq_ids, positions, slots: torch.Tensor, stream=None):
    """Request, position (int32 [n_tokens], either may be None) and page slot (int64 [n_tokens], -1: none) of
    every new token."""
    fn = "kvq_slot_map"
    _here(fn, torch.int32, held=held, seq_start=seq_start, ctx_lens=ctx_lens, block_table=block_table, seq_ids=seq_ids,
          positions=positions)
    _here(fn, torch.int64, slots=slots)
    B, n, shape = held.numel(), slots.numel(), block_table.shape
    if len(shape) != 2 or shape[0] != B or seq_start.numel() != B + 1 or ctx_lens.numel() != B \
            or (seq_ids is not None and seq_ids.numel() != n) or (positions is not None and positions.numel() != n):
        raise ValueError(f"{fn}: held, ctx_lens [batch], seq_start [batch + 1], block_table [batch, pages_per_seq], "
                         "seq_ids, positions, slots [n_tokens]")
    if B > INT32_MAX or shape[1] > INT32_MAX or n > INT32_MAX or not -INT32_MAX <= n_pages <= INT32_MAX:
        raise _too_many(fn)
    _check(fn, load().kvq_slot_map(held.data_ptr(), seq_start.data_ptr(), ctx_lens.data_ptr(), B, block_table.data_ptr(),
                                   shape[1], n_pages, n, None if seq_ids is None else seq_ids.data_ptr(),
                                   None if positions is None else positions.data_ptr(), slots.data_ptr(), _stream(stream)))


def kvq_quantize_slots(handle, K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, stream=None, seq_start=None):
    """Code K, V [n_tokens, n_kv_heads, head_dim] into page slots int64 [n_tokens] (negative: skipped). With
    seq_start (int32 [batch + 1]) only the rows of requests are written (kvq_quantize_slots_rows); without it every
    row counts, so slots that kvq_slot_map left as they were have to be negative."""
    fn = "kvq_quantize_slots"
    if K.dtype not in DTYPES or V.dtype != K.dtype:
        raise TypeError("K and V must both be float32 or bfloat16")
    _here(fn, K=K, V=V)
    _here(fn, torch.int64, slots=slots)
    if seq_start is not None:
        _here(fn, torch.int32, seq_start=seq_start)
    if K.dim() != 3 or K.shape != V.shape or slots.numel() != K.shape[0]:
        raise ValueError("K and V must be [n_tokens, n_kv_heads, head_dim] and slots [n_tokens]")
    n = K.shape[0]
    if n > INT32_MAX:
        raise _too_many(fn)
    if seq_start is None:
        _check(fn, load().kvq_quantize_slots(handle, K.data_ptr(), V.data_ptr(), DTYPES[K.dtype], slots.data_ptr(), n,
                                             _stream(stream)))
    else:
        _check(fn, load().kvq_quantize_slots_rows(handle, K.data_ptr(), V.data_ptr(), DTYPES[K.dtype], slots.data_ptr(), n,
                                                  seq_start.data_ptr(), _stream(stream)))


def kvq_cache_set_lengths(handle, lens, batch: int, stream=None):
    """Set the lengths of all sequences (batch host integers)."""
    a = np.ascontiguousarray(lens)
    if a.shape != (batch,) or a.dtype.kind not in "iu" or (a.size and (a.max() > 2**31 - 1 or a.min() < -2**31)):
        raise ValueError("lens must hold one integer per sequence")
    a = a.astype(np.int32)
    _check("kvq_cache_set_lengths", load().kvq_cache_set_lengths(handle, a.ctypes.data_as(ctypes.c_void_p), _stream(stream)))


def kvq_chunk_workspace_bytes(handle, dtype, n_tokens: int) -> int:
    out = ctypes.c_size_t()
    if not -INT32_MAX <= n_tokens <= INT32_MAX:
        raise _too_many("kvq_chunk_workspace_bytes")
    _check("kvq_chunk_workspace_bytes",
           load().kvq_chunk_workspace_bytes(handle, DTYPES[dtype], n_tokens, ctypes.byref(out)))
    return out.value


def kvq_chunk_attention(handle, q: torch.Tensor, seq_start: torch.Tensor, ctx_lens, out: torch.Tensor,
                        workspace: torch.Tensor, stream=None, held=None):
    """Attention of new tokens' queries q [n_tokens, n_q_heads, head_dim], request b's in rows seq_start[b] ..
    seq_start[b + 1] - 1, over the packed cache of ctx_lens [batch] tokens (None: the cache's lengths). out is
    like q. With held [batch], the lengths before the step, requests that kvq_extend_block_table refused get zeros
    (kvq_chunk_attention_held); without it their rows attend as if their tokens were the last of ctx_lens."""
    fn = "kvq_chunk_attention"
    if q.dtype not in DTYPES or out.dtype != q.dtype:
        raise TypeError("q and out must both be float32 or bfloat16")
    _here(fn, q=q, out=out, workspace=workspace)
    _here(fn, torch.int32, seq_start=seq_start, ctx_lens=ctx_lens, held=held)
    if q.dim() != 3 or out.shape != q.shape:
        raise ValueError("q and out must be [n_tokens, n_q_heads, head_dim]")
    if q.shape[0] > INT32_MAX:
        raise _too_many(fn)
    first = (handle, q.data_ptr(), DTYPES[q.dtype], q.shape[0], seq_start.data_ptr(),
             None if ctx_lens is None else ctx_lens.data_ptr())
    last = out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream)
    if held is None:
        _check(fn, load().kvq_chunk_attention(*first, *last))
    else:
        _check(fn, load().kvq_chunk_attention_held(*first, held.data_ptr(), *last))


def kvq_decode_attention_static(handle, q: torch.Tensor, out: torch.Tensor, stream=None):
    """Decode attention without a workspace (partials in the library's fixed device array)."""
    _on_device("kvq_decode_attention_static", q=q, out=out)
    if q.dtype not in DTYPES or out.dtype != torch.float32:
        raise TypeError("q must be float32/bfloat16 and out float32")
    if not (q.is_contiguous() and out.is_contiguous()):
        raise ValueError("q and out must be contiguous")
    st = load().kvq_decode_attention_static(handle, _ptr(q), DTYPES[q.dtype], _ptr(out), _stream(stream))
    _check("kvq_decode_attention_static", st)


def kvq_cache_status(handle, stream=None) -> int:
    """The cache's device status word (KVQ_STATUS_* bits); waits for the stream."""
    v = ctypes.c_int32(0)
    _check("kvq_cache_status", load().kvq_cache_status(handle, ctypes.byref(v), _stream(stream)))
    return int(v.value)


def kvq_debug_decode_unset_wait(handle, q: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                                wait_limit_cycles: int, stream=None):
    """Test entry: decode with one extra bounded wait on a barrier that nothing completes."""
    _on_device("kvq_debug_decode_unset_wait", q=q, out=out, workspace=workspace)
    if q.dtype not in DTYPES or out.dtype != torch.float32:
        raise TypeError("q must be float32/bfloat16 and out float32")
    if not (q.is_contiguous() and out.is_contiguous()):
        raise ValueError("q and out must be contiguous")
    st = load().kvq_debug_decode_unset_wait(handle, _ptr(q), DTYPES[q.dtype], _ptr(out), _ptr(workspace),
                                            workspace.numel() * workspace.element_size(),
                                            int(wait_limit_cycles), _stream(stream))
    _check("kvq_debug_decode_unset_wait", st)


def kvq_debug_decode_timed(handle, q: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, events,
                           stream=None):
    """Decode recording 4 torch.cuda.Events: start, after prep, after the split kernel, after reduce."""
    _on_device("kvq_debug_decode_timed", q=q, out=out, workspace=workspace)
    if q.dtype not in DTYPES or out.dtype != torch.float32:
        raise TypeError("q must be float32/bfloat16 and out float32")
    if len(events) != 4:
        raise ValueError("four events")
    for e in events:
        if e.cuda_event == 0:  # torch creates the event lazily, on its first record
            e.record()
    arr = (ctypes.c_void_p * 4)(*[ctypes.c_void_p(e.cuda_event) for e in events])
    st = load().kvq_debug_decode_timed(handle, _ptr(q), DTYPES[q.dtype], _ptr(out), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream), arr)
    _check("kvq_debug_decode_timed", st)


def kvq_cache_lengths(handle, batch: int) -> np.ndarray:
    lens = np.zeros(batch, dtype=np.int32)
    _check("kvq_cache_lengths", load().kvq_cache_lengths(handle, lens.ctypes.data_as(ctypes.c_void_p)))
    return lens


def kvq_cache_layout(handle) -> np.ndarray:
    info = np.zeros(24, dtype=np.int64)
    _check("kvq_cache_layout", load().kvq_cache_layout(handle, info.ctypes.data_as(ctypes.c_void_p), 24))
    return info


def kvq_lloyd_max_table(bits: int):
    c = np.zeros(1 << bits, dtype=np.float32)
    t = np.zeros((1 << bits) - 1, dtype=np.float32)
    _check("kvq_lloyd_max_table", load().kvq_lloyd_max_table(bits, c.ctypes.data_as(ctypes.c_void_p),
                                                             t.ctypes.data_as(ctypes.c_void_p)))
    return c, t


def kvq_cache_destroy(handle):
    if handle:
        load().kvq_cache_destroy(handle)


def kvq_kernel_launches() -> int:
    """Kernels the library has enqueued since it was loaded (all threads and devices)."""
    return int(load().kvq_kernel_launches())


def kvq_debug_quantize_rotated(handle, u: torch.Tensor, k_bits: int, qjl: bool, stream=None):
    _on_device("kvq_debug_quantize_rotated", u=u)
    n = u.shape[0]
    planes = torch.zeros((n, k_bits, 4), dtype=torch.int32, device=u.device)
    sketch = torch.zeros((n, 4), dtype=torch.int32, device=u.device) if qjl else None
    gamma = torch.zeros((n,), dtype=torch.int16, device=u.device) if qjl else None
    st = load().kvq_debug_quantize_rotated(handle, _ptr(u), n, _ptr(planes), _ptr(sketch), _ptr(gamma),
                                           _stream(stream))
    _check("kvq_debug_quantize_rotated", st)
    return planes, sketch, gamma


# ---------------------------------------------------------------- convenience object

class KvqCache:
    """A packed cache in a torch-allocated device arena, plus its decode workspace.

    With block_table (an int32 CUDA tensor [batch, pages_per_seq]) and n_pages, the cache is paged:
    its tiles live in a pool of n_pages pages of 64 tokens and the table names the page of each
    64-token page of a sequence; the caller owns the table and fills it before tokens reach a page."""

    def __init__(self, cfg: kvq_cfg, batch: int, capacity: int, rot_signs=None, qjl_matrix=None,
                 device="cuda", block_table=None, n_pages=0):
        if not torch.cuda.is_available():
            raise RuntimeError("kvq needs a CUDA device")
        self.cfg, self.batch = cfg, batch
        if block_table is None:
            nbytes = kvq_cache_bytes(cfg, batch, capacity)
            self.arena = torch.empty(nbytes, dtype=torch.uint8, device=device)
            self.handle = kvq_cache_init(cfg, batch, capacity, self.arena, rot_signs, qjl_matrix)
        else:
            self.block_table = block_table
            nbytes = kvq_cache_bytes_paged(cfg, batch, n_pages)
            self.arena = torch.empty(nbytes, dtype=torch.uint8, device=device)
            self.handle = kvq_cache_init_paged(cfg, batch, n_pages, block_table, self.arena, rot_signs, qjl_matrix)
        self.workspace = torch.empty(max(16, kvq_workspace_bytes(self.handle)), dtype=torch.uint8,
                                     device=device)
        self.chunk_workspaces, self.chunk_lock = {}, threading.Lock()
        self.out_dim = cfg.latent_dim if cfg.k_mode == MODES["fp4"] else cfg.head_dim

    # Shapes the library reads and writes; it cannot see tensor extents, so they are checked here.
    def _kv_shapes(self, n_seq: int, n_new: int):
        cfg = self.cfg
        if cfg.k_mode == MODES["fp4"]:
            return (n_seq, n_new, cfg.latent_dim), (n_seq, n_new, cfg.rope_dim)
        kv = (n_seq, cfg.n_kv_heads, n_new, cfg.head_dim)
        return kv, kv

    def _check_kv(self, fn, K, V, n_seq, n_new):
        if K.dim() < 2 or (tuple(K.shape), tuple(V.shape)) != self._kv_shapes(n_seq, n_new):
            raise ValueError(f"{fn}: K, V must be {self._kv_shapes(n_seq, n_new)}, got {tuple(K.shape)}, {tuple(V.shape)}")

    def _check_q_out(self, fn, q, out):
        cfg = self.cfg
        dq = cfg.latent_dim + cfg.rope_dim if cfg.k_mode == MODES["fp4"] else cfg.head_dim
        if tuple(q.shape) != (self.batch, cfg.n_q_heads, dq):
            raise ValueError(f"{fn}: q must be {(self.batch, cfg.n_q_heads, dq)}, got {tuple(q.shape)}")
        if out is not None and tuple(out.shape) != (self.batch, cfg.n_q_heads, self.out_dim):
            raise ValueError(f"{fn}: out must be {(self.batch, cfg.n_q_heads, self.out_dim)}")

    def quantize(self, K, V, seq_ids=None, stream=None):
        n_seq = K.shape[0] if K.dim() else 0
        if seq_ids is None and n_seq > self.batch:
            raise ValueError("quantize: more sequences than the cache holds")
        self._check_kv("quantize", K, V, n_seq, K.shape[-2] if K.dim() >= 2 else 0)
        kvq_quantize(self.handle, K, V, seq_ids, stream)

    def step(self, K, V, q, out=None, stream=None):
        """Append one token per sequence and decode (kvq_decode_step); returns out."""
        self._check_kv("step", K, V, self.batch, 1)
        self._check_q_out("step", q, out)
        if out is None:
            with _memory_of(stream):
                out = torch.empty((self.batch, self.cfg.n_q_heads, self.out_dim), dtype=torch.float32,
                                  device=q.device)
        kvq_decode_step(self.handle, K, V, q, out, self.workspace, stream)
        return out

    def step_host(self, K, V, q, out=None, stream=None, out_event=None):
        """step() with host (CPU) inputs and output: one call enqueues the input copies, the step
        and the output copy; returns out (valid after the stream reaches it, or, with out_event,
        once that event has completed)."""
        if out is None:
            out = torch.empty((self.batch, self.cfg.n_q_heads, self.out_dim), dtype=torch.float32).pin_memory()
        # the library cannot see host buffer sizes: check them here
        B, Hq, cfg = self.batch, self.cfg.n_q_heads, self.cfg
        if cfg.k_mode == MODES["fp4"]:
            want = (B * cfg.latent_dim, B * cfg.rope_dim, B * Hq * (cfg.latent_dim + cfg.rope_dim))
        else:
            want = (B * cfg.n_kv_heads * cfg.head_dim,) * 2 + (B * Hq * cfg.head_dim,)
        if tuple(t.numel() for t in (K, V, q)) != want or K.dtype != q.dtype or V.dtype != q.dtype:
            raise ValueError(f"step_host: K, V, q must hold {want} elements of one dtype")
        if out.dtype != torch.float32 or out.numel() != B * Hq * self.out_dim:
            raise ValueError("step_host: out must be float32 [batch, n_q_heads, out_dim]")
        need = kvq_step_staging_bytes(self.handle, q.dtype)
        if getattr(self, "staging", None) is None or self.staging.numel() < need:
            with _memory_of(stream):
                self.staging = torch.empty(need, dtype=torch.uint8, device=self.workspace.device)
        return kvq_decode_step_host(self.handle, K, V, q, q.dtype, out, self.staging, self.workspace, stream,
                                    out_event)

    def decode(self, q, out=None, stream=None):
        self._check_q_out("decode", q, out)
        if out is None:
            with _memory_of(stream):
                out = torch.empty((self.batch, self.cfg.n_q_heads, self.out_dim), dtype=torch.float32,
                                  device=q.device)
        kvq_decode_attention(self.handle, q, out, self.workspace, stream)
        return out

    def decode_partials(self, q, partials=None, stream=None):
        """Softmax state of this cache's tokens (kvq_decode_partials): [batch, n_q_heads, 2 + dv]."""
        self._check_q_out("decode_partials", q, None)
        n = kvq_partial_floats(self.handle)
        if partials is None:
            with _memory_of(stream):
                partials = torch.empty((self.batch, self.cfg.n_q_heads, n), dtype=torch.float32, device=q.device)
        if tuple(partials.shape) != (self.batch, self.cfg.n_q_heads, n):
            raise ValueError(f"decode_partials: partials must be {(self.batch, self.cfg.n_q_heads, n)}")
        kvq_decode_partials(self.handle, q, partials, self.workspace, stream)
        return partials

    def quantize_slots(self, K, V, slots, stream=None, seq_start=None):
        """Code a token-major batch K, V [n_tokens, n_kv_heads, head_dim] into page slots (kvq_quantize_slots); with
        seq_start [batch + 1] the rows of requests alone."""
        if K.dim() != 3 or tuple(K.shape[1:]) != (self.cfg.n_kv_heads, self.cfg.head_dim) or K.shape != V.shape:
            raise ValueError(f"quantize_slots: K, V must be [n_tokens, {self.cfg.n_kv_heads}, {self.cfg.head_dim}]")
        if seq_start is not None and seq_start.numel() != self.batch + 1:
            raise ValueError(f"quantize_slots: seq_start [{self.batch + 1}]")
        kvq_quantize_slots(self.handle, K, V, slots, stream, seq_start)

    def set_lengths(self, lens, stream=None):
        """Set every sequence's length (kvq_cache_set_lengths)."""
        kvq_cache_set_lengths(self.handle, lens, self.batch, stream)

    def chunk_attention(self, q, seq_start, ctx_lens=None, out=None, workspace=None, stream=None, held=None):
        """Attention of a ragged batch of new tokens (kvq_chunk_attention; with held, the lengths before the step, refused
        requests get zeros); returns out, like q. Without a workspace the cache keeps one per stream, grown to the largest call there; a captured call takes one
        from the graph's own memory, so that no two graphs share it. Calls of several threads are enqueued one after
        the other; a workspace of one's own is for one call at a time. Kept workspaces go with close()."""
        if q.dim() != 3 or tuple(q.shape[1:]) != (self.cfg.n_q_heads, self.cfg.head_dim):
            raise ValueError(f"chunk_attention: q must be [n_tokens, {self.cfg.n_q_heads}, {self.cfg.head_dim}]")
        if seq_start.numel() != self.batch + 1 or any(t is not None and t.numel() != self.batch for t in (ctx_lens, held)):
            raise ValueError(f"chunk_attention: seq_start [{self.batch + 1}], ctx_lens and held [{self.batch}]")
        if q.dtype not in DTYPES:
            raise TypeError("q must be float32 or bfloat16")
        with _memory_of(stream):
            _here("chunk_attention", q=q)  # before anything is made beside it
            if out is None:
                out = torch.empty_like(q)
            if workspace is not None:
                kvq_chunk_attention(self.handle, q, seq_start, ctx_lens, out, workspace, stream, held)
                return out
            # a call is several launches, and the library releases the interpreter: threads that share a stream, and so
            # a workspace, enqueue theirs one call after the other
            with self.chunk_lock:
                workspace = self._chunk_workspace(kvq_chunk_workspace_bytes(self.handle, q.dtype, q.shape[0]), q.device)
                kvq_chunk_attention(self.handle, q, seq_start, ctx_lens, out, workspace, stream, held)
        return out

    def _chunk_workspace(self, need, device):
        # memory of the current stream: a workspace it outgrows is reused in its order
        if torch.cuda.is_current_stream_capturing():
            return torch.empty(need, dtype=torch.uint8, device=device)
        # every device's default stream has the handle 0
        kept, at = self.chunk_workspaces, (device, _stream())
        have = kept.get(at)
        if have is None or have.numel() < need:
            have = kept[at] = torch.empty(need, dtype=torch.uint8, device=device)
        return have

    def lengths(self):
        return kvq_cache_lengths(self.handle, self.batch)

    def layout(self):
        return kvq_cache_layout(self.handle)

    def close(self):
        if self.handle:
            kvq_cache_destroy(self.handle)
            self.handle = None
            self.chunk_workspaces.clear()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
