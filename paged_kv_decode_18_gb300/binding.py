"""Thin Python binding of libpagedattn's C ABI (include/pa.h).

Argument marshalling only: every function takes torch CUDA tensors, checks
dtype / contiguity / device, passes raw device pointers, the shape struct and
the current CUDA stream to the C entry point of the same name, and raises
``PAError`` on a non-zero status. All arithmetic runs in the library's CUDA
kernels; there is no fallback. If the library has not been built the first
call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libpagedattn.so")

PA_OK = 0
PA_ERR_ARG = -1
PA_ERR_UNSUPPORTED = -2
PA_ERR_WORKSPACE = -3
PA_ERR_CUDA = -4
PA_ERR_DEVICE = -5

PA_DEVERR_SLOT_RANGE = 0x1
PA_DEVERR_BLOCK_RANGE = 0x2
PA_DEVERR_CONTEXT_RANGE = 0x4
PA_DEVERR_QLEN_RANGE = 0x8
PA_DEVERR_PIPE_TIMEOUT = 0x10
PA_DEVERR_PLAN_OVERFLOW = 0x20
PA_DEVERR_TREE_RANGE = 0x40
PA_DEVERR_BUDGET_RANGE = 0x80

# pool formats of the calls that take any of the library's pools
PA_KV_BF16 = 0
PA_KV_INT8 = 1
PA_KV_FP8 = 2

# every symbol include/pa.h declares
EXPORTED = (
    "pa_reshape_and_cache",
    "pa_decode",
    "pa_decode_workspace_size",
    "pa_decode_static_scratch",
    "pa_append_decode",
    "pa_decode_varlen",
    "pa_decode_varlen_workspace_size",
    "pa_reshape_and_cache_int8",
    "pa_decode_int8",
    "pa_decode_int8_workspace_size",
    "pa_reshape_and_cache_fp8",
    "pa_decode_fp8",
    "pa_decode_fp8_workspace_size",
    "pa_decode_cascade",
    "pa_decode_cascade_ex",
    "pa_decode_cascade_workspace_size",
    "pa_tree_mask",
    "pa_decode_tree",
    "pa_decode_tree_workspace_size",
    "pa_commit_path",
    "pa_accumulate_weights",
    "pa_evict",
    "pa_rotation_init",
    "pa_rotation_set",
    "pa_rotate",
    "pa_rotate_and_cache",
    "pa_rotate_cached",
    "pa_decode_diff",
    "pa_decode_diff_workspace_size",
    "pa_splitk_reduce",
    "pa_status_string",
    "pa_debug_read_error",
    "pa_debug_inject_missing_copy",
    "pa_version",
)


class pa_shape(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int),
        ("num_q_heads", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("block_size", ctypes.c_int),
        ("max_blocks_per_seq", ctypes.c_int),
        ("num_blocks", ctypes.c_int64),
    ]


class pa_rotation(ctypes.Structure):
    _fields_ = [
        ("rot_dim", ctypes.c_int),
        ("interleaved", ctypes.c_int),
        ("magnitude", ctypes.c_float),
        ("turns", ctypes.c_uint64 * 64),
    ]


class pa_row_view(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
    ]


class PAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {pa_status_string(status)} ({status})")


_lib = None
_lock = threading.Lock()


def load(path: str | None = None):
    """Load the library (once). Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"libpagedattn.so not found at {p}; build it first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(p)
        V, S = ctypes.c_void_p, ctypes.POINTER(pa_shape)
        i32, i64, f32, sz = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        lib.pa_reshape_and_cache.restype = i32
        lib.pa_reshape_and_cache.argtypes = [V, V, V, i64, V, V, S, V]
        lib.pa_decode.restype = i32
        lib.pa_decode.argtypes = [V, V, V, V, V, f32, V, V, S, i32, V, sz, V]
        lib.pa_decode_workspace_size.restype = sz
        lib.pa_decode_workspace_size.argtypes = [S, i32]
        lib.pa_append_decode.restype = i32
        lib.pa_append_decode.argtypes = [V, V, V, i64, V, V, V, V, V, f32, V, V, S, V, sz, V]
        lib.pa_decode_static_scratch.restype = i32
        lib.pa_decode_static_scratch.argtypes = [V, V, V, V, V, f32, V, V, S, V]
        lib.pa_decode_varlen.restype = i32
        lib.pa_decode_varlen.argtypes = [V, V, V, V, V, V, i64, i32, i32, f32, V, V, S, V, sz, V]
        lib.pa_decode_varlen_workspace_size.restype = sz
        lib.pa_decode_varlen_workspace_size.argtypes = [S, i64, i32]
        lib.pa_reshape_and_cache_int8.restype = i32
        lib.pa_reshape_and_cache_int8.argtypes = [V, V, V, i64, V, V, S, V]
        lib.pa_decode_int8.restype = i32
        lib.pa_decode_int8.argtypes = [V, V, V, V, V, f32, V, V, S, i32, V, sz, V]
        lib.pa_decode_int8_workspace_size.restype = sz
        lib.pa_decode_int8_workspace_size.argtypes = [S, i32]
        lib.pa_reshape_and_cache_fp8.restype = i32
        lib.pa_reshape_and_cache_fp8.argtypes = [V, V, V, i64, V, V, S, V]
        lib.pa_decode_fp8.restype = i32
        lib.pa_decode_fp8.argtypes = [V, V, V, V, V, f32, V, V, S, i32, V, sz, V]
        lib.pa_decode_fp8_workspace_size.restype = sz
        lib.pa_decode_fp8_workspace_size.argtypes = [S, i32]
        lib.pa_decode_cascade.restype = i32
        lib.pa_decode_cascade.argtypes = [V, V, V, V, V, V, i32, V, V, V, i32, i32, i32, f32,
                                          V, V, S, V, sz, V]
        lib.pa_decode_cascade_ex.restype = i32
        lib.pa_decode_cascade_ex.argtypes = [V, V, V, V, V, V, i32, V, V, V, i32, i32, i32, f32,
                                             V, V, S, i32, V, sz, V]
        lib.pa_decode_cascade_workspace_size.restype = sz
        lib.pa_decode_cascade_workspace_size.argtypes = [S, i32, i32, i32, i32]
        lib.pa_tree_mask.restype = i32
        lib.pa_tree_mask.argtypes = [V, V, i32, i64, i32, V, i32, V, V]
        lib.pa_decode_tree.restype = i32
        lib.pa_decode_tree.argtypes = [V, V, V, V, V, V, V, i32, i64, i32, f32, V, V, S, V, sz,
                                       V]
        lib.pa_decode_tree_workspace_size.restype = sz
        lib.pa_decode_tree_workspace_size.argtypes = [S, i64, i32]
        lib.pa_commit_path.restype = i32
        lib.pa_commit_path.argtypes = [V, V, i32, V, V, V, V, V, i32, V, S, V]
        lib.pa_accumulate_weights.restype = i32
        lib.pa_accumulate_weights.argtypes = [V, V, i32, V, V, V, V, i64, i32, f32, i32, V, i64,
                                              S, V]
        lib.pa_evict.restype = i32
        lib.pa_evict.argtypes = [V, V, i32, V, V, V, i64, V, i32, i32, i32, V, V, S, V]
        R, Rows, f64 = ctypes.POINTER(pa_rotation), ctypes.POINTER(pa_row_view), ctypes.c_double
        lib.pa_rotation_init.restype = i32
        lib.pa_rotation_init.argtypes = [R, i32, i32, f64, i32, f64, f64, f64, f64]
        lib.pa_rotation_set.restype = i32
        lib.pa_rotation_set.argtypes = [R, i32, i32, ctypes.POINTER(f64), f32]
        lib.pa_rotate.restype = i32
        lib.pa_rotate.argtypes = [Rows, V, i64, i32, i32, R, i32, Rows, V]
        lib.pa_rotate_and_cache.restype = i32
        lib.pa_rotate_and_cache.argtypes = [Rows, Rows, Rows, V, V, i64, R, Rows, V, V, i32, S, V]
        lib.pa_rotate_cached.restype = i32
        lib.pa_rotate_cached.argtypes = [V, i32, V, V, V, i32, V, i32, R, S, V]
        lib.pa_decode_diff.restype = i32
        lib.pa_decode_diff.argtypes = [V, V, V, V, V, V, i64, i32, i32, f32, V, V, f32, f32, V, V,
                                       S, V, sz, V]
        lib.pa_decode_diff_workspace_size.restype = sz
        lib.pa_decode_diff_workspace_size.argtypes = [S, i64, i32]
        lib.pa_splitk_reduce.restype = i32
        lib.pa_splitk_reduce.argtypes = [V, V, i64, i32, i32, i32, V, V, V]
        lib.pa_status_string.restype = ctypes.c_char_p
        lib.pa_status_string.argtypes = [i32]
        lib.pa_debug_read_error.restype = i32
        lib.pa_debug_read_error.argtypes = [V]
        lib.pa_debug_inject_missing_copy.restype = i32
        lib.pa_debug_inject_missing_copy.argtypes = [i32]
        lib.pa_version.restype = ctypes.c_char_p
        lib.pa_version.argtypes = []
        _lib = lib
        return lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtype, ndim=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    return t


def _check(rc: int, what: str):
    if rc != PA_OK:
        raise PAError(rc, what)


def make_shape(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq,
               num_blocks) -> pa_shape:
    return pa_shape(int(num_seqs), int(num_q_heads), int(num_kv_heads), int(head_dim),
                    int(block_size), int(max_blocks_per_seq), int(num_blocks))


# bytes of one (block, KV head) tile of the int8 and FP8 pools: 16 x 128
# one-byte codes, then the 16 rows' fp32 scales
PA_INT8_TILE_BYTES = 2112
INT8_BLOCK, INT8_HEAD_DIM = 16, 128


def shape_of(q, k_cache, block_tables, num_seqs=None) -> pa_shape:
    """Shape struct from the tensors: q [*, Hq, D], k_cache [NB, Hkv, BS, D]
    (bf16) or [NB, Hkv, PA_INT8_TILE_BYTES] (uint8, the int8 or FP8 pool),
    block_tables [S, max_blocks]."""
    if k_cache.dim() == 3 and k_cache.dtype == torch.uint8:
        if k_cache.shape[2] != PA_INT8_TILE_BYTES:
            raise ValueError(f"8-bit pool tiles must be {PA_INT8_TILE_BYTES} bytes")
        NB, Hkv = k_cache.shape[:2]
        BS, D = INT8_BLOCK, INT8_HEAD_DIM
    else:
        NB, Hkv, BS, D = k_cache.shape
    S = block_tables.shape[0] if num_seqs is None else num_seqs
    return make_shape(S, q.shape[1], Hkv, D, BS, block_tables.shape[1], NB)


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def pa_status_string(status: int) -> str:
    return load().pa_status_string(int(status)).decode()


def pa_version() -> str:
    return load().pa_version().decode()


def pa_debug_read_error(stream=None) -> int:
    rc = load().pa_debug_read_error(_stream(stream))
    if rc < 0:
        raise PAError(rc, "pa_debug_read_error")
    return rc


def pa_debug_inject_missing_copy(flat_tile: int) -> None:
    """Failure-detection hook: the next decode launch leaves out the copy of
    one tile, so its bounded wait expires and flags PA_DEVERR_PIPE_TIMEOUT."""
    _check(load().pa_debug_inject_missing_copy(int(flat_tile)), "pa_debug_inject_missing_copy")


def pa_reshape_and_cache(k, v, slot_mapping, k_cache, v_cache, stream=None) -> None:
    _need(k, "k", torch.bfloat16, 3)
    _need(v, "v", torch.bfloat16, 3)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    if k.shape != v.shape or k_cache.shape != v_cache.shape:
        raise ValueError("k/v or cache shapes differ")
    if slot_mapping.shape[0] != k.shape[0]:
        raise ValueError("slot_mapping length != number of tokens")
    NB, Hkv, BS, D = k_cache.shape
    if k.shape[1:] != (Hkv, D):
        raise ValueError("k rows do not match the cache's [Hkv, D]")
    sh = make_shape(0, Hkv, Hkv, D, BS, 0, NB)
    _check(load().pa_reshape_and_cache(_ptr(k), _ptr(v), _ptr(slot_mapping), k.shape[0],
                                       _ptr(k_cache), _ptr(v_cache), ctypes.byref(sh),
                                       _stream(stream)), "pa_reshape_and_cache")


def pa_decode_workspace_size(shape: pa_shape, num_splits: int = 0) -> int:
    return int(load().pa_decode_workspace_size(ctypes.byref(shape), int(num_splits)))


def _cache_write_q8(name, k, v, slot_mapping, k_cache, v_cache, stream):
    _need(k, "k", torch.bfloat16, 3)
    _need(v, "v", torch.bfloat16, 3)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    _need(k_cache, "k_cache", torch.uint8, 3)
    _need(v_cache, "v_cache", torch.uint8, 3)
    if k.shape != v.shape or k_cache.shape != v_cache.shape:
        raise ValueError("k/v or cache shapes differ")
    if slot_mapping.shape[0] != k.shape[0]:
        raise ValueError("slot_mapping length != number of tokens")
    sh = shape_of(k, k_cache, torch.empty((0, 0)))
    if k.shape[1:] != (sh.num_kv_heads, sh.head_dim):
        raise ValueError("k rows do not match the cache")
    _check(getattr(load(), name)(_ptr(k), _ptr(v), _ptr(slot_mapping), k.shape[0],
                                 _ptr(k_cache), _ptr(v_cache), ctypes.byref(sh),
                                 _stream(stream)), name)


def pa_reshape_and_cache_int8(k, v, slot_mapping, k_cache, v_cache, stream=None) -> None:
    """Quantising cache write into the int8 pool (uint8 tiles [NB, Hkv, 2112]:
    a tile's 16 x 128 codes, then its 16 fp32 row scales)."""
    _cache_write_q8("pa_reshape_and_cache_int8", k, v, slot_mapping, k_cache, v_cache, stream)


def pa_reshape_and_cache_fp8(k, v, slot_mapping, k_cache, v_cache, stream=None) -> None:
    """Quantising cache write into the FP8 (E4M3) pool (same tiles as int8)."""
    _cache_write_q8("pa_reshape_and_cache_fp8", k, v, slot_mapping, k_cache, v_cache, stream)


def pa_decode_cascade_workspace_size(shape: pa_shape, num_groups: int, num_members: int,
                                     max_group_size: int, max_prefix_len: int) -> int:
    return int(load().pa_decode_cascade_workspace_size(ctypes.byref(shape), int(num_groups),
                                                       int(num_members), int(max_group_size),
                                                       int(max_prefix_len)))


PA_CASCADE_AUTO = 0
PA_CASCADE_ALWAYS = 1
PA_CASCADE_PLAIN = 2


def pa_decode_cascade(q, k_cache, v_cache, block_tables, context_lens, seq_group, cu_group,
                      group_members, prefix_lens, max_group_size, max_prefix_len, scale, out,
                      lse=None, workspace=None, stream=None, policy=PA_CASCADE_AUTO) -> None:
    """Decode with shared prefixes attended once per group (same result as
    pa_decode). policy: PA_CASCADE_AUTO (the library decides whether the
    cascade pays), PA_CASCADE_ALWAYS or PA_CASCADE_PLAIN."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(seq_group, "seq_group", torch.int32, 1)
    _need(cu_group, "cu_group", torch.int32, 1)
    _need(prefix_lens, "prefix_lens", torch.int32, 1)
    if group_members.numel():
        _need(group_members, "group_members", torch.int32, 1)
    _need(out, "out", torch.bfloat16, 3)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    sh = shape_of(q, k_cache, block_tables)
    G = prefix_lens.shape[0]
    if cu_group.shape[0] != G + 1 or seq_group.shape[0] != sh.num_seqs:
        raise ValueError("group description shapes do not match")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().pa_decode_cascade_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache),
                                       _ptr(block_tables), _ptr(context_lens), _ptr(seq_group),
                                       G, _ptr(cu_group),
                                       _ptr(group_members) if group_members.numel() else None,
                                       _ptr(prefix_lens), int(group_members.numel()),
                                       int(max_group_size), int(max_prefix_len), float(scale),
                                       _ptr(out), _ptr(lse), ctypes.byref(sh), int(policy),
                                       _ptr(workspace), ws_bytes, _stream(stream)),
           "pa_decode_cascade")


def pa_decode_int8_workspace_size(shape: pa_shape, num_splits: int = 0) -> int:
    return int(load().pa_decode_int8_workspace_size(ctypes.byref(shape), int(num_splits)))


def pa_decode_fp8_workspace_size(shape: pa_shape, num_splits: int = 0) -> int:
    return int(load().pa_decode_fp8_workspace_size(ctypes.byref(shape), int(num_splits)))


def _decode_q8(name, q, k_cache, v_cache, block_tables, context_lens, scale, out, lse,
               num_splits, workspace, stream):
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.uint8, 3)
    _need(v_cache, "v_cache", torch.uint8, 3)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(out, "out", torch.bfloat16, 3)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    if k_cache.shape != v_cache.shape:
        raise ValueError("k / v cache shapes differ")
    sh = shape_of(q, k_cache, block_tables)
    if q.shape[0] != sh.num_seqs or context_lens.shape[0] != sh.num_seqs:
        raise ValueError("q / context_lens rows != number of sequences")
    if out.shape != q.shape:
        raise ValueError("out shape != q shape")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(getattr(load(), name)(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                 _ptr(context_lens), float(scale), _ptr(out), _ptr(lse),
                                 ctypes.byref(sh), int(num_splits), _ptr(workspace), ws_bytes,
                                 _stream(stream)), name)


def pa_decode_int8(q, k_cache, v_cache, block_tables, context_lens, scale, out, lse=None,
                   num_splits: int = 0, workspace=None, stream=None) -> None:
    """Decode over the int8 pool with the dequantisation fused."""
    _decode_q8("pa_decode_int8", q, k_cache, v_cache, block_tables, context_lens, scale, out,
               lse, num_splits, workspace, stream)


def pa_decode_fp8(q, k_cache, v_cache, block_tables, context_lens, scale, out, lse=None,
                  num_splits: int = 0, workspace=None, stream=None) -> None:
    """Decode over the FP8 (E4M3) pool with the dequantisation fused."""
    _decode_q8("pa_decode_fp8", q, k_cache, v_cache, block_tables, context_lens, scale, out,
               lse, num_splits, workspace, stream)


def _prepared(cfn, args, stream, what, keep):
    """A zero-argument callable that makes one C-ABI call with arguments that
    were checked and converted once (the tensors in `keep` stay referenced).
    The stream goes last: fixed now when one was given, else the current
    torch stream of the tensors' device at each call (so the call can also be
    captured in a graph), taken as a raw handle: torch's stream object costs
    2.8 us, half of a small call."""
    if stream is not None:
        full = args + (_stream(stream),)

        def call():
            rc = cfn(*full)
            if rc != PA_OK:
                raise PAError(rc, what)
    else:
        device = keep[0].device.index

        def call():
            rc = cfn(*args, _raw_stream(device))
            if rc != PA_OK:
                raise PAError(rc, what)
    call.keep = keep
    return call


def prepare_decode(q, k_cache, v_cache, block_tables, context_lens, scale, out, lse=None,
                   num_splits: int = 0, workspace=None, stream=None):
    """pa_decode with its arguments checked and marshalled now; the returned
    callable makes the call each time it is invoked, on `stream` if one is
    given, else on the torch stream current at that moment. For serving loops
    that issue the same call on fixed buffers."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(out, "out", torch.bfloat16, 3)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    sh = shape_of(q, k_cache, block_tables)
    if q.shape[0] != sh.num_seqs or context_lens.shape[0] != sh.num_seqs:
        raise ValueError("q / context_lens rows != number of sequences")
    if out.shape != q.shape:
        raise ValueError("out shape != q shape")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
            ctypes.c_float(scale), _ptr(out), _ptr(lse), ctypes.byref(sh),
            ctypes.c_int(num_splits), _ptr(workspace), ctypes.c_size_t(ws_bytes))
    keep = (q, k_cache, v_cache, block_tables, context_lens, out, lse, workspace, sh)
    return _prepared(load().pa_decode, args, stream, "pa_decode", keep)


def pa_decode(q, k_cache, v_cache, block_tables, context_lens, scale, out, lse=None,
              num_splits: int = 0, workspace=None, stream=None) -> None:
    prepare_decode(q, k_cache, v_cache, block_tables, context_lens, scale, out, lse,
                   num_splits, workspace, stream)()


def prepare_append_decode(k_new, v_new, slot_mapping, q, k_cache, v_cache, block_tables,
                          context_lens, scale, out, lse=None, workspace=None, stream=None):
    """pa_append_decode with its arguments checked and marshalled now (see
    prepare_decode)."""
    _need(k_new, "k_new", torch.bfloat16, 3)
    _need(v_new, "v_new", torch.bfloat16, 3)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(out, "out", torch.bfloat16, 3)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    if k_new.shape != v_new.shape or slot_mapping.shape[0] != k_new.shape[0]:
        raise ValueError("k_new / v_new / slot_mapping disagree")
    sh = shape_of(q, k_cache, block_tables)
    if q.shape[0] != sh.num_seqs or context_lens.shape[0] != sh.num_seqs:
        raise ValueError("q / context_lens rows != number of sequences")
    if out.shape != q.shape:
        raise ValueError("out shape != q shape")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), ctypes.c_int64(k_new.shape[0]),
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
            ctypes.c_float(scale), _ptr(out), _ptr(lse), ctypes.byref(sh), _ptr(workspace),
            ctypes.c_size_t(ws_bytes))
    keep = (k_new, v_new, slot_mapping, q, k_cache, v_cache, block_tables, context_lens, out,
            lse, workspace, sh)
    return _prepared(load().pa_append_decode, args, stream, "pa_append_decode", keep)


def pa_append_decode(k_new, v_new, slot_mapping, q, k_cache, v_cache, block_tables,
                     context_lens, scale, out, lse=None, workspace=None, stream=None) -> None:
    """Cache write of the step's new K/V rows, then decode (balanced split), as
    one call whose decode preparation overlaps the write."""
    prepare_append_decode(k_new, v_new, slot_mapping, q, k_cache, v_cache, block_tables,
                          context_lens, scale, out, lse, workspace, stream)()


def pa_decode_static_scratch(q, k_cache, v_cache, block_tables, context_lens, scale, out,
                             lse=None, stream=None) -> None:
    """pa_decode (balanced split) without a workspace, for callers that cannot
    allocate device memory: the split scratch is a fixed 8 MiB array inside the
    library. Calls that may overlap on the GPU share that array and race."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(out, "out", torch.bfloat16, 3)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    sh = shape_of(q, k_cache, block_tables)
    if q.shape[0] != sh.num_seqs or context_lens.shape[0] != sh.num_seqs:
        raise ValueError("q / context_lens rows != number of sequences")
    if out.shape != q.shape:
        raise ValueError("out shape != q shape")
    _check(load().pa_decode_static_scratch(_ptr(q), _ptr(k_cache), _ptr(v_cache),
                                           _ptr(block_tables), _ptr(context_lens), float(scale),
                                           _ptr(out), _ptr(lse), ctypes.byref(sh),
                                           _stream(stream)), "pa_decode_static_scratch")


def pa_decode_varlen_workspace_size(shape: pa_shape, num_q_tokens: int, max_q_len: int) -> int:
    return int(load().pa_decode_varlen_workspace_size(ctypes.byref(shape), int(num_q_tokens),
                                                      int(max_q_len)))


def pa_decode_varlen(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, max_q_len,
                     scale, out, lse=None, causal: bool = True, workspace=None,
                     stream=None) -> None:
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(out, "out", torch.bfloat16, 3)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    sh = shape_of(q, k_cache, block_tables)
    if context_lens.shape[0] != sh.num_seqs or cu_seqlens_q.shape[0] != sh.num_seqs + 1:
        raise ValueError("context_lens / cu_seqlens_q length mismatch")
    if out.shape != q.shape:
        raise ValueError("out shape != q shape")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().pa_decode_varlen(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                   _ptr(context_lens), _ptr(cu_seqlens_q), q.shape[0],
                                   int(max_q_len), 1 if causal else 0, float(scale), _ptr(out),
                                   _ptr(lse), ctypes.byref(sh), _ptr(workspace), ws_bytes,
                                   _stream(stream)), "pa_decode_varlen")

# ---------------------------------------------------------------------------
# speculative decoding with a tree of drafted tokens
# ---------------------------------------------------------------------------

def _here(*tensors):
    """All tensors on the current CUDA device: the library works on it alone."""
    now = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.device.index != now:
            raise ValueError(f"tensor on {t.device}, but the current CUDA device is {now}")


def _max_q_len(max_q_len, num_words):
    if not 0 <= int(max_q_len) <= 32 * num_words:
        raise ValueError(f"max_q_len {max_q_len} needs 0 .. 32 * mask words ({32 * num_words})")
    return int(max_q_len)


def prepare_tree_mask(parents, cu_seqlens_q, max_q_len, tree_mask, depths=None, stream=None):
    """pa_tree_mask with its arguments checked and marshalled now (see
    prepare_decode)."""
    _need(parents, "parents", torch.int32, 1)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(tree_mask, "tree_mask", torch.int32, 2)
    if depths is not None:
        _need(depths, "depths", torch.int32, 1)
        if depths.shape != parents.shape:
            raise ValueError("depths shape != parents shape")
    if tree_mask.shape[0] != parents.shape[0]:
        raise ValueError("tree_mask rows != number of tokens")
    if cu_seqlens_q.shape[0] < 1:
        raise ValueError("cu_seqlens_q needs num_seqs + 1 entries")
    _here(parents, cu_seqlens_q, tree_mask, depths)
    words = tree_mask.shape[1]
    args = (_ptr(parents), _ptr(cu_seqlens_q), ctypes.c_int(cu_seqlens_q.shape[0] - 1),
            ctypes.c_int64(parents.shape[0]), ctypes.c_int(_max_q_len(max_q_len, words)),
            _ptr(tree_mask), ctypes.c_int(words), _ptr(depths))
    keep = (parents, cu_seqlens_q, tree_mask, depths)
    return _prepared(load().pa_tree_mask, args, stream, "pa_tree_mask", keep)


def pa_tree_mask(parents, cu_seqlens_q, max_q_len, tree_mask, depths=None, stream=None) -> None:
    """Ancestor bits of a window's tokens from their parents: parents [Tq] int32
    (-1: follows the cached context), tree_mask [Tq, words] int32 (bit patterns),
    depths [Tq] int32."""
    prepare_tree_mask(parents, cu_seqlens_q, max_q_len, tree_mask, depths, stream)()


def pa_decode_tree_workspace_size(shape: pa_shape, num_q_tokens: int, max_q_len: int) -> int:
    return int(load().pa_decode_tree_workspace_size(ctypes.byref(shape), int(num_q_tokens),
                                                    int(max_q_len)))


def prepare_decode_tree(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, tree_mask,
                        max_q_len, scale, out, lse=None, workspace=None, stream=None):
    """pa_decode_tree with its arguments checked and marshalled now (see
    prepare_decode)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(tree_mask, "tree_mask", torch.int32, 2)
    _need(out, "out", torch.bfloat16, 3)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
        if lse.shape != q.shape[:2]:
            raise ValueError("lse shape != q rows x heads")
    if k_cache.shape != v_cache.shape:
        raise ValueError("k / v cache shapes differ")
    sh = shape_of(q, k_cache, block_tables)
    if q.shape[2] != sh.head_dim:
        raise ValueError("q head_dim != the cache's")
    if context_lens.shape[0] != sh.num_seqs or cu_seqlens_q.shape[0] != sh.num_seqs + 1:
        raise ValueError("context_lens / cu_seqlens_q length mismatch")
    if out.shape != q.shape:
        raise ValueError("out shape != q shape")
    if tree_mask.shape[0] != q.shape[0]:
        raise ValueError("tree_mask rows != number of query tokens")
    _here(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, tree_mask, out, lse,
          workspace)
    words = tree_mask.shape[1]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
            _ptr(cu_seqlens_q), _ptr(tree_mask), ctypes.c_int(words),
            ctypes.c_int64(q.shape[0]), ctypes.c_int(_max_q_len(max_q_len, words)),
            ctypes.c_float(scale), _ptr(out), _ptr(lse), ctypes.byref(sh), _ptr(workspace),
            ctypes.c_size_t(ws_bytes))
    keep = (q, k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, tree_mask, out, lse,
            workspace, sh)
    return _prepared(load().pa_decode_tree, args, stream, "pa_decode_tree", keep)


def pa_decode_tree(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, tree_mask,
                   max_q_len, scale, out, lse=None, workspace=None, stream=None) -> None:
    """Attention for a window whose queries see the cached context before it and
    the window keys of their mask row (pa_tree_mask)."""
    prepare_decode_tree(q, k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, tree_mask,
                        max_q_len, scale, out, lse, workspace, stream)()


def _pool_pair(k_cache, v_cache):
    """Checks of a pool pair whose rows are moved; its format."""
    if k_cache.dim() == 3:
        _need(k_cache, "k_cache", torch.uint8, 3)
        _need(v_cache, "v_cache", torch.uint8, 3)
        fmt = PA_KV_INT8  # the FP8 pool's rows are the same bytes
    else:
        _need(k_cache, "k_cache", torch.bfloat16, 4)
        _need(v_cache, "v_cache", torch.bfloat16, 4)
        fmt = PA_KV_BF16
    if k_cache.shape != v_cache.shape:
        raise ValueError("k / v cache shapes differ")
    return fmt


def _pool_shape(k_cache, block_tables) -> pa_shape:
    """shape_of for calls without queries (one query head per KV head)."""
    return shape_of(torch.empty((0, k_cache.shape[1], 0)), k_cache, block_tables)


def prepare_commit_path(k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, path,
                        path_lens, new_lens, stream=None):
    """pa_commit_path with its arguments checked and marshalled now (see
    prepare_decode)."""
    fmt = _pool_pair(k_cache, v_cache)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(path, "path", torch.int32, 2)
    _need(path_lens, "path_lens", torch.int32, 1)
    _need(new_lens, "new_lens", torch.int32, 1)
    sh = _pool_shape(k_cache, block_tables)
    S = sh.num_seqs
    if (context_lens.shape[0] != S or path.shape[0] != S or path_lens.shape[0] != S or
            new_lens.shape[0] != S or cu_seqlens_q.shape[0] != S + 1):
        raise ValueError("a per-sequence tensor does not have one entry per sequence")
    _here(k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, path, path_lens, new_lens)
    args = (_ptr(k_cache), _ptr(v_cache), ctypes.c_int(fmt), _ptr(block_tables),
            _ptr(context_lens), _ptr(cu_seqlens_q), _ptr(path), _ptr(path_lens),
            ctypes.c_int(path.shape[1]), _ptr(new_lens), ctypes.byref(sh))
    keep = (k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, path, path_lens,
            new_lens, sh)
    return _prepared(load().pa_commit_path, args, stream, "pa_commit_path", keep)


def pa_commit_path(k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, path, path_lens,
                   new_lens, stream=None) -> None:
    """Move the accepted path's cached rows to the front of their window: path
    [S, max_path] int32 increasing window indices, path_lens [S]; new_lens [S]
    receives context_len - Lq + path_len (it may be context_lens itself)."""
    prepare_commit_path(k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, path,
                        path_lens, new_lens, stream)()


# ---------------------------------------------------------------------------
# eviction by accumulated attention weight
# ---------------------------------------------------------------------------

def prepare_accumulate_weights(q, k_cache, lse, block_tables, context_lens, scale, weights,
                               cu_seqlens_q=None, max_q_len: int = 1, accumulate: bool = True,
                               kv_format: int | None = None, stream=None):
    """pa_accumulate_weights with its arguments checked and marshalled now (see
    prepare_decode)."""
    _need(q, "q", torch.bfloat16, 3)
    if k_cache.dim() == 3:
        _need(k_cache, "k_cache", torch.uint8, 3)
        if kv_format not in (PA_KV_INT8, PA_KV_FP8):
            raise ValueError("an 8-bit pool needs kv_format PA_KV_INT8 or PA_KV_FP8")
    else:
        _need(k_cache, "k_cache", torch.bfloat16, 4)
        if kv_format not in (None, PA_KV_BF16):
            raise ValueError("a bf16 pool has kv_format PA_KV_BF16")
        kv_format = PA_KV_BF16
    _need(lse, "lse", torch.float32, 2)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(weights, "weights", torch.float32, 3)
    sh = shape_of(q, k_cache, block_tables)
    if q.shape[2] != sh.head_dim:
        raise ValueError("q head_dim != the cache's")
    if lse.shape != q.shape[:2]:
        raise ValueError("lse shape != q rows x heads")
    if context_lens.shape[0] != sh.num_seqs:
        raise ValueError("context_lens length != number of sequences")
    if weights.shape[:2] != (sh.num_seqs, sh.num_kv_heads):
        raise ValueError("weights must be [num_seqs, num_kv_heads, positions]")
    if cu_seqlens_q is None:
        if q.shape[0] != sh.num_seqs:
            raise ValueError("without cu_seqlens_q there is one query per sequence")
    else:
        _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
        if cu_seqlens_q.shape[0] != sh.num_seqs + 1:
            raise ValueError("cu_seqlens_q needs num_seqs + 1 entries")
    _here(q, k_cache, lse, block_tables, context_lens, weights, cu_seqlens_q)
    args = (_ptr(q), _ptr(k_cache), ctypes.c_int(kv_format), _ptr(lse), _ptr(block_tables),
            _ptr(context_lens), _ptr(cu_seqlens_q), ctypes.c_int64(q.shape[0]),
            ctypes.c_int(int(max_q_len)), ctypes.c_float(scale),
            ctypes.c_int(1 if accumulate else 0), _ptr(weights),
            ctypes.c_int64(weights.shape[2]), ctypes.byref(sh))
    keep = (q, k_cache, lse, block_tables, context_lens, weights, cu_seqlens_q, sh)
    return _prepared(load().pa_accumulate_weights, args, stream, "pa_accumulate_weights", keep)


def pa_accumulate_weights(q, k_cache, lse, block_tables, context_lens, scale, weights,
                          cu_seqlens_q=None, max_q_len: int = 1, accumulate: bool = True,
                          kv_format: int | None = None, stream=None) -> None:
    """Attention weight that each cached position draws from these queries, added
    to weights [S, Hkv, positions] fp32 (or written: accumulate=False); lse is
    what the attention call over the same queries returned."""
    prepare_accumulate_weights(q, k_cache, lse, block_tables, context_lens, scale, weights,
                               cu_seqlens_q, max_q_len, accumulate, kv_format, stream)()


def prepare_evict(k_cache, v_cache, block_tables, context_lens, weights, budgets, num_sinks,
                  num_recent, kept, new_lens, stream=None):
    """pa_evict with its arguments checked and marshalled now (see
    prepare_decode)."""
    fmt = _pool_pair(k_cache, v_cache)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(weights, "weights", torch.float32, 3)
    _need(budgets, "budgets", torch.int32, 1)
    _need(kept, "kept", torch.int32, 3)
    _need(new_lens, "new_lens", torch.int32, 1)
    sh = _pool_shape(k_cache, block_tables)
    S = sh.num_seqs
    if context_lens.shape[0] != S or budgets.shape[0] != S or new_lens.shape[0] != S:
        raise ValueError("a per-sequence tensor does not have one entry per sequence")
    if weights.shape[:2] != (S, sh.num_kv_heads):
        raise ValueError("weights must be [num_seqs, num_kv_heads, positions]")
    if kept.shape[:2] != (S, sh.num_kv_heads):
        raise ValueError("kept must be [num_seqs, num_kv_heads, max_budget]")
    _here(k_cache, v_cache, block_tables, context_lens, weights, budgets, kept, new_lens)
    args = (_ptr(k_cache), _ptr(v_cache), ctypes.c_int(fmt), _ptr(block_tables),
            _ptr(context_lens), _ptr(weights), ctypes.c_int64(weights.shape[2]), _ptr(budgets),
            ctypes.c_int(kept.shape[2]), ctypes.c_int(int(num_sinks)),
            ctypes.c_int(int(num_recent)), _ptr(kept), _ptr(new_lens), ctypes.byref(sh))
    keep = (k_cache, v_cache, block_tables, context_lens, weights, budgets, kept, new_lens, sh)
    return _prepared(load().pa_evict, args, stream, "pa_evict", keep)


def pa_evict(k_cache, v_cache, block_tables, context_lens, weights, budgets, num_sinks,
             num_recent, kept, new_lens, stream=None) -> None:
    """Shrink each sequence's cache to budgets[s] positions per KV head: the
    first num_sinks, the last num_recent and the heaviest between them stay and
    move together in order, with their weights. kept [S, Hkv, max_budget]
    receives their old positions, new_lens [S] the new lengths."""
    prepare_evict(k_cache, v_cache, block_tables, context_lens, weights, budgets, num_sinks,
                  num_recent, kept, new_lens, stream)()


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

ROTATION_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}


def make_rotation(rot_dim: int = 128, interleaved: bool = False, base: float = 10000.0,
                  scaling: str = "none", factor: float = 1.0, original_len: float = 0.0,
                  low: float = 1.0, high: float = 4.0) -> pa_rotation:
    """A rotary-position map of a head's first rot_dim dimensions, pairs (i, i +
    rot_dim/2) or (2i, 2i+1), with angles base^(-2i/rot_dim) per position.
    scaling: "none", "linear", "base", "bands" or "ramp", for contexts that are
    `factor` times the original_len tokens of training; bands and ramp change
    between pairs that make `low` and `high` turns over that length."""
    if scaling not in ROTATION_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROTATION_SCALINGS)}, got {scaling!r}")
    rot = pa_rotation()
    _check(load().pa_rotation_init(ctypes.byref(rot), int(rot_dim), 1 if interleaved else 0,
                                   float(base), ROTATION_SCALINGS[scaling], float(factor),
                                   float(original_len), float(low), float(high)),
           "pa_rotation_init")
    return rot


def make_rotation_from(radians, interleaved: bool = False, magnitude: float = 1.0) -> pa_rotation:
    """A rotary-position map from the angles per position of its rot_dim/2 pairs
    (numbers, or a CPU tensor)."""
    values = [float(x) for x in radians]
    rot = pa_rotation()
    _check(load().pa_rotation_set(ctypes.byref(rot), 2 * len(values), 1 if interleaved else 0,
                                  (ctypes.c_double * max(1, len(values)))(*values),
                                  float(magnitude)), "pa_rotation_set")
    return rot


def _row_view(x, name):
    """[tokens, heads, head_dim] bf16 with any token and head strides."""
    if x is None:
        raise ValueError(f"{name} is required")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {x.dtype}")
    if x.dim() != 3:
        raise ValueError(f"{name} must have 3 dims, got {x.dim()}")
    if x.shape[2] > 1 and x.stride(2) != 1:
        raise ValueError(f"{name} must hold a head's values side by side")
    # (the stride of an axis of one entry says nothing)
    return pa_row_view(x.data_ptr(), x.stride(0) if x.shape[0] > 1 else 0,
                       x.stride(1) if x.shape[1] > 1 else 0)


def _rotation(rot):
    """A copy of the caller's map: a prepared call keeps what it was made with."""
    if not isinstance(rot, pa_rotation):
        raise TypeError("rotation must be a pa_rotation (make_rotation)")
    return pa_rotation.from_buffer_copy(rot)


def prepare_rotate(x, positions, rotation, y, transpose: bool = False, stream=None):
    """pa_rotate with its arguments checked and marshalled now (see
    prepare_decode)."""
    xv, yv = _row_view(x, "x"), _row_view(y, "y")
    _need(positions, "positions", torch.int32, 1)
    if y.shape != x.shape:
        raise ValueError("y shape != x shape")
    if positions.shape[0] != x.shape[0]:
        raise ValueError("positions length != number of tokens")
    _here(x, positions, y)
    rot = _rotation(rotation)
    args = (ctypes.byref(xv), _ptr(positions), ctypes.c_int64(x.shape[0]),
            ctypes.c_int(x.shape[1]), ctypes.c_int(x.shape[2]), ctypes.byref(rot),
            ctypes.c_int(1 if transpose else 0), ctypes.byref(yv))
    keep = (x, positions, y, xv, yv, rot)
    return _prepared(load().pa_rotate, args, stream, "pa_rotate", keep)


def pa_rotate(x, positions, rotation, y, transpose: bool = False, stream=None) -> None:
    """y = x [T, H, 128] with row t of every head rotated by positions[t] (int32);
    y may be x. transpose: the transposed map, the gradient of the rotation."""
    prepare_rotate(x, positions, rotation, y, transpose, stream)()


def _kv_format(k_cache, kv_format):
    """The format of a pool array: 8-bit tiles do not tell int8 from FP8."""
    if k_cache.dim() == 3:
        _need(k_cache, "k_cache", torch.uint8, 3)
        if kv_format not in (PA_KV_INT8, PA_KV_FP8):
            raise ValueError("an 8-bit pool needs kv_format PA_KV_INT8 or PA_KV_FP8")
        return kv_format
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    if kv_format not in (None, PA_KV_BF16):
        raise ValueError("a bf16 pool has kv_format PA_KV_BF16")
    return PA_KV_BF16


def prepare_rotate_and_cache(k, v, positions, slot_mapping, rotation, k_cache, v_cache, q=None,
                             q_out=None, kv_format: int | None = None, stream=None):
    """pa_rotate_and_cache with its arguments checked and marshalled now (see
    prepare_decode)."""
    kv, vv = _row_view(k, "k"), _row_view(v, "v")
    _need(positions, "positions", torch.int32, 1)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    fmt = _kv_format(k_cache, kv_format)
    _need(v_cache, "v_cache", k_cache.dtype, k_cache.dim())
    if k.shape != v.shape or k_cache.shape != v_cache.shape:
        raise ValueError("k/v or cache shapes differ")
    T = k.shape[0]
    if positions.shape[0] != T or slot_mapping.shape[0] != T:
        raise ValueError("positions / slot_mapping length != number of tokens")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    qv = ov = None
    if q is not None:
        qv, ov = _row_view(q, "q"), _row_view(q_out, "q_out")
        if q.shape[0] != T or q_out.shape != q.shape:
            raise ValueError("q / q_out rows != number of tokens")
    sh = shape_of(k if q is None else q, k_cache, torch.empty((0, 0)))
    if k.shape[1:] != (sh.num_kv_heads, sh.head_dim):
        raise ValueError("k rows do not match the cache's [Hkv, D]")
    if q is not None and q.shape[2] != sh.head_dim:
        raise ValueError("q head_dim != the cache's")
    _here(k, v, positions, slot_mapping, k_cache, v_cache, q, q_out)
    rot = _rotation(rotation)
    args = (ctypes.byref(qv) if qv else None, ctypes.byref(kv), ctypes.byref(vv),
            _ptr(positions), _ptr(slot_mapping), ctypes.c_int64(T), ctypes.byref(rot),
            ctypes.byref(ov) if ov else None, _ptr(k_cache), _ptr(v_cache), ctypes.c_int(fmt),
            ctypes.byref(sh))
    keep = (k, v, positions, slot_mapping, k_cache, v_cache, q, q_out, qv, kv, vv, ov, rot, sh)
    return _prepared(load().pa_rotate_and_cache, args, stream, "pa_rotate_and_cache", keep)


def pa_rotate_and_cache(k, v, positions, slot_mapping, rotation, k_cache, v_cache, q=None,
                        q_out=None, kv_format: int | None = None, stream=None) -> None:
    """A step's rows into the cache with the rotation on the way: k [T, Hkv, 128]
    rotated by positions [T] int32 and v as it is go to their slots, q
    [T, Hq, 128] rotated goes to q_out (which may be q)."""
    prepare_rotate_and_cache(k, v, positions, slot_mapping, rotation, k_cache, v_cache, q, q_out,
                             kv_format, stream)()


def prepare_rotate_cached(k_cache, block_tables, context_lens, rotation, shifts=None, kept=None,
                          first: int = 0, kv_format: int | None = None, stream=None):
    """pa_rotate_cached with its arguments checked and marshalled now (see
    prepare_decode)."""
    fmt = _kv_format(k_cache, kv_format)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    sh = _pool_shape(k_cache, block_tables)
    S = sh.num_seqs
    if context_lens.shape[0] != S:
        raise ValueError("context_lens length != number of sequences")
    if (shifts is None) == (kept is None):
        raise ValueError("one of shifts and kept is needed")
    if shifts is not None:
        _need(shifts, "shifts", torch.int32, 1)
        if shifts.shape[0] != S:
            raise ValueError("shifts length != number of sequences")
    else:
        _need(kept, "kept", torch.int32, 3)
        if kept.shape[:2] != (S, sh.num_kv_heads):
            raise ValueError("kept must be [num_seqs, num_kv_heads, positions]")
        if first:
            raise ValueError("first goes with shifts")
    _here(k_cache, block_tables, context_lens, shifts, kept)
    rot = _rotation(rotation)
    args = (_ptr(k_cache), ctypes.c_int(fmt), _ptr(block_tables), _ptr(context_lens),
            _ptr(shifts), ctypes.c_int(int(first)), _ptr(kept),
            ctypes.c_int(0 if kept is None else kept.shape[2]), ctypes.byref(rot),
            ctypes.byref(sh))
    keep = (k_cache, block_tables, context_lens, shifts, kept, rot, sh)
    return _prepared(load().pa_rotate_cached, args, stream, "pa_rotate_cached", keep)


def pa_rotate_cached(k_cache, block_tables, context_lens, rotation, shifts=None, kept=None,
                     first: int = 0, kv_format: int | None = None, stream=None) -> None:
    """Turn cached keys on to new positions, in place: by shifts [S] int32 from
    position `first` on, or each from the position kept [S, Hkv, n] int32
    (pa_evict) to the one it has now."""
    prepare_rotate_cached(k_cache, block_tables, context_lens, rotation, shifts, kept, first,
                          kv_format, stream)()


# ---------------------------------------------------------------------------
# differential attention
# ---------------------------------------------------------------------------

def pa_decode_diff_workspace_size(shape: pa_shape, num_q_tokens: int, max_q_len: int = 1) -> int:
    return int(load().pa_decode_diff_workspace_size(ctypes.byref(shape), int(num_q_tokens),
                                                    int(max_q_len)))


def prepare_decode_diff(q, k_cache, v_cache, block_tables, context_lens, scale, lambdas, out,
                        lse=None, cu_seqlens_q=None, max_q_len: int = 1, causal: bool = True,
                        norm_weight=None, norm_eps: float = 1e-5, out_scale: float = 1.0,
                        workspace=None, stream=None):
    """pa_decode_diff with its arguments checked and marshalled now (see
    prepare_decode)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(lambdas, "lambdas", torch.float32, 1)
    _need(out, "out", torch.bfloat16, 3)
    if k_cache.shape != v_cache.shape:
        raise ValueError("k / v cache shapes differ")
    sh = shape_of(q, k_cache, block_tables)
    T, Hq, D = q.shape
    if D != sh.head_dim:
        raise ValueError("q head_dim != the cache's")
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
        if lse.shape != (T, Hq):
            raise ValueError("lse shape != q rows x heads")
    if Hq % 2 or lambdas.shape[0] != Hq // 2:
        raise ValueError("lambdas must have one entry per two query heads")
    if out.shape != (T, Hq // 2, 2 * D):
        raise ValueError("out must be [tokens, query heads / 2, 2 * head_dim]")
    if norm_weight is not None:
        _need(norm_weight, "norm_weight", torch.float32, 1)
        if norm_weight.shape[0] != 2 * D:
            raise ValueError("norm_weight must have 2 * head_dim entries")
    if context_lens.shape[0] != sh.num_seqs:
        raise ValueError("context_lens length != number of sequences")
    if cu_seqlens_q is None:
        if T != sh.num_seqs or int(max_q_len) != 1:
            raise ValueError("without cu_seqlens_q there is one query per sequence")
    else:
        _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
        if cu_seqlens_q.shape[0] != sh.num_seqs + 1:
            raise ValueError("cu_seqlens_q needs num_seqs + 1 entries")
    _here(q, k_cache, v_cache, block_tables, context_lens, lambdas, out, lse, cu_seqlens_q,
          norm_weight, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
            _ptr(cu_seqlens_q), ctypes.c_int64(T), ctypes.c_int(int(max_q_len)),
            ctypes.c_int(1 if causal else 0), ctypes.c_float(scale), _ptr(lambdas),
            _ptr(norm_weight), ctypes.c_float(norm_eps), ctypes.c_float(out_scale), _ptr(out),
            _ptr(lse), ctypes.byref(sh), _ptr(workspace), ctypes.c_size_t(ws_bytes))
    keep = (q, k_cache, v_cache, block_tables, context_lens, lambdas, out, lse, cu_seqlens_q,
            norm_weight, workspace, sh)
    return _prepared(load().pa_decode_diff, args, stream, "pa_decode_diff", keep)


def pa_decode_diff(q, k_cache, v_cache, block_tables, context_lens, scale, lambdas, out, lse=None,
                   cu_seqlens_q=None, max_q_len: int = 1, causal: bool = True, norm_weight=None,
                   norm_eps: float = 1e-5, out_scale: float = 1.0, workspace=None,
                   stream=None) -> None:
    """Differential attention: head p*G+g of out [T, Hq/2, 256] is the attention of
    query head 2p*G+g over KV head 2p's keys minus lambdas[p*G+g] times that of
    query head (2p+1)*G+g over KV head 2p+1's, both over the two heads' values side
    by side, then (norm_weight) normed by its root mean square, times out_scale."""
    prepare_decode_diff(q, k_cache, v_cache, block_tables, context_lens, scale, lambdas, out, lse,
                        cu_seqlens_q, max_q_len, causal, norm_weight, norm_eps, out_scale,
                        workspace, stream)()


def pa_splitk_reduce(part_out, part_lse, out, lse=None, stream=None) -> None:
    """part_out [rows, heads, P, D] fp32, part_lse [rows, heads, P] fp32 ->
    out [rows, heads, D] bf16, lse [rows, heads] fp32."""
    _need(part_out, "part_out", torch.float32, 4)
    _need(part_lse, "part_lse", torch.float32, 3)
    _need(out, "out", torch.bfloat16, 3)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    R, H, P, D = part_out.shape
    if part_lse.shape != (R, H, P) or out.shape != (R, H, D):
        raise ValueError("split-K shapes disagree")
    _check(load().pa_splitk_reduce(_ptr(part_out), _ptr(part_lse), R, H, P, D, _ptr(out),
                                   _ptr(lse), _stream(stream)), "pa_splitk_reduce")


# ---------------------------------------------------------------------------
# workspace convenience
# ---------------------------------------------------------------------------

def workspace(nbytes: int, device=None):
    """A device byte buffer of at least nbytes (256-byte aligned by torch's
    allocator), or None when nbytes is 0."""
    if nbytes <= 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
