"""Paged KV cache write and paged attention for GB300 (sm_103a).

A thin binding over the C ABI in ``include/pkv.h`` (``libpkv.so``, built
in-tree by ``paged_kv_cache_write_gb300.build``): ctypes, and for the norm,
rotation and 4-bit entries a CPython extension.  Each function here
has the name of the C entry point without its ``pkv_`` prefix and only
marshals arguments: it checks tensor devices, dtypes and layouts, passes
raw device pointers and the current CUDA stream, and raises on a non-zero
status.  Every step of the computation runs in the library's CUDA kernels;
there is no CPU or PyTorch fallback: the library is loaded on first use
and every call raises ImportError if it has not been built.

PyTorch is used only for device memory and streams.
"""
from __future__ import annotations

import ctypes
import importlib
import os

import torch

__all__ = [
    "lib", "library_path", "PoolDesc", "PKV_F32", "PKV_BF16", "DEVERR",
    "slot_mapping", "kv_write", "kv_gather", "copy_blocks", "decode_workspace_bytes",
    "paged_attention_decode", "paged_attention_decode_append",
    "decode_shared_prefix_workspace_bytes", "paged_attention_decode_shared_prefix",
    "decode_plan", "paged_attention_decode_planned", "prefill_workspace_bytes",
    "paged_attention_prefill", "status_string", "abi_version", "paged_attention_decode_noalloc",
    "selftest_bounded_wait", "PKV_FP8_E4M3", "kv_write_fp8", "kv_gather_fp8",
    "decode_fp8_workspace_bytes", "paged_attention_decode_fp8", "paged_attention_prefill_fp8",
    "selftest_bounded_wait_fp8", "PKV_FP4_E2M1", "NormRopeDesc", "qk_norm_rope",
    "qk_norm_rope_write", "qk_norm_rope_write_fp4", "kv_write_fp4", "kv_gather_fp4",
    "decode_fp4_workspace_bytes", "paged_attention_decode_fp4", "paged_attention_prefill_fp4",
]

HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(HERE, "libpkv.so")

PKV_F32 = 0
PKV_BF16 = 1
PKV_FP8_E4M3 = 2
PKV_FP4_E2M1 = 3
DEVERR = {"block_id": 1, "slot": 2, "table_width": 4, "length": 8, "timeout": 16, "prefix": 32,
          "plan": 64, "scale": 128}


class PoolDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("n_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class NormRopeDesc(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("num_positions", ctypes.c_int32), ("cos_sin", ctypes.c_void_p),
                ("positions", ctypes.c_void_p)]


_lib = None
_p = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t
_f = ctypes.c_float
_desc = ctypes.POINTER(PoolDesc)
_turn = ctypes.POINTER(NormRopeDesc)


def _load():
    """Load libpkv.so once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise ImportError(
            f"{library_path} is missing: build it with "
            "`python -m paged_kv_cache_write_gb300.build` (needs nvcc with sm_103a support)")
    L = ctypes.CDLL(library_path)
    L.pkv_status_string.restype = ctypes.c_char_p
    L.pkv_status_string.argtypes = [_i32]
    L.pkv_abi_version.restype = _i32
    L.pkv_abi_version.argtypes = []
    L.pkv_slot_mapping.restype = _i32
    L.pkv_slot_mapping.argtypes = [_p, _i32, _p, _p, _i32, _i32, _i32, _i32, _p, _p, _p]
    L.pkv_kv_write.restype = _i32
    L.pkv_kv_write.argtypes = [_p, _p, _p, _i32, _p, _p, _desc, _p, _p]
    L.pkv_selftest_bounded_wait.restype = _i32
    L.pkv_selftest_bounded_wait.argtypes = [_i32, _p, _p]
    L.pkv_copy_blocks.restype = _i32
    L.pkv_copy_blocks.argtypes = [_p, _p, _desc, _p, _i32, _p, _p]
    L.pkv_kv_gather.restype = _i32
    L.pkv_kv_gather.argtypes = [_p, _p, _desc, _p, _i32, _p, _p, _i32, _i32, _p, _p, _p, _p]
    L.pkv_decode_workspace_bytes.restype = _sz
    L.pkv_decode_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
    L.pkv_paged_attention_decode.restype = _i32
    L.pkv_paged_attention_decode.argtypes = [_p, _i32, _i32, _p, _p, _desc, _p, _i32, _p, _i32,
                                             _f, _i32, _p, _p, _sz, _p, _p]
    L.pkv_decode_shared_prefix_workspace_bytes.restype = _sz
    L.pkv_decode_shared_prefix_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, _i32]
    L.pkv_paged_attention_decode_shared_prefix.restype = _i32
    L.pkv_paged_attention_decode_shared_prefix.argtypes = [_p, _i32, _i32, _p, _p, _desc, _p, _i32,
                                                           _p, _i32, _i32, _f, _i32, _p, _p, _sz,
                                                           _p, _p]
    L.pkv_paged_attention_decode_append.restype = _i32
    L.pkv_paged_attention_decode_append.argtypes = [_p, _p, _p, _i32, _i32, _p, _p, _desc, _p,
                                                    _i32, _p, _i32, _f, _i32, _p, _p, _sz, _p, _p]
    L.pkv_decode_plan.restype = _i32
    L.pkv_decode_plan.argtypes = [_i32, _i32, _desc, _i32, _p, _i32, _i32, _i32, _p, _sz, _p, _p]
    L.pkv_paged_attention_decode_planned.restype = _i32
    L.pkv_paged_attention_decode_planned.argtypes = [_p, _p, _p, _i32, _i32, _p, _p, _desc, _p,
                                                     _i32, _p, _i32, _i32, _f, _i32, _p, _p, _sz,
                                                     _p, _p]
    L.pkv_prefill_workspace_bytes.restype = _sz
    L.pkv_prefill_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32]
    L.pkv_paged_attention_prefill.restype = _i32
    L.pkv_paged_attention_prefill.argtypes = [_p, _p, _i32, _i32, _i32, _i32, _p, _p, _desc, _p,
                                              _i32, _p, _i32, _f, _p, _p, _sz, _p, _p]
    L.pkv_selftest_bounded_wait_fp8.restype = _i32
    L.pkv_selftest_bounded_wait_fp8.argtypes = [_i32, _p, _p]
    L.pkv_kv_write_fp8.restype = _i32
    L.pkv_kv_write_fp8.argtypes = [_p, _p, _i32, _p, _i32, _p, _p, _i32, _i32, _p, _p, _p, _p, _desc,
                                   _p, _p]
    L.pkv_kv_gather_fp8.restype = _i32
    L.pkv_kv_gather_fp8.argtypes = [_p, _p, _p, _p, _desc, _p, _i32, _p, _p, _i32, _i32, _i32, _p,
                                    _p, _p, _p]
    L.pkv_decode_fp8_workspace_bytes.restype = _sz
    L.pkv_decode_fp8_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
    L.pkv_paged_attention_decode_fp8.restype = _i32
    L.pkv_paged_attention_decode_fp8.argtypes = [_p, _i32, _i32, _i32, _p, _p, _p, _p, _desc, _p,
                                                 _i32, _p, _i32, _f, _i32, _p, _p, _sz, _p, _p]
    L.pkv_paged_attention_prefill_fp8.restype = _i32
    L.pkv_paged_attention_prefill_fp8.argtypes = [_p, _i32, _p, _i32, _i32, _i32, _i32, _p, _p, _p,
                                                  _p, _desc, _p, _i32, _p, _i32, _f, _p, _p, _p]
    L.pkv_qk_norm_rope.restype = _i32
    L.pkv_qk_norm_rope.argtypes = [_p, _i64, _p, _i64, _i32, _i32, _i32, _i32, _i32, _turn, _p, _i64,
                                   _p, _i64, _p, _p]
    L.pkv_qk_norm_rope_write.restype = _i32
    L.pkv_qk_norm_rope_write.argtypes = [_p, _i64, _p, _i64, _p, _i64, _i32, _i32, _turn, _p, _i64, _p,
                                         _p, _p, _desc, _p, _p]
    L.pkv_qk_norm_rope_write_fp4.restype = _i32
    L.pkv_qk_norm_rope_write_fp4.argtypes = [_p, _i64, _p, _i64, _p, _i64, _i32, _i32, _i32, _turn, _p,
                                             _i64, _p, _p, _p, _p, _p, _p, _p, _desc, _p, _p]
    L.pkv_kv_write_fp4.restype = _i32
    L.pkv_kv_write_fp4.argtypes = [_p, _i64, _p, _i64, _i32, _p, _i32, _p, _p, _p, _p, _p, _p, _desc,
                                   _p, _p]
    L.pkv_kv_gather_fp4.restype = _i32
    L.pkv_kv_gather_fp4.argtypes = [_p, _p, _p, _p, _p, _p, _desc, _p, _i32, _p, _p, _i32, _i32, _i32,
                                    _p, _p, _p, _p]
    L.pkv_decode_fp4_workspace_bytes.restype = _sz
    L.pkv_decode_fp4_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32]
    L.pkv_paged_attention_decode_fp4.restype = _i32
    L.pkv_paged_attention_decode_fp4.argtypes = [_p, _i32, _i32, _i32, _p, _p, _p, _p, _p, _p, _desc,
                                                 _p, _i32, _p, _i32, _f, _i32, _p, _p, _sz, _p, _p]
    L.pkv_paged_attention_prefill_fp4.restype = _i32
    L.pkv_paged_attention_prefill_fp4.argtypes = [_p, _i32, _p, _i32, _i32, _i32, _i32, _p, _p, _p, _p,
                                                  _p, _p, _desc, _p, _i32, _p, _i32, _f, _p, _p, _p]
    _lib = L
    return L


def __getattr__(name):
    # `pkv.lib` loads the library on first access
    if name == "lib":
        return _load()
    raise AttributeError(name)


def status_string(status: int) -> str:
    return _load().pkv_status_string(int(status)).decode()


def abi_version() -> int:
    return int(_load().pkv_abi_version())


class PkvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


def _check(fn: str, status: int):
    if status != 0:
        raise PkvError(fn, status)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return PKV_F32
    if t == torch.bfloat16:
        return PKV_BF16
    raise TypeError(f"unsupported dtype {t}: float32 or bfloat16")


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _opt(t, name, dtype=None):
    return None if t is None else _dev(t, name, dtype)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def pool_desc(k_pool: torch.Tensor) -> PoolDesc:
    if k_pool.dim() != 4:
        raise ValueError("pool must be [num_blocks, block_size, n_kv, head_dim]")
    nb, bs, nkv, hd = k_pool.shape
    return PoolDesc(nb, bs, nkv, hd, _dtype_code(k_pool.dtype))


def slot_mapping(block_tables, seq_lens, cu_new_lens, num_tokens: int, block_size: int,
                 num_blocks: int, *, out=None, err=None, stream=None):
    """int64 [num_tokens] flat pool slot of each token written this step."""
    B, W = block_tables.shape
    if out is None:
        out = torch.empty(num_tokens, dtype=torch.int64, device=block_tables.device)
    _check("pkv_slot_mapping", _load().pkv_slot_mapping(
        _dev(block_tables, "block_tables", torch.int32), W, _dev(seq_lens, "seq_lens", torch.int32),
        _dev(cu_new_lens, "cu_new_lens", torch.int32), B, int(num_tokens), int(block_size),
        int(num_blocks), _dev(out, "out", torch.int64), _opt(err, "err", torch.int32),
        _stream(stream)))
    return out


def kv_write(k, v, slot_mapping, k_pool, v_pool, *, err=None, stream=None):
    """Scatter k/v [T, n_kv, head_dim] into the pools at slot_mapping [T]."""
    desc = pool_desc(k_pool)
    if tuple(v_pool.shape) != tuple(k_pool.shape) or v_pool.dtype != k_pool.dtype:
        raise ValueError("k_pool and v_pool must have the same shape and dtype")
    T = k.shape[0]
    if tuple(k.shape) != (T, desc.n_kv, desc.head_dim) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k, v must be [T, n_kv, head_dim] matching the pool")
    if slot_mapping.shape[0] != T:
        raise ValueError("slot_mapping must have one entry per token")
    _check("pkv_kv_write", _load().pkv_kv_write(
        _dev(k, "k", k_pool.dtype), _dev(v, "v", k_pool.dtype),
        _dev(slot_mapping, "slot_mapping", torch.int64), T, _dev(k_pool, "k_pool"),
        _dev(v_pool, "v_pool"), ctypes.byref(desc), _opt(err, "err", torch.int32),
        _stream(stream)))


def selftest_bounded_wait(err, polls: int = 4096, *, stream=None):
    """Run one wait that nothing completes, bounded by ``polls``; the
    kernel ORs the timeout bit into the device int32 ``err`` and returns."""
    _check("pkv_selftest_bounded_wait", _load().pkv_selftest_bounded_wait(
        int(polls), _dev(err, "err", torch.int32), _stream(stream)))


def copy_blocks(k_pool, v_pool, block_pairs, *, err=None, stream=None):
    """Copy whole blocks of both pools: for each row (src, dst) of the
    int32 [n, 2] ``block_pairs``, block dst becomes a copy of block src
    (copy-on-write).  Destinations must be distinct and not sources."""
    desc = pool_desc(k_pool)
    if block_pairs.dim() != 2 or block_pairs.shape[1] != 2:
        raise ValueError("block_pairs must be [n, 2]")
    _check("pkv_copy_blocks", _load().pkv_copy_blocks(
        _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"), ctypes.byref(desc),
        _dev(block_pairs, "block_pairs", torch.int32), int(block_pairs.shape[0]),
        _opt(err, "err", torch.int32), _stream(stream)))


def kv_gather(k_pool, v_pool, block_tables, seq_lens, cu_seq_lens, total_tokens: int, *,
              k_out=None, v_out=None, err=None, stream=None):
    """Contiguous [total_tokens, n_kv, head_dim] K and V in logical order."""
    desc = pool_desc(k_pool)
    B, W = block_tables.shape
    shape = (int(total_tokens), desc.n_kv, desc.head_dim)
    if k_out is None:
        k_out = torch.empty(shape, dtype=k_pool.dtype, device=k_pool.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=k_pool.dtype, device=k_pool.device)
    _check("pkv_kv_gather", _load().pkv_kv_gather(
        _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"), ctypes.byref(desc),
        _dev(block_tables, "block_tables", torch.int32), W, _dev(seq_lens, "seq_lens", torch.int32),
        _dev(cu_seq_lens, "cu_seq_lens", torch.int32), B, int(total_tokens),
        _dev(k_out, "k_out", k_pool.dtype), _dev(v_out, "v_out", k_pool.dtype),
        _opt(err, "err", torch.int32), _stream(stream)))
    return k_out, v_out


def decode_workspace_bytes(num_seqs, n_heads, head_dim, max_seq_len, max_ctas=0, block_size=16):
    return int(_load().pkv_decode_workspace_bytes(num_seqs, n_heads, head_dim, max_seq_len, max_ctas,
                                              block_size))


def paged_attention_decode(q, k_pool, v_pool, block_tables, seq_lens, scale: float,
                           max_seq_len: int | None = None, *, out=None, workspace=None,
                           max_ctas: int = 0, err=None, stream=None):
    """Decode attention [B, n_heads, head_dim] over the paged history.

    ``max_seq_len`` is a host-side bound on ``seq_lens`` (reading it from
    the device synchronises; pass it when known).  ``workspace`` is a
    device uint8 tensor of at least ``decode_workspace_bytes(...)`` bytes
    (allocated here when omitted).
    """
    desc = pool_desc(k_pool)
    B, H, hd = q.shape
    W = block_tables.shape[1]
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    if out is None:
        out = torch.empty_like(q)
    need = decode_workspace_bytes(B, H, hd, max_seq_len, max_ctas, desc.block_size)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check("pkv_paged_attention_decode", _load().pkv_paged_attention_decode(
        _dev(q, "q", k_pool.dtype), B, H, _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"),
        ctypes.byref(desc), _dev(block_tables, "block_tables", torch.int32), W,
        _dev(seq_lens, "seq_lens", torch.int32), int(max_seq_len), float(scale), int(max_ctas),
        _dev(out, "out", k_pool.dtype), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _opt(err, "err", torch.int32),
        _stream(stream)))
    return out


def decode_shared_prefix_workspace_bytes(num_seqs, n_heads, head_dim, max_seq_len,
                                         shared_prefix_blocks, max_ctas=0, block_size=16):
    return int(_load().pkv_decode_shared_prefix_workspace_bytes(
        num_seqs, n_heads, head_dim, max_seq_len, shared_prefix_blocks, max_ctas, block_size))


def paged_attention_decode_shared_prefix(q, k_pool, v_pool, block_tables, seq_lens, scale: float,
                                         shared_prefix_blocks: int,
                                         max_seq_len: int | None = None, *, out=None,
                                         workspace=None, max_ctas: int = 0, err=None,
                                         stream=None):
    """Decode attention where the first ``shared_prefix_blocks`` table
    entries of every sequence are the same blocks, read once per step."""
    desc = pool_desc(k_pool)
    B, H, hd = q.shape
    W = block_tables.shape[1]
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    if out is None:
        out = torch.empty_like(q)
    need = decode_shared_prefix_workspace_bytes(B, H, hd, max_seq_len, shared_prefix_blocks,
                                                max_ctas, desc.block_size)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check("pkv_paged_attention_decode_shared_prefix",
           _load().pkv_paged_attention_decode_shared_prefix(
               _dev(q, "q", k_pool.dtype), B, H, _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"),
               ctypes.byref(desc), _dev(block_tables, "block_tables", torch.int32), W,
               _dev(seq_lens, "seq_lens", torch.int32), int(max_seq_len),
               int(shared_prefix_blocks), float(scale), int(max_ctas),
               _dev(out, "out", k_pool.dtype), _dev(workspace, "workspace"),
               workspace.numel() * workspace.element_size(), _opt(err, "err", torch.int32),
               _stream(stream)))
    return out


def paged_attention_decode_append(q, k_new, v_new, k_pool, v_pool, block_tables, seq_lens,
                                  scale: float, max_seq_len: int | None = None, *, out=None,
                                  workspace=None, max_ctas: int = 0, err=None, stream=None):
    """Store this step's ``k_new``/``v_new`` [B, n_kv, head_dim] at each
    sequence's last position (``seq_lens[b] - 1``) and return decode
    attention [B, n_heads, head_dim] over the updated pages, in one launch.
    Same as ``kv_write`` at those slots followed by ``paged_attention_decode``.
    """
    desc = pool_desc(k_pool)
    B, H, hd = q.shape
    W = block_tables.shape[1]
    if k_new.shape != (B, desc.n_kv, hd) or v_new.shape != k_new.shape:
        raise ValueError(f"k_new/v_new must be {(B, desc.n_kv, hd)}")
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    if out is None:
        out = torch.empty_like(q)
    need = decode_workspace_bytes(B, H, hd, max_seq_len, max_ctas, desc.block_size)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check("pkv_paged_attention_decode_append", _load().pkv_paged_attention_decode_append(
        _dev(q, "q", k_pool.dtype), _dev(k_new, "k_new", k_pool.dtype),
        _dev(v_new, "v_new", k_pool.dtype), B, H, _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"),
        ctypes.byref(desc), _dev(block_tables, "block_tables", torch.int32), W,
        _dev(seq_lens, "seq_lens", torch.int32), int(max_seq_len), float(scale), int(max_ctas),
        _dev(out, "out", k_pool.dtype), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _opt(err, "err", torch.int32),
        _stream(stream)))
    return out


def decode_plan(k_pool, seq_lens, n_heads: int, max_blocks_per_seq: int, max_seq_len: int, *,
                workspace, shared_prefix_blocks: int = 0, max_ctas: int = 0, err=None,
                stream=None):
    """Split a decode step's blocks over the decode grid once, into
    ``workspace``, for every layer's ``paged_attention_decode_planned``
    (same lengths, tables, shapes, shared prefix and ``max_ctas`` until the
    step ends)."""
    desc = pool_desc(k_pool)
    B = seq_lens.shape[0]
    _check("pkv_decode_plan", _load().pkv_decode_plan(
        B, int(n_heads), ctypes.byref(desc), int(max_blocks_per_seq),
        _dev(seq_lens, "seq_lens", torch.int32), int(max_seq_len), int(shared_prefix_blocks),
        int(max_ctas),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _opt(err, "err", torch.int32), _stream(stream)))
    return workspace


def paged_attention_decode_planned(q, k_pool, v_pool, block_tables, seq_lens, scale: float,
                                   max_seq_len: int, *, workspace, k_new=None, v_new=None,
                                   shared_prefix_blocks: int = 0, out=None, max_ctas: int = 0,
                                   err=None, stream=None):
    """``paged_attention_decode`` (with ``k_new``/``v_new``,
    ``paged_attention_decode_append``; with ``shared_prefix_blocks``,
    ``paged_attention_decode_shared_prefix``) using the plan
    ``decode_plan`` left in ``workspace``."""
    desc = pool_desc(k_pool)
    B, H, hd = q.shape
    W = block_tables.shape[1]
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new go together")
    if k_new is not None and (k_new.shape != (B, desc.n_kv, hd) or v_new.shape != k_new.shape):
        raise ValueError(f"k_new/v_new must be {(B, desc.n_kv, hd)}")
    if out is None:
        out = torch.empty_like(q)
    _check("pkv_paged_attention_decode_planned", _load().pkv_paged_attention_decode_planned(
        _dev(q, "q", k_pool.dtype),
        None if k_new is None else _dev(k_new, "k_new", k_pool.dtype),
        None if v_new is None else _dev(v_new, "v_new", k_pool.dtype), B, H,
        _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"), ctypes.byref(desc),
        _dev(block_tables, "block_tables", torch.int32), W,
        _dev(seq_lens, "seq_lens", torch.int32), int(max_seq_len), int(shared_prefix_blocks),
        float(scale), int(max_ctas), _dev(out, "out", k_pool.dtype), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _opt(err, "err", torch.int32),
        _stream(stream)))
    return out


def prefill_workspace_bytes(num_seqs, total_q, n_heads, head_dim, max_seq_len):
    return int(_load().pkv_prefill_workspace_bytes(num_seqs, total_q, n_heads, head_dim, max_seq_len))


def paged_attention_prefill(q, cu_q_lens, k_pool, v_pool, block_tables, seq_lens, scale: float,
                            max_q_len: int | None = None, max_seq_len: int | None = None, *,
                            out=None, workspace=None, err=None, stream=None):
    """Causal chunked-prefill attention [total_q, n_heads, head_dim]."""
    desc = pool_desc(k_pool)
    T, H, hd = q.shape
    B, W = block_tables.shape
    if max_q_len is None:
        max_q_len = int((cu_q_lens[1:] - cu_q_lens[:-1]).max().item()) if B else 0
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    if out is None:
        out = torch.empty_like(q)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size())
    _check("pkv_paged_attention_prefill", _load().pkv_paged_attention_prefill(
        _dev(q, "q", k_pool.dtype), _dev(cu_q_lens, "cu_q_lens", torch.int32), B, T,
        int(max_q_len), H, _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"), ctypes.byref(desc),
        _dev(block_tables, "block_tables", torch.int32), W,
        _dev(seq_lens, "seq_lens", torch.int32), int(max_seq_len), float(scale),
        _dev(out, "out", k_pool.dtype), ws_ptr, ws_bytes, _opt(err, "err", torch.int32),
        _stream(stream)))
    return out


def paged_attention_decode_noalloc(q, k_pool, v_pool, block_tables, seq_lens, scale: float,
                                   max_seq_len: int, *, out=None, max_ctas: int = 0, err=None,
                                   stream=None):
    """Decode attention using the library's built-in scratch instead of a
    caller workspace (for callers that cannot allocate device memory).

    Same result as :func:`paged_attention_decode`.  Calls overlapping on
    the GPU share the built-in scratch and race; the first call on a
    device should come before any stream capture.
    """
    L = _load()
    fn = L.pkv_paged_attention_decode_noalloc
    fn.restype = _i32
    fn.argtypes = [_p, _i32, _i32, _p, _p, _desc, _p, _i32, _p, _i32, _f, _i32, _p, _p, _p]
    desc = pool_desc(k_pool)
    B, H, hd = q.shape
    if out is None:
        out = torch.empty_like(q)
    _check("pkv_paged_attention_decode_noalloc", fn(
        _dev(q, "q", k_pool.dtype), B, H, _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"),
        ctypes.byref(desc), _dev(block_tables, "block_tables", torch.int32),
        block_tables.shape[1], _dev(seq_lens, "seq_lens", torch.int32), int(max_seq_len),
        float(scale), int(max_ctas), _dev(out, "out", k_pool.dtype),
        _opt(err, "err", torch.int32), _stream(stream)))
    return out


# ------------------------------------------------------------ 8-bit cache
#
# A decode step's kernels take 3-5 us, so what a call costs on the host counts:
# each tensor is checked in one pass (device, type, layout), and the current
# stream is asked for as a bare handle.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_f8 = torch.float8_e4m3fn
_f32 = torch.float32
_int = torch.int32


def _ptr(t, name, dtype, index):
    """Address of a contiguous tensor of ``dtype`` on CUDA device ``index``."""
    try:
        if t.get_device() == index and t.dtype is dtype and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if isinstance(t, torch.Tensor) and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{index}")
    return _dev(t, name, dtype)  # raises: it is not the type or layout asked for


def _context(stream, index):
    """What a call on a cache of device ``index`` has to run under (it then
    repeats itself there), or None: the stream it was given, so that what it
    allocates and reads belongs to that stream, or the cache's device."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = (torch.cuda.ExternalStream(int(stream), device=index) if int(stream)
                      else torch.cuda.default_stream(index))
        if stream.device_index != index:
            raise ValueError(f"stream is on device {stream.device_index}, the cache on {index}")
        return torch.cuda.stream(stream)
    return None if torch.cuda.current_device() == index else torch.cuda.device(index)


_TYPE_CODES = {torch.float32: PKV_F32, torch.bfloat16: PKV_BF16}


def _type_code(dtype):
    code = _TYPE_CODES.get(dtype)
    return _dtype_code(dtype) if code is None else code  # (raises)


def _fp8_pool(k_pool, v_pool, k_scales, v_scales):
    """Device, descriptor and addresses of an 8-bit cache, its four tensors checked."""
    shape = k_pool.shape
    if len(shape) != 4:
        raise ValueError("pool must be [num_blocks, block_size, n_kv, head_dim]")
    if v_pool.shape != shape:
        raise ValueError("k_pool and v_pool must have the same shape")
    nb, bs, nkv, hd = shape
    per = (nb, nkv)
    if k_scales.shape != per or v_scales.shape != per:
        raise ValueError(f"k_scales and v_scales must be {per}: one per block and KV head")
    index = k_pool.get_device()
    if index < 0:
        raise ValueError("k_pool must be a CUDA tensor (the library has no CPU path)")
    desc = PoolDesc(nb, bs, nkv, hd, PKV_FP8_E4M3)
    return (index, desc, _ptr(k_pool, "k_pool", _f8, index), _ptr(v_pool, "v_pool", _f8, index),
            _ptr(k_scales, "k_scales", _f32, index), _ptr(v_scales, "v_scales", _f32, index))


def _batch(block_tables, seq_lens):
    """(num_seqs, table width) of a batch's tables and lengths."""
    shape = block_tables.shape
    if len(shape) != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    if seq_lens.shape != shape[:1]:
        raise ValueError(f"seq_lens must be {tuple(shape[:1])}: one per row of block_tables")
    return shape


def _offsets(cu, name, B, index):
    if cu.shape != (B + 1,):
        raise ValueError(f"{name} must be {(B + 1,)}")
    return _ptr(cu, name, _int, index)


def kv_write_fp8(k, v, block_tables, seq_lens, cu_new_lens, k_pool, v_pool, k_scales, v_scales, *,
                 err=None, stream=None):
    """Quantise k/v [T, n_kv, head_dim] (float32 or bfloat16) into an 8-bit
    cache: pools of ``torch.float8_e4m3fn`` [num_blocks, block_size, n_kv,
    head_dim] and float32 scales [num_blocks, n_kv], powers of two.

    Sequence b's rows ``cu_new_lens[b] : cu_new_lens[b+1]`` go to its last
    positions, up to ``seq_lens[b] - 1``.  A block that holds earlier tokens
    keeps at least its scale; where a new token needs a larger one the earlier
    rows are moved to it.
    """
    i, desc, kp, vp, ks, vs = _fp8_pool(k_pool, v_pool, k_scales, v_scales)
    there = _context(stream, i)
    if there is not None:
        with there:
            return kv_write_fp8(k, v, block_tables, seq_lens, cu_new_lens, k_pool, v_pool,
                                k_scales, v_scales, err=err)
    B, W = _batch(block_tables, seq_lens)
    shape = k.shape
    if len(shape) != 3 or shape != (shape[0], desc.n_kv, desc.head_dim) or v.shape != shape:
        raise ValueError("k, v must be [T, n_kv, head_dim] matching the pool")
    dt = k.dtype
    status = (_lib or _load()).pkv_kv_write_fp8(
        _ptr(k, "k", dt, i), _ptr(v, "v", dt, i), _type_code(dt),
        _ptr(block_tables, "block_tables", _int, i), W, _ptr(seq_lens, "seq_lens", _int, i),
        _offsets(cu_new_lens, "cu_new_lens", B, i), B, shape[0], kp, vp, ks, vs,
        ctypes.byref(desc), None if err is None else _ptr(err, "err", _int, i),
        _raw_stream(i))
    if status:
        raise PkvError("pkv_kv_write_fp8", status)


def kv_gather_fp8(k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens, cu_seq_lens,
                  total_tokens: int, *, dtype=torch.bfloat16, k_out=None, v_out=None, err=None,
                  stream=None):
    """Contiguous [total_tokens, n_kv, head_dim] K and V of an 8-bit cache in
    logical order, each value times its scale, in ``dtype`` (float32 or
    bfloat16; that of ``k_out`` / ``v_out`` where given)."""
    i, desc, kp, vp, ks, vs = _fp8_pool(k_pool, v_pool, k_scales, v_scales)
    there = _context(stream, i)
    if there is not None:
        with there:
            return kv_gather_fp8(k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens,
                                 cu_seq_lens, total_tokens, dtype=dtype, k_out=k_out,
                                 v_out=v_out, err=err)
    B, W = _batch(block_tables, seq_lens)
    dt = k_out.dtype if k_out is not None else v_out.dtype if v_out is not None else dtype
    code = _type_code(dt)
    shape = (int(total_tokens), desc.n_kv, desc.head_dim)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dt, device=k_pool.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dt, device=k_pool.device)
    if k_out.shape != shape or v_out.shape != shape:
        raise ValueError(f"k_out, v_out must be {shape}")
    status = (_lib or _load()).pkv_kv_gather_fp8(
        kp, vp, ks, vs, ctypes.byref(desc), _ptr(block_tables, "block_tables", _int, i), W,
        _ptr(seq_lens, "seq_lens", _int, i), _offsets(cu_seq_lens, "cu_seq_lens", B, i), B,
        shape[0], code, _ptr(k_out, "k_out", dt, i), _ptr(v_out, "v_out", dt, i),
        None if err is None else _ptr(err, "err", _int, i),
        _raw_stream(i))
    if status:
        raise PkvError("pkv_kv_gather_fp8", status)
    return k_out, v_out


def decode_fp8_workspace_bytes(num_seqs, n_heads, head_dim, max_seq_len, max_ctas=0, block_size=16):
    return int(_load().pkv_decode_fp8_workspace_bytes(num_seqs, n_heads, head_dim, max_seq_len,
                                                      max_ctas, block_size))


def _fp8_query(q, head_dim, out):
    """(out, rows, heads) of an attention call."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != head_dim:
        raise ValueError("q must be [rows, n_heads, head_dim] with the pool's head_dim")
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != shape:
        raise ValueError(f"out must be {tuple(shape)}")
    return out, shape[0], shape[1]


def paged_attention_decode_fp8(q, k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens,
                               scale: float, max_seq_len: int | None = None, *, out=None,
                               workspace=None, max_ctas: int = 0, err=None, stream=None):
    """Decode attention [B, n_heads, head_dim] (float32 or bfloat16) over the
    paged history of an 8-bit cache (see :func:`kv_write_fp8`).

    ``max_seq_len`` and ``workspace`` are as for
    :func:`paged_attention_decode`, with ``decode_fp8_workspace_bytes(...)``
    bytes; calls that may run at the same time need a workspace each.
    """
    i, desc, kp, vp, ks, vs = _fp8_pool(k_pool, v_pool, k_scales, v_scales)
    there = _context(stream, i)
    if there is not None:
        with there:
            return paged_attention_decode_fp8(q, k_pool, v_pool, k_scales, v_scales, block_tables,
                                              seq_lens, scale, max_seq_len, out=out,
                                              workspace=workspace, max_ctas=max_ctas, err=err)
    B, W = _batch(block_tables, seq_lens)
    out, rows, H = _fp8_query(q, desc.head_dim, out)
    if rows != B:
        raise ValueError("q must have one row per sequence")
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    if workspace is None:
        need = decode_fp8_workspace_bytes(B, H, desc.head_dim, max_seq_len, max_ctas)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    dt = q.dtype
    status = (_lib or _load()).pkv_paged_attention_decode_fp8(
        _ptr(q, "q", dt, i), _type_code(dt), B, H, kp, vp, ks, vs, ctypes.byref(desc),
        _ptr(block_tables, "block_tables", _int, i), W, _ptr(seq_lens, "seq_lens", _int, i),
        int(max_seq_len), float(scale), int(max_ctas), _ptr(out, "out", dt, i),
        _ptr(workspace, "workspace", workspace.dtype, i), workspace.nbytes,
        None if err is None else _ptr(err, "err", _int, i),
        _raw_stream(i))
    if status:
        raise PkvError("pkv_paged_attention_decode_fp8", status)
    return out


def paged_attention_prefill_fp8(q, cu_q_lens, k_pool, v_pool, k_scales, v_scales, block_tables,
                                seq_lens, scale: float, max_q_len: int | None = None,
                                max_seq_len: int | None = None, *, out=None, err=None,
                                stream=None):
    """Causal chunked-prefill attention [total_q, n_heads, head_dim] (float32
    or bfloat16) over the paged history of an 8-bit cache."""
    i, desc, kp, vp, ks, vs = _fp8_pool(k_pool, v_pool, k_scales, v_scales)
    there = _context(stream, i)
    if there is not None:
        with there:
            return paged_attention_prefill_fp8(q, cu_q_lens, k_pool, v_pool, k_scales, v_scales,
                                               block_tables, seq_lens, scale, max_q_len,
                                               max_seq_len, out=out, err=err)
    B, W = _batch(block_tables, seq_lens)
    out, rows, H = _fp8_query(q, desc.head_dim, out)
    if max_q_len is None:
        max_q_len = int((cu_q_lens[1:] - cu_q_lens[:-1]).max().item()) if B else 0
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if B else 0
    dt = q.dtype
    status = (_lib or _load()).pkv_paged_attention_prefill_fp8(
        _ptr(q, "q", dt, i), _type_code(dt), _offsets(cu_q_lens, "cu_q_lens", B, i), B, rows,
        int(max_q_len), H, kp, vp, ks, vs, ctypes.byref(desc),
        _ptr(block_tables, "block_tables", _int, i), W, _ptr(seq_lens, "seq_lens", _int, i),
        int(max_seq_len), float(scale), _ptr(out, "out", dt, i),
        None if err is None else _ptr(err, "err", _int, i),
        _raw_stream(i))
    if status:
        raise PkvError("pkv_paged_attention_prefill_fp8", status)
    return out


def selftest_bounded_wait_fp8(err, polls: int = 64, *, stream=None):
    """:func:`selftest_bounded_wait` for the 8-bit kernels' waits, which a whole
    warp gives up together."""
    _check("pkv_selftest_bounded_wait_fp8", _load().pkv_selftest_bounded_wait_fp8(
        int(polls), _dev(err, "err", torch.int32), _stream(stream)))


# ------------------------------------- queries and keys before the cache
#
# These entries' tensors are checked, and their calls made, by a CPython extension
# (csrc/binding.cpp): in a decode step the host's part of a call would else take
# several times the kernel's.  Rows [tokens, heads, head_dim] may be parts of one
# projection's output: a token's heads lie together, tokens any multiple of 16 bytes
# apart.

_native = None


def _load_binding():
    """The extension; raises if it has not been built."""
    global _native
    if _native is None:
        _load()
        try:
            _native = importlib.import_module("._binding", __name__)
        except ImportError as e:
            raise ImportError(f"the extension in {HERE} cannot be loaded: build it with "
                              f"`python -m paged_kv_cache_write_gb300.build` ({e})") from e
    return _native


def _on(stream, t, name):
    """The stream a call was given as a context, so that what it allocates and reads
    belongs to that stream."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    return _context(stream, t.get_device())


def _rows_like(t):
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def qk_norm_rope(q, k, cos_sin, positions, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, err=None, stream=None):
    """Norm and rotation of a step's queries [T, n_heads, head_dim] and keys
    [T, n_kv, head_dim] (float32 or bfloat16); returns both.

    With a weight [head_dim], each head's row is first divided by its root mean
    square (``eps`` inside the root) and multiplied by the weight.  The first
    ``rot_dim`` dims are then turned by the angles of the token's row of
    ``cos_sin``, float32 [num_positions, rot_dim] (cosines, then sines): dim i with
    i + rot_dim / 2, or 2i with 2i + 1 where ``interleaved``.  ``positions`` is int32
    [T].  All in fp32, rounded once.  Rows may be views of one projection's output;
    ``q_out`` / ``k_out`` may be ``q`` / ``k`` themselves.
    """
    if stream is not None:
        with _on(stream, q, "q"):
            return qk_norm_rope(q, k, cos_sin, positions, q_weight=q_weight, k_weight=k_weight, eps=eps,
                                interleaved=interleaved, q_out=q_out, k_out=k_out, err=err)
    if q_out is None:
        q_out = _rows_like(q)
    if k_out is None:
        k_out = _rows_like(k)
    status = (_native or _load_binding()).qk_norm_rope(q, k, cos_sin, positions, q_weight, k_weight, eps,
                                                  interleaved, q_out, k_out, err)
    if status:
        raise PkvError("pkv_qk_norm_rope", status)
    return q_out, k_out


def qk_norm_rope_write(q, k, v, cos_sin, positions, slot_mapping, k_pool, v_pool, *, q_weight=None,
                       k_weight=None, eps: float = 1e-6, interleaved: bool = False, q_out=None,
                       err=None, stream=None):
    """:func:`qk_norm_rope`, its keys and the values ``v`` [T, n_kv, head_dim] written
    to their slots as by :func:`kv_write`, in one launch; returns the queries."""
    if stream is not None:
        with _on(stream, k_pool, "k_pool"):
            return qk_norm_rope_write(q, k, v, cos_sin, positions, slot_mapping, k_pool, v_pool,
                                      q_weight=q_weight, k_weight=k_weight, eps=eps,
                                      interleaved=interleaved, q_out=q_out, err=err)
    if q_out is None:
        q_out = _rows_like(q)
    status = (_native or _load_binding()).qk_norm_rope_write(q, k, v, cos_sin, positions, slot_mapping, k_pool,
                                                        v_pool, q_weight, k_weight, eps, interleaved,
                                                        q_out, err)
    if status:
        raise PkvError("pkv_qk_norm_rope_write", status)
    return q_out


# ------------------------------------------------------------ 4-bit cache

def kv_write_fp4(k, v, slot_mapping, k_pool, v_pool, k_groups, v_groups, k_scale, v_scale, *, err=None,
                 stream=None):
    """Quantise k/v [T, n_kv, head_dim] (float32 or bfloat16) into a 4-bit cache at
    slot_mapping [T]: pools of e2m1 codes, two to a byte, uint8 [num_blocks, n_kv,
    block_size, head_dim / 2]; a ``torch.float8_e4m3fn`` scale per 16 elements of a
    row, [num_blocks, n_kv, block_size, head_dim / 16]; and a float32 scale per KV
    head, a power of two, [n_kv], which the caller chooses once for the cache (another is
    reported in ``err``, and that head not written).

    A token's codes depend on that token alone.  Values past 2,688 x its head's
    scale saturate; a group's scale loses precision below 0.1 x it.
    """
    if stream is not None:
        with _on(stream, k_pool, "k_pool"):
            return kv_write_fp4(k, v, slot_mapping, k_pool, v_pool, k_groups, v_groups, k_scale,
                                v_scale, err=err)
    status = (_native or _load_binding()).kv_write_fp4(k, v, slot_mapping, k_pool, v_pool, k_groups, v_groups,
                                                  k_scale, v_scale, err)
    if status:
        raise PkvError("pkv_kv_write_fp4", status)


def qk_norm_rope_write_fp4(q, k, v, cos_sin, positions, slot_mapping, k_pool, v_pool, k_groups,
                           v_groups, k_scale, v_scale, *, q_weight=None, k_weight=None,
                           eps: float = 1e-6, interleaved: bool = False, q_out=None, err=None,
                           stream=None):
    """:func:`qk_norm_rope`, its keys and the values ``v`` quantised into a 4-bit cache
    as by :func:`kv_write_fp4`, in one launch; returns the queries."""
    if stream is not None:
        with _on(stream, k_pool, "k_pool"):
            return qk_norm_rope_write_fp4(q, k, v, cos_sin, positions, slot_mapping, k_pool, v_pool,
                                          k_groups, v_groups, k_scale, v_scale, q_weight=q_weight,
                                          k_weight=k_weight, eps=eps, interleaved=interleaved,
                                          q_out=q_out, err=err)
    if q_out is None:
        q_out = _rows_like(q)
    status = (_native or _load_binding()).qk_norm_rope_write_fp4(
        q, k, v, cos_sin, positions, slot_mapping, k_pool, v_pool, k_groups, v_groups, k_scale, v_scale,
        q_weight, k_weight, eps, interleaved, q_out, err)
    if status:
        raise PkvError("pkv_qk_norm_rope_write_fp4", status)
    return q_out


def kv_gather_fp4(k_pool, v_pool, k_groups, v_groups, k_scale, v_scale, block_tables, seq_lens,
                  cu_seq_lens, total_tokens: int, *, dtype=torch.bfloat16, k_out=None, v_out=None,
                  err=None, stream=None):
    """Contiguous [total_tokens, n_kv, head_dim] K and V of a 4-bit cache in logical
    order, each code times its scales, in ``dtype`` (float32 or bfloat16; that of
    ``k_out`` / ``v_out`` where given)."""
    if stream is not None:
        with _on(stream, k_pool, "k_pool"):
            return kv_gather_fp4(k_pool, v_pool, k_groups, v_groups, k_scale, v_scale, block_tables,
                                 seq_lens, cu_seq_lens, total_tokens, dtype=dtype, k_out=k_out,
                                 v_out=v_out, err=err)
    if k_out is None or v_out is None:
        dt = k_out.dtype if k_out is not None else v_out.dtype if v_out is not None else dtype
        shape = (int(total_tokens), k_pool.shape[1], 2 * k_pool.shape[3])
        k_out = torch.empty(shape, dtype=dt, device=k_pool.device) if k_out is None else k_out
        v_out = torch.empty(shape, dtype=dt, device=k_pool.device) if v_out is None else v_out
    status = (_native or _load_binding()).kv_gather_fp4(
        k_pool, v_pool, k_groups, v_groups, k_scale, v_scale, block_tables, seq_lens, cu_seq_lens,
        total_tokens, k_out, v_out, err)
    if status:
        raise PkvError("pkv_kv_gather_fp4", status)
    return k_out, v_out


def decode_fp4_workspace_bytes(num_seqs, n_heads, head_dim, max_seq_len, max_ctas=0, block_size=16):
    return int(_load().pkv_decode_fp4_workspace_bytes(num_seqs, n_heads, head_dim, max_seq_len,
                                                      max_ctas, block_size))


def paged_attention_decode_fp4(q, k_pool, v_pool, k_groups, v_groups, k_scale, v_scale, block_tables,
                               seq_lens, scale: float, max_seq_len: int | None = None, *, out=None,
                               workspace=None, max_ctas: int = 0, err=None, stream=None):
    """Decode attention [B, n_heads, head_dim] (float32 or bfloat16) over the paged
    history of a 4-bit cache (see :func:`kv_write_fp4`).

    ``max_seq_len`` and ``workspace`` are as for :func:`paged_attention_decode`, with
    ``decode_fp4_workspace_bytes(...)`` bytes; calls that may run at the same time need a
    workspace each.
    """
    if stream is not None:
        with _on(stream, k_pool, "k_pool"):
            return paged_attention_decode_fp4(q, k_pool, v_pool, k_groups, v_groups, k_scale, v_scale,
                                              block_tables, seq_lens, scale, max_seq_len, out=out,
                                              workspace=workspace, max_ctas=max_ctas, err=err)
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if len(seq_lens) else 0
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        with torch.cuda.device(q.device):  # (as large as that device's grid)
            need = decode_fp4_workspace_bytes(*q.shape, max_seq_len, max_ctas)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    status = (_native or _load_binding()).paged_attention_decode_fp4(
        q, k_pool, v_pool, k_groups, v_groups, k_scale, v_scale, block_tables, seq_lens, scale,
        max_seq_len, out, workspace, max_ctas, err)
    if status:
        raise PkvError("pkv_paged_attention_decode_fp4", status)
    return out


def paged_attention_prefill_fp4(q, cu_q_lens, k_pool, v_pool, k_groups, v_groups, k_scale, v_scale,
                                block_tables, seq_lens, scale: float, max_q_len: int | None = None,
                                max_seq_len: int | None = None, *, out=None, err=None, stream=None):
    """Causal chunked-prefill attention [total_q, n_heads, head_dim] (float32 or
    bfloat16) over the paged history of a 4-bit cache."""
    if stream is not None:
        with _on(stream, k_pool, "k_pool"):
            return paged_attention_prefill_fp4(q, cu_q_lens, k_pool, v_pool, k_groups, v_groups, k_scale,
                                               v_scale, block_tables, seq_lens, scale, max_q_len,
                                               max_seq_len, out=out, err=err)
    if max_q_len is None:
        max_q_len = int((cu_q_lens[1:] - cu_q_lens[:-1]).max().item()) if len(seq_lens) else 0
    if max_seq_len is None:
        max_seq_len = int(seq_lens.max().item()) if len(seq_lens) else 0
    if out is None:
        out = torch.empty_like(q)
    status = (_native or _load_binding()).paged_attention_prefill_fp4(
        q, cu_q_lens, k_pool, v_pool, k_groups, v_groups, k_scale, v_scale, block_tables, seq_lens,
        scale, max_q_len, max_seq_len, out, err)
    if status:
        raise PkvError("pkv_paged_attention_prefill_fp4", status)
    return out
