"""GB300-native block-paged KV attention: Python binding of ``libpkv.so``.

The functions here only marshal arguments (torch tensors -> device pointers,
sizes and the current CUDA stream) into the C ABI declared in
``include/pkv.h``; every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if the library is missing, importing
this package raises.

Layouts (see ``include/pkv.h``): pools ``[num_blocks, num_kv_heads,
block_size, head_dim]``; ``q``/``out`` ``[batch, num_q_heads, head_dim]``
(prefill: ``[sum C, num_q_heads, head_dim]``); block tables int32
``[batch, max_blocks_per_seq]``; ``seq_lens`` int32 ``[batch]`` counting the
tokens appended this step; rotary ``positions`` int32 ``[num_axes, tokens]``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Tuple

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_CUDA, PKV_ERR_WORKSPACE, PKV_ERR_OUT_OF_BLOCKS = range(6)
PKV_ERR_HOST_MEMORY = 6
PKV_F32, PKV_BF16, PKV_FP8_E4M3 = 0, 1, 2
DEV_BAD_BLOCK, DEV_BAD_SLOT, DEV_BAD_LEN, DEV_BAD_PREFIX, DEV_TIMEOUT = 1, 2, 4, 8, 16
DEV_Q_RANGE, DEV_BAD_PATH = 32, 64

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it first "
                      "(python -c 'import __graft_entry__ as g; g.build()')")
_lib = ctypes.CDLL(LIB_PATH)


class _Pool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_blocks", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class _Prefix(ctypes.Structure):
    _fields_ = [("num_groups", ctypes.c_int32), ("max_group_rows", ctypes.c_int32),
                ("max_prefix_blocks", ctypes.c_int32), ("group_of_row", ctypes.c_void_p),
                ("prefix_blocks", ctypes.c_void_p)]


class _Group(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("pool", _Pool),
                ("block_tables", ctypes.c_void_p), ("max_blocks_per_seq", ctypes.c_int32),
                ("seq_lens", ctypes.c_void_p), ("max_seq_len", ctypes.c_int32),
                ("window", ctypes.c_int32), ("scale", ctypes.c_float)]


ROPE_MAX_AXES, ROPE_MAX_PAIRS = 4, 128


class _Rope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("factor", ctypes.c_float),
                ("freq", ctypes.c_uint64 * ROPE_MAX_PAIRS), ("axis", ctypes.c_uint8 * ROPE_MAX_PAIRS)]


class _LatentPool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("latent_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32), ("dtype", ctypes.c_int)]


MAX_DECODE_GROUPS = 4
MAX_TREE = 64

_vp, _i32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_PP, _XP = ctypes.POINTER(_Pool), ctypes.POINTER(_Prefix)
_GP = ctypes.POINTER(_Group)

_lib.paged_kv_append.argtypes = [_PP, _vp, _i32, _vp, _vp, _vp, _vp]
_lib.paged_kv_append.restype = ctypes.c_int
_lib.paged_decode_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _XP]
_lib.paged_decode_workspace_size.restype = _sz
_lib.paged_decode_attention.argtypes = [_vp, _i32, _PP, _vp, _i32, _vp, _i32, _i32, _i32,
                                        ctypes.c_float, _vp, _vp, _sz, _XP, _vp, _vp]
_lib.paged_decode_attention.restype = ctypes.c_int
_lib.paged_decode_groups_workspace_size.argtypes = [_GP, _i32, _i32, _i32]
_lib.paged_decode_groups_workspace_size.restype = _sz
_lib.paged_decode_attention_groups.argtypes = [_GP, _i32, _i32, _i32, _vp, _sz, _vp, _vp]
_lib.paged_decode_attention_groups.restype = ctypes.c_int
_lib.paged_prefill_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32]
_lib.paged_prefill_workspace_size.restype = _sz
_lib.paged_prefill_chunk_attention.argtypes = [_vp, _vp, _i32, _PP, _vp, _i32, _vp, _i32, _i32,
                                               _i32, _i32, ctypes.c_float, _vp, _vp, _sz, _vp, _vp]
_lib.paged_prefill_chunk_attention.restype = ctypes.c_int
_lib.pkv_status_string.argtypes = [ctypes.c_int]
_lib.pkv_status_string.restype = ctypes.c_char_p
_lib.pkv_slot_mapping_host.argtypes = [_vp, _i32, _i32, _i32, _vp, _vp, _i32, _i32, _vp]
_lib.pkv_slot_mapping_host.restype = ctypes.c_int
_lib.pkv_prefix_groups_host.argtypes = [_vp, _i32, _vp, _i32, _i32, _vp, _vp]
_lib.pkv_prefix_groups_host.restype = _i32
_lib.pkv_set_decode_split_blocks.argtypes = [_i32]
_lib.pkv_set_decode_split_blocks.restype = _i32
_lib.pkv_set_wait_drill.argtypes = [ctypes.c_uint64, ctypes.c_uint32]
_lib.pkv_set_wait_drill.restype = ctypes.c_int
_lib.pkv_decode_plan.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                 ctypes.POINTER(_i32)]
_lib.pkv_decode_plan.restype = _i32
_lib.pkv_version.restype = ctypes.c_char_p
_lib.pkv_profile_enable.argtypes = [ctypes.c_uint32]
_lib.pkv_profile_enable.restype = ctypes.c_int
_lib.pkv_profile_mask.argtypes = [ctypes.c_uint32]
_lib.pkv_profile_mask.restype = ctypes.c_int
_lib.pkv_profile_read.argtypes = [_i32, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_double)]
_lib.pkv_profile_read.restype = ctypes.c_int
_lib.pkv_profile_times.argtypes = [_i32, _vp, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
_lib.pkv_profile_times.restype = ctypes.c_int
_lib.pkv_launch_count.restype = ctypes.c_int64
_lib.paged_decode_attention_no_alloc.argtypes = [_vp, _i32, _PP, _vp, _i32, _vp, _i32, _i32, _i32,
                                                 ctypes.c_float, _vp, _XP, _vp, _vp]
_lib.paged_decode_attention_no_alloc.restype = ctypes.c_int
NO_ALLOC_SCRATCH_BYTES = 16 << 20
_u64p = ctypes.POINTER(ctypes.c_uint64)
_i64, _RP = ctypes.c_int64, ctypes.POINTER(_Rope)
_lib.pkv_rope_init.argtypes = [_RP, _i32, _vp, _i32, _vp, _i32, ctypes.c_float]
_lib.pkv_rope_init.restype = ctypes.c_int
_lib.paged_kv_append_rope.argtypes = [_PP, _vp, _i32, _vp, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _i64,
                                      _RP, _vp, _i64, _vp, _vp]
_lib.paged_kv_append_rope.restype = ctypes.c_int
_lib.paged_copy_blocks.argtypes = [_PP, _PP, _i32, _vp, _vp, _i32, _vp, _vp]
_lib.paged_copy_blocks.restype = ctypes.c_int
_i32p = ctypes.POINTER(ctypes.c_int32)
_lib.pkv_slot_mapping_check_host.argtypes = [_vp, _i32, _i32, _i32, _i32p]
_lib.pkv_slot_mapping_check_host.restype = ctypes.c_int
_lib.paged_decode_sinks_workspace_size.argtypes = [_i32] * 8
_lib.paged_decode_sinks_workspace_size.restype = _sz
_lib.paged_decode_attention_sinks.argtypes = [_vp, _i32, _PP, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                              ctypes.c_float, _vp, _vp, _sz, _vp, _vp]
_lib.paged_decode_attention_sinks.restype = ctypes.c_int
_lib.paged_decode_groups_sinks_workspace_size.argtypes = [_GP, _vp, _i32, _i32, _i32]
_lib.paged_decode_groups_sinks_workspace_size.restype = _sz
_lib.paged_decode_attention_groups_sinks.argtypes = [_GP, _vp, _i32, _i32, _i32, _vp, _sz, _vp, _vp]
_lib.paged_decode_attention_groups_sinks.restype = ctypes.c_int
_lib.paged_prefill_sinks_workspace_size.argtypes = [_i32] * 9
_lib.paged_prefill_sinks_workspace_size.restype = _sz
_lib.paged_prefill_chunk_attention_sinks.argtypes = [_vp, _vp, _i32, _PP, _vp, _i32, _vp, _i32, _i32, _i32,
                                                     _i32, _i32, ctypes.c_float, _vp, _vp, _sz, _vp, _vp]
_lib.paged_prefill_chunk_attention_sinks.restype = ctypes.c_int
_lib.pkv_block_copies_check_host.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _i32p]
_lib.pkv_block_copies_check_host.restype = ctypes.c_int
_lib.pkv_allocator_expire_window.argtypes = [_vp, _i32, _i32, _i32]
_lib.pkv_allocator_expire_window.restype = ctypes.c_int
_lib.pkv_allocator_fork.argtypes = [_vp, _i32, _i32, _i32p, _i32p, _i32p]
_lib.pkv_allocator_fork.restype = ctypes.c_int
_lib.pkv_allocator_truncate.argtypes = [_vp, _i32, _i32, _i32p, _i32p]
_lib.pkv_allocator_truncate.restype = ctypes.c_int
_lib.pkv_allocator_compact.argtypes = [_vp, _i32, _vp, _vp, _i32, _i32p]
_lib.pkv_allocator_compact.restype = ctypes.c_int
_lib.pkv_allocator_create.argtypes = [_i32, _i32, _i32]
_lib.pkv_allocator_create.restype = _vp
_lib.pkv_allocator_destroy.argtypes = [_vp]
_lib.pkv_allocator_destroy.restype = None
_lib.pkv_allocator_begin.argtypes = [_vp]
_lib.pkv_allocator_begin.restype = _i32
_lib.pkv_allocator_find_cached_prefix.argtypes = [_vp, _i32, _vp, _i32, _vp, _i32p]
_lib.pkv_allocator_find_cached_prefix.restype = ctypes.c_int
_lib.pkv_allocator_reserve.argtypes = [_vp, _i32, _i32]
_lib.pkv_allocator_reserve.restype = ctypes.c_int
_lib.pkv_allocator_publish.argtypes = [_vp, _i32, _vp, _i32, _vp]
_lib.pkv_allocator_publish.restype = ctypes.c_int
_lib.pkv_allocator_expire.argtypes = [_vp, _i32, _i32]
_lib.pkv_allocator_expire.restype = ctypes.c_int
_lib.pkv_allocator_release.argtypes = [_vp, _i32]
_lib.pkv_allocator_release.restype = ctypes.c_int
_lib.pkv_allocator_table.argtypes = [_vp, _i32, _vp, _i32, _i32p]
_lib.pkv_allocator_table.restype = ctypes.c_int
_lib.pkv_allocator_refcount.argtypes = [_vp, _i32]
_lib.pkv_allocator_refcount.restype = _i32
_lib.pkv_allocator_stats.argtypes = [_vp, _i32p, _i32p, _i32p, _i32p]
_lib.pkv_allocator_stats.restype = ctypes.c_int
_LP = ctypes.POINTER(_LatentPool)
_lib.paged_tree_workspace_size.argtypes = [_i32] * 8
_lib.paged_tree_workspace_size.restype = _sz
_lib.paged_tree_attention.argtypes = [_vp, _vp, _vp, _i32, _PP, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                      ctypes.c_float, _vp, _vp, _sz, _vp, _vp]
_lib.paged_tree_attention.restype = ctypes.c_int
_lib.paged_tree_attention_queries.argtypes = [_vp, _i32, *_lib.paged_tree_attention.argtypes[1:]]
_lib.paged_tree_attention_queries.restype = ctypes.c_int
_lib.pkv_tree_masks_host.argtypes = [_vp, _vp, _i32, _vp]
_lib.pkv_tree_masks_host.restype = ctypes.c_int
_lib.paged_tree_commit.argtypes = [_PP, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _vp]
_lib.paged_tree_commit.restype = ctypes.c_int
_lib.paged_latent_tree_commit.argtypes = [_LP, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _vp]
_lib.paged_latent_tree_commit.restype = ctypes.c_int
_lib.paged_latent_append.argtypes = [_LP, _vp, _i32, _vp, _i64, _vp, _i64, _vp, ctypes.c_float, _vp, _i64, _i64,
                                     _i32, _vp, _i64, _RP, _vp, _i64, _i64, _vp, _vp]
_lib.paged_latent_append.restype = ctypes.c_int
_lib.paged_latent_workspace_size.argtypes = [_i32] * 7
_lib.paged_latent_workspace_size.restype = _sz
_lib.paged_latent_attention.argtypes = [_vp, _i32, _vp, _vp, _i32, _LP, _vp, _i32, _vp, _i32, _i32, _i32,
                                        ctypes.c_float, _vp, _vp, _sz, _vp, _vp]
_lib.paged_latent_attention.restype = ctypes.c_int

KERNEL_APPEND, KERNEL_DECODE_PREFIX, KERNEL_DECODE_SPLIT, KERNEL_DECODE_COMBINE, KERNEL_PREFILL, KERNEL_COPY = range(6)
KERNEL_LATENT = 6

EXPORTED = ["paged_kv_append", "paged_decode_workspace_size", "paged_decode_attention",
            "paged_prefill_workspace_size", "paged_prefill_chunk_attention", "pkv_status_string",
            "pkv_slot_mapping_host", "pkv_slot_mapping_check_host", "pkv_prefix_groups_host",
            "pkv_set_decode_split_blocks", "pkv_set_wait_drill",
            "pkv_decode_plan", "pkv_version", "pkv_profile_enable", "pkv_profile_mask", "pkv_profile_read", "pkv_profile_times",
            "pkv_launch_count", "paged_decode_attention_no_alloc", "paged_decode_groups_workspace_size",
            "paged_decode_attention_groups", "pkv_allocator_create",
            "pkv_allocator_destroy", "pkv_allocator_begin", "pkv_allocator_find_cached_prefix",
            "pkv_allocator_reserve", "pkv_allocator_publish", "pkv_allocator_expire",
            "pkv_allocator_release",
            "pkv_allocator_table", "pkv_allocator_refcount", "pkv_allocator_stats",
            "pkv_rope_init", "paged_kv_append_rope", "paged_copy_blocks", "pkv_block_copies_check_host",
            "paged_decode_sinks_workspace_size", "paged_decode_attention_sinks",
            "paged_decode_groups_sinks_workspace_size", "paged_decode_attention_groups_sinks",
            "paged_prefill_sinks_workspace_size", "paged_prefill_chunk_attention_sinks",
            "pkv_allocator_expire_window", "pkv_allocator_fork", "pkv_allocator_truncate",
            "pkv_allocator_compact", "paged_tree_workspace_size", "paged_tree_attention",
            "paged_tree_attention_queries", "pkv_tree_masks_host",
            "paged_tree_commit", "paged_latent_tree_commit", "paged_latent_append", "paged_latent_workspace_size",
            "paged_latent_attention"]


class PkvError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {_lib.pkv_status_string(code).decode()} (status {code})")
        self.code = code


def _check(fn: str, code: int) -> None:
    if code != PKV_OK:
        raise PkvError(fn, code)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return PKV_F32
    if t == torch.bfloat16:
        return PKV_BF16
    if t == torch.uint8:
        return PKV_FP8_E4M3
    raise TypeError(f"unsupported dtype {t}: the pools hold float32, bfloat16 or FP8 (uint8) codes")


def _act_dtype(pool_dtype: torch.dtype) -> torch.dtype:
    """dtype of queries, outputs and new rows for a pool: bf16 beside FP8 pools."""
    return torch.bfloat16 if pool_dtype == torch.uint8 else pool_dtype


FP8_BLOCK_SIZE = 16


def fp8_pools(num_blocks: int, num_kv_heads: int, head_dim: int, device) -> Tuple[torch.Tensor, torch.Tensor]:
    """A pair of FP8 (E4M3) pools: uint8 tile bytes [num_blocks, num_kv_heads,
    16 * head_dim] (block size 16, tile bytes in the library's fragment order)."""
    shape = (num_blocks, num_kv_heads, FP8_BLOCK_SIZE * head_dim)
    return (torch.zeros(shape, dtype=torch.uint8, device=device),
            torch.zeros(shape, dtype=torch.uint8, device=device))


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> int:
    return _raw_stream(device.index)


_NULL = contextlib.nullcontext()
# the bindings under torch.cuda's calls, which cost more than the library's own
# checks; a torch built without CUDA lacks them (the allocator and the host
# helpers work there all the same)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(device: torch.device):
    """Make `device` current for a library call (the library plans for, and
    takes scratch from, the current device); a no-op when it already is."""
    if _current_device() == device.index:
        return _NULL
    return torch.cuda.device(device)


def _require(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


# Host cost of a call matters at decode sizes (a launch takes 3 us): the checks
# below read each attribute once, in one expression per call, and only a call
# that fails one goes through the messages.
def _pool(k_pool: torch.Tensor, v_pool: torch.Tensor, k_scale: Optional[float] = None,
          v_scale: Optional[float] = None) -> _Pool:
    dt, shape = k_pool.dtype, k_pool.shape
    if not (dt is v_pool.dtype and shape == v_pool.shape and k_pool.is_cuda and
            v_pool.get_device() == k_pool.get_device() and k_pool.is_contiguous() and
            v_pool.is_contiguous()):
        _require(dt is v_pool.dtype and shape == v_pool.shape, "K and V pools share a dtype and a shape")
        _require(k_pool.is_cuda and v_pool.is_cuda, "pools live on the GPU")
        _require(v_pool.device == k_pool.device, "K and V pools live on one GPU")
        raise ValueError("pools are contiguous")
    if dt is torch.uint8:
        _require(len(shape) == 3 and shape[2] % FP8_BLOCK_SIZE == 0,
                 "FP8 pools are [num_blocks, num_kv_heads, 16 * head_dim] uint8")
        _require(k_scale is not None and v_scale is not None, "FP8 pools need k_scale and v_scale")
        nb, hkv, n = shape
        return _Pool(k_pool.data_ptr(), v_pool.data_ptr(), nb, FP8_BLOCK_SIZE, hkv,
                     n // FP8_BLOCK_SIZE, PKV_FP8_E4M3, k_scale, v_scale)
    _require(len(shape) == 4, "pools are [num_blocks, num_kv_heads, block_size, head_dim]")
    nb, hkv, bs, d = shape
    return _Pool(k_pool.data_ptr(), v_pool.data_ptr(), nb, bs, hkv, d,
                 PKV_BF16 if dt is torch.bfloat16 else _dtype_code(dt), 0.0, 0.0)


def _on_device(t: Optional[torch.Tensor], name: str, device) -> None:
    """Buffers the kernels read or write must live on the pools' GPU: the
    pointer of a host tensor, or of another GPU's, would be dereferenced by
    the kernel."""
    if t is not None:
        _require(t.is_cuda and t.device == device, f"{name} lives on {device}")


def _status_ok(status: Optional[torch.Tensor], device) -> None:
    if status is not None:
        _on_device(status, "status", device)
        _require(status.dtype == torch.int32 and status.numel() >= 1, "status is an int32 word")


def _i32_dev(t: torch.Tensor, name: str, device) -> torch.Tensor:
    _require(t.dtype == torch.int32 and t.is_contiguous() and t.device == device,
             f"{name} is a contiguous int32 tensor on {device}")
    return t


@dataclass
class PrefixDesc:
    """Shared-prefix descriptor: device arrays plus the host-side bounds."""
    num_groups: int
    max_group_rows: int
    max_prefix_blocks: int
    group_of_row: torch.Tensor   # int32 [batch] on the device
    prefix_blocks: torch.Tensor  # int32 [num_groups] (at least 1 element) on the device

    def _c(self) -> _Prefix:
        return _Prefix(self.num_groups, self.max_group_rows, self.max_prefix_blocks,
                       self.group_of_row.data_ptr(), self.prefix_blocks.data_ptr())


def _prefix_ok(prefix: Optional[PrefixDesc], device) -> None:
    if prefix is not None:
        _i32_dev(prefix.group_of_row, "prefix.group_of_row", device)
        _i32_dev(prefix.prefix_blocks, "prefix.prefix_blocks", device)


def prefix_groups_host(block_tables: np.ndarray, seq_lens: np.ndarray,
                       block_size: int) -> Tuple[np.ndarray, np.ndarray]:
    """Shared-prefix groups of host block tables (library helper)."""
    t = np.ascontiguousarray(block_tables, dtype=np.int32)
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    B = t.shape[0]
    gor = np.empty(B, dtype=np.int32)
    pb = np.zeros(max(B, 1), dtype=np.int32)
    n = _lib.pkv_prefix_groups_host(t.ctypes.data, t.shape[1], sl.ctypes.data, B, block_size,
                                    gor.ctypes.data, pb.ctypes.data)
    if n < 0:
        raise ValueError("pkv_prefix_groups_host: invalid arguments")
    return gor, pb[:n].copy()


def make_prefix_desc(block_tables: np.ndarray, seq_lens: np.ndarray, block_size: int,
                     device) -> Optional[PrefixDesc]:
    """Derive the groups on the host and upload them; None when no rows share."""
    gor, pb = prefix_groups_host(block_tables, seq_lens, block_size)
    if len(pb) == 0:
        return None
    counts = np.bincount(gor[gor >= 0], minlength=len(pb))
    return PrefixDesc(len(pb), int(counts.max()), int(pb.max()),
                      torch.from_numpy(gor).to(device), torch.from_numpy(pb).to(device))


def slot_mapping_host(block_tables: np.ndarray, num_blocks: int, rows: np.ndarray,
                      positions: np.ndarray, block_size: int) -> np.ndarray:
    """slot = table[row][pos // bs] * bs + pos % bs (library helper); raises on a missing entry."""
    t = np.ascontiguousarray(block_tables, dtype=np.int32)
    r = np.ascontiguousarray(rows, dtype=np.int32)
    p = np.ascontiguousarray(positions, dtype=np.int32)
    out = np.empty(r.shape[0], dtype=np.int32)
    code = _lib.pkv_slot_mapping_host(t.ctypes.data, t.shape[1], t.shape[0], num_blocks,
                                      r.ctypes.data, p.ctypes.data, r.shape[0], block_size,
                                      out.ctypes.data)
    _check("pkv_slot_mapping_host", code)
    return out


def check_slot_mapping(slots: np.ndarray, num_blocks: int, block_size: int) -> None:
    """Debug check before an append (library helper, host arrays): every slot
    >= 0 inside the pool and no slot named by two tokens (their stores would
    race).  Raises ValueError naming the first token at fault."""
    s = np.ascontiguousarray(slots, dtype=np.int32)
    bad = ctypes.c_int32(-1)
    code = _lib.pkv_slot_mapping_check_host(s.ctypes.data, s.shape[0], num_blocks, block_size,
                                            ctypes.byref(bad))
    if code != PKV_OK:
        if bad.value < 0:
            raise ValueError("check_slot_mapping: invalid arguments")
        slot = int(s[bad.value])
        what = "lies past the pool" if slot >= num_blocks * block_size else "repeats an earlier token's"
        raise ValueError(f"check_slot_mapping: token {bad.value}'s slot {slot} {what}")


def paged_kv_append(k_pool: torch.Tensor, v_pool: torch.Tensor, slot_mapping: torch.Tensor,
                    k_new: torch.Tensor, v_new: torch.Tensor,
                    status: Optional[torch.Tensor] = None, k_scale: Optional[float] = None,
                    v_scale: Optional[float] = None) -> None:
    """Write ``k_new``/``v_new`` [T, Hkv, D] into the pools at ``slot_mapping`` [T]
    (quantized with ``k_scale``/``v_scale`` into FP8 pools)."""
    pool = _pool(k_pool, v_pool, k_scale, v_scale)
    dev = k_pool.device
    _i32_dev(slot_mapping, "slot_mapping", dev)
    _require(k_new.shape == v_new.shape and k_new.dim() == 3 and
             k_new.shape[1:] == (pool.num_kv_heads, pool.head_dim),
             "k_new/v_new are [T, num_kv_heads, head_dim]")
    act = _act_dtype(k_pool.dtype)
    _require(k_new.dtype == act and v_new.dtype == act, "new rows match the pool dtype (bf16 for FP8)")
    _require(k_new.is_contiguous() and v_new.is_contiguous(), "new rows are contiguous")
    _require(slot_mapping.dim() == 1 and slot_mapping.shape[0] == k_new.shape[0],
             "one slot per new token")
    _on_device(k_new, "k_new", dev)
    _on_device(v_new, "v_new", dev)
    _status_ok(status, dev)
    with _on(dev):
        _check("paged_kv_append", _lib.paged_kv_append(
            ctypes.byref(pool), slot_mapping.data_ptr(), k_new.shape[0], k_new.data_ptr(),
            v_new.data_ptr(), _ptr(status), _stream(dev)))


class RopeDesc:
    """Rotary descriptor (host memory, passed by value into every launch)."""

    def __init__(self, c: _Rope):
        self._c, self.rotary_dim, self.num_axes = c, int(c.rotary_dim), int(c.num_axes)


def make_rope(inv_freq, axis_of_pair=None, num_axes: Optional[int] = None, interleaved: bool = False,
              factor: float = 1.0) -> RopeDesc:
    """Rotary descriptor of ``rotary_dim = 2 * len(inv_freq)`` dims: pair i turns
    by ``positions[axis_of_pair[i]] * inv_freq[i]`` radians (float64).
    ``axis_of_pair`` defaults to one axis, ``num_axes`` to its largest entry + 1;
    ``interleaved`` pairs (2i, 2i + 1) instead of (i, i + rotary_dim / 2);
    ``factor`` multiplies the rotated dims."""
    f = np.ascontiguousarray(np.asarray(inv_freq, dtype=np.float64)).reshape(-1)
    a = None
    if axis_of_pair is not None:
        a = np.ascontiguousarray(np.asarray(axis_of_pair, dtype=np.int32)).reshape(-1)
        _require(a.shape == f.shape, "one axis per pair")
    if num_axes is None:
        num_axes = int(a.max()) + 1 if a is not None and a.size else 1
    c = _Rope()
    _check("pkv_rope_init", _lib.pkv_rope_init(
        ctypes.byref(c), 2 * f.size, f.ctypes.data if f.size else None, num_axes,
        a.ctypes.data if a is not None else None, int(interleaved), float(factor)))
    return RopeDesc(c)


def _token_stride(strides, tokens: int, rows: int, dim: int) -> int:
    """Elements between a [tokens, rows, dim] operand's tokens, -1 when a token's rows are not contiguous."""
    a, b, c = strides
    if (c != 1 and dim != 1) or (b != dim and rows != 1):
        return -1
    return a if tokens > 1 else rows * dim


def _rope_refuse(pool, dev, act, slot_mapping, q, k_new, v_new, positions, rope, q_out, status):
    """The messages of paged_kv_append_rope's checks."""
    hkv, D = pool.num_kv_heads, pool.head_dim
    _i32_dev(slot_mapping, "slot_mapping", dev)
    T = slot_mapping.shape[0] if slot_mapping.dim() == 1 else -1
    for t, name in ((k_new, "k_new"), (v_new, "v_new"), (q, "q"), (q_out, "q_out")):
        if t is None:
            continue
        _on_device(t, name, dev)
        _require(t.dtype == act, f"{name} matches the pool dtype (bf16 for FP8)")
        _require(t.dim() == 3 and t.shape[0] == T and t.shape[2] == D and
                 (name[0] == "q" or t.shape[1] == hkv),
                 f"{name} is [T, heads, head_dim], one slot per token")
        _require(_token_stride(t.stride(), t.shape[0], t.shape[1], D) >= 0 or t.numel() == 0,
                 f"{name}: each token's [heads, head_dim] rows are contiguous")
    _require(q is not None or q_out is None, "q_out without q")
    _require(q_out is None or q_out.shape == q.shape, "q_out matches q")
    _require(positions.dtype == torch.int32 and positions.device == dev and
             (positions.shape == (rope.num_axes, T) or (rope.num_axes == 1 and positions.shape == (T,))) and
             (positions.stride(-1) == 1 or T <= 1),
             "positions are int32 [num_axes, T] (or [T]) on the pools' GPU, each axis contiguous")
    _status_ok(status, dev)


def paged_kv_append_rope(k_pool: torch.Tensor, v_pool: torch.Tensor, slot_mapping: torch.Tensor,
                         q: Optional[torch.Tensor], k_new: torch.Tensor, v_new: torch.Tensor,
                         positions: torch.Tensor, rope: RopeDesc,
                         q_out: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None, k_scale: Optional[float] = None,
                         v_scale: Optional[float] = None) -> Optional[torch.Tensor]:
    """Rotate ``q`` [T, Hq, D] and ``k_new`` [T, Hkv, D] by ``positions`` ([T], or
    [num_axes, T], which may be one row expanded; int32) and append the rotated k
    and ``v_new`` into the pools at ``slot_mapping`` [T]; returns the rotated q
    (``q_out``, which may be ``q``).
    Token rows may be cut from a wider projection output.  ``q`` None: k alone."""
    pool = _pool(k_pool, v_pool, k_scale, v_scale)
    gpu, pdt = k_pool.get_device(), k_pool.dtype
    act = torch.float32 if pdt is torch.float32 else torch.bfloat16
    hkv, D, T, axes, i32 = pool.num_kv_heads, pool.head_dim, slot_mapping.numel(), rope.num_axes, torch.int32
    kshape, pshape = k_new.shape, positions.shape
    ok = (slot_mapping.dtype is i32 and slot_mapping.ndim == 1 and slot_mapping.is_contiguous() and
          slot_mapping.get_device() == gpu and kshape == (T, hkv, D) and v_new.shape == kshape and
          k_new.dtype is act and v_new.dtype is act and k_new.get_device() == gpu and
          v_new.get_device() == gpu and positions.dtype is i32 and positions.get_device() == gpu and
          (pshape == (axes, T) or (axes == 1 and pshape == (T,))) and
          (positions.is_contiguous() or positions.stride(-1) == 1 or T <= 1) and
          (status is None or (status.get_device() == gpu and status.dtype is i32 and status.numel() >= 1)))
    ks = vs = qs = os_ = 0
    hq, qp, op = 0, None, None
    if ok:
        ks = _token_stride(k_new.stride(), T, hkv, D)
        vs = _token_stride(v_new.stride(), T, hkv, D)
        if q is None:
            ok = q_out is None
        else:
            qshape = q.shape
            ok = len(qshape) == 3 and qshape[0] == T and qshape[2] == D and q.dtype is act and \
                q.get_device() == gpu and \
                (q_out is None or (q_out.shape == qshape and q_out.dtype is act and q_out.get_device() == gpu))
            if ok:
                if q_out is None:
                    q_out = torch.empty(qshape, dtype=act, device=q.device)
                hq, qp, op = qshape[1], q.data_ptr(), q_out.data_ptr()
                if hq:
                    qs = _token_stride(q.stride(), T, hq, D)
                    os_ = _token_stride(q_out.stride(), T, hq, D)
        ok = ok and (T == 0 or (ks >= 0 and vs >= 0 and qs >= 0 and os_ >= 0))
    if not ok:
        _rope_refuse(pool, k_pool.device, act, slot_mapping, q, k_new, v_new, positions, rope, q_out, status)
        raise ValueError("paged_kv_append_rope: invalid arguments")
    args = (ctypes.byref(pool), slot_mapping.data_ptr(), T, qp, qs, hq, k_new.data_ptr(), ks,
            v_new.data_ptr(), vs, positions.data_ptr(), positions.stride(0) if axes > 1 else T,
            ctypes.byref(rope._c), op, os_, None if status is None else status.data_ptr(), _raw_stream(gpu))
    if _current_device() == gpu:
        code = _lib.paged_kv_append_rope(*args)
    else:
        with torch.cuda.device(gpu):
            code = _lib.paged_kv_append_rope(*args)
    if code != PKV_OK:
        raise PkvError("paged_kv_append_rope", code)
    return q_out


class PoolSet:
    """The (K, V) pools of several layers that share block ids, checked once: what
    ``paged_copy_blocks`` copies in.  Holds the tensors."""

    def __init__(self, pools):
        self.pools = [(k, v) for k, v in pools]
        _require(len(self.pools) > 0, "at least one pool")
        self.device, self.n = self.pools[0][0].device, len(self.pools)
        self.gpu = self.pools[0][0].get_device()
        # page copies move bytes: FP8 scales play no part
        self._c = (_Pool * len(self.pools))(*[_pool(k, v, 1.0, 1.0) for k, v in self.pools])
        f = self._c[0]
        for (k, v), c in zip(self.pools, self._c):
            _require(k.device == self.device and v.device == self.device, "every pool on one GPU")
            _require((c.dtype, c.block_size, c.num_kv_heads, c.head_dim) ==
                     (f.dtype, f.block_size, f.num_kv_heads, f.head_dim),
                     "the pools share dtype, block size, kv heads and head_dim")

    def __len__(self) -> int:
        return self.n


def paged_copy_blocks(pools: PoolSet, src_blocks: torch.Tensor, dst_blocks: torch.Tensor,
                      dst_pools: Optional[PoolSet] = None,
                      status: Optional[torch.Tensor] = None) -> None:
    """Copy pages ``src_blocks[i]`` of every pool to pages ``dst_blocks[i]`` (int32
    [n]) of the same pool, or of ``dst_pools``'; negative ids are skipped.  Within
    a call no page may be written twice, nor written and read
    (``check_block_copies``)."""
    gpu, n, i32 = pools.gpu, src_blocks.numel(), torch.int32
    if not (src_blocks.dtype is i32 and dst_blocks.dtype is i32 and src_blocks.dim() == 1 and
            dst_blocks.shape == src_blocks.shape and src_blocks.get_device() == gpu and
            dst_blocks.get_device() == gpu and src_blocks.is_contiguous() and dst_blocks.is_contiguous() and
            (dst_pools is None or (dst_pools.gpu == gpu and dst_pools.n == pools.n)) and
            (status is None or (status.get_device() == gpu and status.dtype is i32 and status.numel() >= 1))):
        dev = pools.device
        _i32_dev(src_blocks, "src_blocks", dev)
        _i32_dev(dst_blocks, "dst_blocks", dev)
        _require(src_blocks.dim() == 1 and src_blocks.shape == dst_blocks.shape,
                 "one destination page per source page")
        _status_ok(status, dev)
        raise ValueError("as many destination pools as source pools, on one GPU")
    args = (pools._c, None if dst_pools is None else dst_pools._c, pools.n, src_blocks.data_ptr(),
            dst_blocks.data_ptr(), n, None if status is None else status.data_ptr(), _raw_stream(gpu))
    if _current_device() == gpu:
        code = _lib.paged_copy_blocks(*args)
    else:
        with torch.cuda.device(gpu):
            code = _lib.paged_copy_blocks(*args)
    if code != PKV_OK:
        raise PkvError("paged_copy_blocks", code)


def check_block_copies(src_blocks, dst_blocks, num_blocks: int,
                       dst_num_blocks: Optional[int] = None) -> None:
    """Debug check of a page copy list (library helper, host arrays): ids inside
    the pools, no page written twice or both written and read.  Raises ValueError
    naming the first pair at fault.  ``dst_num_blocks``: the destination is
    another pool, of that size."""
    s = np.ascontiguousarray(np.asarray(src_blocks, dtype=np.int32)).reshape(-1)
    d = np.ascontiguousarray(np.asarray(dst_blocks, dtype=np.int32)).reshape(-1)
    _require(s.shape == d.shape, "one destination page per source page")
    bad = ctypes.c_int32(-1)
    same = dst_num_blocks is None
    code = _lib.pkv_block_copies_check_host(s.ctypes.data, d.ctypes.data, s.size, num_blocks,
                                            num_blocks if same else dst_num_blocks, int(same),
                                            ctypes.byref(bad))
    if code != PKV_OK:
        if bad.value < 0:
            raise ValueError("check_block_copies: invalid arguments")
        raise ValueError(f"check_block_copies: pair {bad.value} ({int(s[bad.value])} -> "
                         f"{int(d[bad.value])}) lies past a pool or meets an earlier pair's page")


def decode_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                          block_size: int, max_seq_len: int, window: int = 0,
                          prefix: Optional[PrefixDesc] = None, sinks: int = 0) -> int:
    if sinks and prefix is None:
        return int(_lib.paged_decode_sinks_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                          block_size, max_seq_len, window, sinks))
    px = ctypes.byref(prefix._c()) if prefix is not None else None
    return int(_lib.paged_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                block_size, max_seq_len, window, px))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    """A 256-byte-aligned device buffer (torch allocations are)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def paged_decode_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                           block_tables: torch.Tensor, seq_lens: torch.Tensor, window: int,
                           scale: float, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None,
                           max_seq_len: Optional[int] = None,
                           prefix: Optional[PrefixDesc] = None,
                           status: Optional[torch.Tensor] = None,
                           k_scale: Optional[float] = None,
                           v_scale: Optional[float] = None, sinks: int = 0) -> torch.Tensor:
    """Batched paged decode attention; returns ``out`` [B, Hq, D].

    ``max_seq_len`` is a host bound on ``seq_lens`` (default: the block-table
    capacity); ``workspace`` defaults to a fresh buffer of the queried size.
    FP8 pools (uint8) take bf16 queries and their ``k_scale``/``v_scale``.
    With a ``window``, the first ``sinks`` positions of a row stay visible
    (not together with ``prefix``).
    """
    pool = _pool(k_pool, v_pool, k_scale, v_scale)
    gpu, i32, qshape, tshape = k_pool.get_device(), torch.int32, q.shape, block_tables.shape
    if not (len(qshape) == 3 and qshape[2] == pool.head_dim and q.is_contiguous() and
            q.get_device() == gpu and q.dtype is (torch.float32 if pool.dtype == PKV_F32 else torch.bfloat16) and
            block_tables.dtype is i32 and block_tables.is_contiguous() and
            block_tables.get_device() == gpu and len(tshape) == 2 and tshape[0] == qshape[0] and
            seq_lens.dtype is i32 and seq_lens.is_contiguous() and seq_lens.get_device() == gpu and
            seq_lens.shape == qshape[:1] and
            (out is None or (out.shape == qshape and out.dtype is q.dtype and out.is_contiguous() and
                             out.get_device() == gpu)) and
            (workspace is None or workspace.get_device() == gpu) and
            (status is None or (status.get_device() == gpu and status.dtype is i32 and status.numel() >= 1))):
        dev = k_pool.device
        _require(q.dim() == 3 and q.shape[2] == pool.head_dim and q.dtype == _act_dtype(k_pool.dtype) and
                 q.is_contiguous() and q.device == dev, "q is [B, Hq, D], contiguous, pool dtype")
        _i32_dev(block_tables, "block_tables", dev)
        _i32_dev(seq_lens, "seq_lens", dev)
        _require(block_tables.dim() == 2 and block_tables.shape[0] == q.shape[0] and
                 seq_lens.shape == q.shape[:1], "block_tables [B, max_blocks], seq_lens [B]")
        _on_device(out, "out", dev)
        _require(out is None or (out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous()),
                 "out matches q")
        _on_device(workspace, "workspace", dev)
        _status_ok(status, dev)
        raise ValueError("paged_decode_attention: invalid arguments")
    B, hq, D = qshape
    width = tshape[1]
    if max_seq_len is None:
        max_seq_len = width * pool.block_size
    if prefix is not None:
        _prefix_ok(prefix, k_pool.device)
        if sinks and (window or sinks < 0):
            raise PkvError("paged_decode_attention (sinks with a shared prefix)",
                           PKV_ERR_UNSUPPORTED if sinks > 0 else PKV_ERR_INVALID_ARG)
    # the plan reads the SM count of the current device
    with _NULL if _current_device() == gpu else torch.cuda.device(gpu):
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            workspace = alloc_workspace(
                decode_workspace_size(B, hq, pool.num_kv_heads, D, pool.block_size, max_seq_len, window,
                                      prefix, sinks), k_pool.device)
        ws, nbytes = workspace.data_ptr(), workspace.nbytes
        st = None if status is None else status.data_ptr()
        if sinks and prefix is None:
            code = _lib.paged_decode_attention_sinks(
                q.data_ptr(), hq, ctypes.byref(pool), block_tables.data_ptr(), width, seq_lens.data_ptr(),
                B, max_seq_len, window, sinks, scale, out.data_ptr(), ws, nbytes, st, _raw_stream(gpu))
        else:
            code = _lib.paged_decode_attention(
                q.data_ptr(), hq, ctypes.byref(pool), block_tables.data_ptr(), width, seq_lens.data_ptr(),
                B, max_seq_len, window, scale, out.data_ptr(), ws, nbytes,
                ctypes.byref(prefix._c()) if prefix is not None else None, st, _raw_stream(gpu))
    if code != PKV_OK:
        raise PkvError("paged_decode_attention_sinks" if sinks else "paged_decode_attention", code)
    return out


def prefill_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                           block_size: int, max_q_len: int, max_seq_len: int,
                           window: int = 0, sinks: int = 0) -> int:
    if sinks:
        return int(_lib.paged_prefill_sinks_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                           block_size, max_q_len, max_seq_len, window,
                                                           sinks))
    return int(_lib.paged_prefill_workspace_size(batch, num_q_heads, num_kv_heads, head_dim,
                                                 block_size, max_q_len, max_seq_len, window))


def paged_prefill_chunk_attention(q: torch.Tensor, cu_q_lens: torch.Tensor, k_pool: torch.Tensor,
                                  v_pool: torch.Tensor, block_tables: torch.Tensor,
                                  seq_lens: torch.Tensor, max_q_len: int, window: int,
                                  scale: float, out: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None,
                                  max_seq_len: Optional[int] = None,
                                  status: Optional[torch.Tensor] = None,
                                  k_scale: Optional[float] = None,
                                  v_scale: Optional[float] = None, sinks: int = 0) -> torch.Tensor:
    """Chunked prefill against the paged prefix; returns ``out`` [sum C, Hq, D].
    With a ``window``, the first ``sinks`` positions of a row stay visible."""
    pool = _pool(k_pool, v_pool, k_scale, v_scale)
    dev = k_pool.device
    _require(q.dim() == 3 and q.shape[2] == pool.head_dim and q.dtype == _act_dtype(k_pool.dtype) and
             q.is_contiguous() and q.device == dev, "q is [sum C, Hq, D], contiguous, pool dtype")
    _i32_dev(cu_q_lens, "cu_q_lens", dev)
    _i32_dev(block_tables, "block_tables", dev)
    _i32_dev(seq_lens, "seq_lens", dev)
    B = seq_lens.shape[0]
    _require(cu_q_lens.shape == (B + 1,) and block_tables.shape[0] == B,
             "cu_q_lens [B+1], block_tables [B, max_blocks]")
    width = block_tables.shape[1]
    if max_seq_len is None:
        max_seq_len = width * pool.block_size
    if out is None:
        out = torch.empty_like(q)
    _require(out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous(), "out matches q")
    _on_device(out, "out", dev)
    _on_device(workspace, "workspace", dev)
    _status_ok(status, dev)
    hq = q.shape[1]
    with _on(dev):  # the plan reads the SM count of the current device
        if workspace is None:
            workspace = alloc_workspace(
                prefill_workspace_size(B, hq, pool.num_kv_heads, pool.head_dim, pool.block_size,
                                       max_q_len, max_seq_len, window, sinks), dev)
        if sinks:
            _check("paged_prefill_chunk_attention_sinks", _lib.paged_prefill_chunk_attention_sinks(
                q.data_ptr(), cu_q_lens.data_ptr(), hq, ctypes.byref(pool), block_tables.data_ptr(),
                width, seq_lens.data_ptr(), B, max_q_len, max_seq_len, window, sinks, scale,
                out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                _ptr(status), _stream(dev)))
            return out
        _check("paged_prefill_chunk_attention", _lib.paged_prefill_chunk_attention(
            q.data_ptr(), cu_q_lens.data_ptr(), hq, ctypes.byref(pool), block_tables.data_ptr(),
            width, seq_lens.data_ptr(), B, max_q_len, max_seq_len, window, float(scale),
            out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _ptr(status), _stream(dev)))
    return out


def tree_masks_host(parents, cu_q_lens) -> np.ndarray:
    """Masks of drafted trees (library helper, host arrays): node i of row r, at
    ``cu_q_lens[r] + i``, has parent ``parents[..]`` in -1 .. i - 1 (-1: the last
    cached token) and attends its ancestors and itself.  int64 bit patterns, as
    ``paged_tree_attention`` and ``paged_latent_attention`` take them."""
    up = np.ascontiguousarray(np.asarray(parents, dtype=np.int32)).reshape(-1)
    cu = np.ascontiguousarray(np.asarray(cu_q_lens, dtype=np.int32)).reshape(-1)
    _require(cu.size >= 1 and cu[0] == 0 and cu[-1] == up.size, "cu_q_lens runs from 0 to the number of parents")
    _require(bool((np.diff(cu) >= 0).all()), "cu_q_lens does not descend")
    out = np.empty(up.size, dtype=np.int64)
    _check("pkv_tree_masks_host", _lib.pkv_tree_masks_host(
        up.ctypes.data if up.size else None, cu.ctypes.data, cu.size - 1, out.ctypes.data if up.size else None))
    return out


def tree_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
                        max_q_len: int, max_seq_len: int, window: int = 0) -> int:
    return int(_lib.paged_tree_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, block_size,
                                              max_q_len, max_seq_len, window))


def _status_word(status, gpu) -> bool:
    return status is None or (status.get_device() == gpu and status.dtype is torch.int32 and status.numel() >= 1)


def paged_tree_attention(q: torch.Tensor, cu_q_lens: torch.Tensor, tree_masks: torch.Tensor,
                         k_pool: torch.Tensor, v_pool: torch.Tensor, block_tables: torch.Tensor,
                         seq_lens: torch.Tensor, max_q_len: int, window: int, scale: float,
                         out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         max_seq_len: Optional[int] = None, status: Optional[torch.Tensor] = None,
                         k_scale: Optional[float] = None, v_scale: Optional[float] = None) -> torch.Tensor:
    """Attention of drafted trees against the paged cache; returns ``out`` [sum C, Hq, D].

    Row r's ``C`` drafts sit at the last ``C`` positions of its ``seq_lens``; draft
    i's query attends the cached tokens and the drafts whose bits ``tree_masks``
    [sum C] (int64 bit patterns, ``tree_masks_host``) has set, j <= i.  With a
    ``window`` (at least ``max_q_len``) a node counts from its depth in the tree.
    ``max_q_len`` is at most ``MAX_TREE``.  A row whose drafts lie past ``q`` is left
    out (``DEV_BAD_LEN``)."""
    pool = _pool(k_pool, v_pool, k_scale, v_scale)
    gpu, i32, qshape, tshape = k_pool.get_device(), torch.int32, q.shape, block_tables.shape
    if not (len(qshape) == 3 and qshape[2] == pool.head_dim and q.is_contiguous() and q.get_device() == gpu and
            q.dtype is (torch.float32 if pool.dtype == PKV_F32 else torch.bfloat16) and
            block_tables.dtype is i32 and block_tables.is_contiguous() and block_tables.get_device() == gpu and
            len(tshape) == 2 and seq_lens.dtype is i32 and seq_lens.is_contiguous() and
            seq_lens.get_device() == gpu and seq_lens.ndim == 1 and seq_lens.numel() == tshape[0] and
            cu_q_lens.dtype is i32 and cu_q_lens.is_contiguous() and cu_q_lens.get_device() == gpu and
            cu_q_lens.ndim == 1 and cu_q_lens.numel() == tshape[0] + 1 and
            tree_masks.dtype is torch.int64 and tree_masks.ndim == 1 and tree_masks.numel() == qshape[0] and
            tree_masks.is_contiguous() and tree_masks.get_device() == gpu and
            (out is None or (out.shape == qshape and out.dtype is q.dtype and out.is_contiguous() and
                             out.get_device() == gpu)) and
            (workspace is None or (workspace.get_device() == gpu and workspace.is_contiguous())) and
            (status is None or _status_word(status, gpu))):
        dev = k_pool.device
        _require(q.dim() == 3 and q.shape[2] == pool.head_dim and q.dtype == _act_dtype(k_pool.dtype) and
                 q.is_contiguous() and q.device == dev, "q is [sum C, Hq, D], contiguous, pool dtype")
        _i32_dev(cu_q_lens, "cu_q_lens", dev)
        _i32_dev(block_tables, "block_tables", dev)
        _i32_dev(seq_lens, "seq_lens", dev)
        _require(block_tables.dim() == 2 and seq_lens.shape == block_tables.shape[:1] and
                 cu_q_lens.shape == (block_tables.shape[0] + 1,),
                 "block_tables [B, max_blocks], seq_lens [B], cu_q_lens [B+1]")
        _require(tree_masks.dtype == torch.int64 and tree_masks.shape == q.shape[:1] and
                 tree_masks.is_contiguous() and tree_masks.device == dev,
                 f"tree_masks are contiguous int64 [sum C] on {dev}")
        _on_device(out, "out", dev)
        _require(out is None or (out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous()),
                 "out matches q")
        _on_device(workspace, "workspace", dev)
        _status_ok(status, dev)
        raise ValueError("paged_tree_attention: invalid arguments")
    B, width = tshape
    hq = qshape[1]
    if max_seq_len is None:
        max_seq_len = width * pool.block_size
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        with torch.cuda.device(gpu):  # the plan reads the SM count of the current device
            workspace = alloc_workspace(
                tree_workspace_size(B, hq, pool.num_kv_heads, pool.head_dim, pool.block_size, max_q_len,
                                    max_seq_len, window), k_pool.device)
    args = (q.data_ptr(), qshape[0], cu_q_lens.data_ptr(), tree_masks.data_ptr(), hq, ctypes.byref(pool),
            block_tables.data_ptr(), width, seq_lens.data_ptr(), B, max_q_len, max_seq_len, window, scale,
            out.data_ptr(), workspace.data_ptr(), workspace.nbytes,
            None if status is None else status.data_ptr(), _raw_stream(gpu))
    if _current_device() == gpu:
        code = _lib.paged_tree_attention_queries(*args)
    else:
        with torch.cuda.device(gpu):
            code = _lib.paged_tree_attention_queries(*args)
    if code != PKV_OK:
        raise PkvError("paged_tree_attention", code)
    return out


def _latent_pool(pool: torch.Tensor, latent_dim: int, shape, dt, gpu: int) -> _LatentPool:
    if not (len(shape) == 3 and gpu >= 0 and pool.is_contiguous() and 0 < latent_dim < shape[2]):
        _require(len(shape) == 3, "a latent pool is [num_blocks, block_size, latent_dim + rope_dim]")
        _require(gpu >= 0, "pools live on the GPU")
        _require(pool.is_contiguous(), "pools are contiguous")
        raise ValueError("latent_dim lies below the pool's row")
    return _LatentPool(pool.data_ptr(), shape[0], shape[1], latent_dim, shape[2] - latent_dim,
                       PKV_BF16 if dt is torch.bfloat16 else _dtype_code(dt))


class LatentPoolSet:
    """The latent pools [num_blocks, block_size, latent_dim + rope_dim] of several
    layers that share block ids, checked once: what ``paged_tree_commit`` moves
    rows in.  Holds the tensors."""

    def __init__(self, pools):
        self.pools = list(pools)
        _require(len(self.pools) > 0, "at least one pool")
        self.device, self.n, self.gpu = self.pools[0].device, len(self.pools), self.pools[0].get_device()
        # rows move whole: where the latent ends plays no part
        self._c = (_LatentPool * self.n)(*[_latent_pool(t, t.shape[-1] - 1, t.shape, t.dtype, t.get_device())
                                           for t in self.pools])
        f = self.pools[0]
        for t in self.pools:
            _require(t.device == self.device, "every pool on one GPU")
            _require(t.dtype == f.dtype and t.shape[1:] == f.shape[1:], "the pools share dtype, block size and row")

    def __len__(self) -> int:
        return self.n


def paged_tree_commit(pools, block_tables: torch.Tensor, seq_lens: torch.Tensor, cu_q_lens: torch.Tensor,
                      path: torch.Tensor, path_lens: torch.Tensor, new_seq_lens: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Move the rows of an accepted path behind the cached tokens, in every pool of
    ``pools`` (a ``PoolSet`` or a ``LatentPoolSet``); returns the rows' new lengths.

    ``path`` [B, max_path] holds draft indexes, strictly ascending, of which row r's
    first ``path_lens[r]`` count: draft ``path[r, i]``'s row goes to position n + i
    (n: the row's tokens before its drafts)."""
    gpu, i32 = pools.gpu, torch.int32
    tshape, pshape = block_tables.shape, path.shape
    if not (block_tables.dtype is i32 and seq_lens.dtype is i32 and cu_q_lens.dtype is i32 and path.dtype is i32 and
            path_lens.dtype is i32 and block_tables.get_device() == gpu and seq_lens.get_device() == gpu and
            cu_q_lens.get_device() == gpu and path.get_device() == gpu and path_lens.get_device() == gpu and
            block_tables.is_contiguous() and seq_lens.is_contiguous() and cu_q_lens.is_contiguous() and
            path.is_contiguous() and path_lens.is_contiguous() and len(tshape) == 2 and len(pshape) == 2 and
            pshape[0] == tshape[0] and seq_lens.ndim == 1 and seq_lens.numel() == tshape[0] and
            path_lens.ndim == 1 and path_lens.numel() == tshape[0] and cu_q_lens.ndim == 1 and
            cu_q_lens.numel() == tshape[0] + 1 and
            (new_seq_lens is None or (new_seq_lens.dtype is i32 and new_seq_lens.ndim == 1 and
                                      new_seq_lens.numel() == tshape[0] and
                                      new_seq_lens.is_contiguous() and new_seq_lens.get_device() == gpu)) and
            (status is None or _status_word(status, gpu))):
        dev = pools.device
        for t, name in ((block_tables, "block_tables"), (seq_lens, "seq_lens"), (cu_q_lens, "cu_q_lens"),
                        (path, "path"), (path_lens, "path_lens"), (new_seq_lens, "new_seq_lens")):
            if t is not None:
                _i32_dev(t, name, dev)
        _status_ok(status, dev)
        raise ValueError("block_tables [B, max_blocks], path [B, max_path], seq_lens, path_lens and new_seq_lens "
                         "[B], cu_q_lens [B+1]")
    if new_seq_lens is None:
        new_seq_lens = torch.empty_like(seq_lens)
    call = _lib.paged_latent_tree_commit if isinstance(pools, LatentPoolSet) else _lib.paged_tree_commit
    args = (pools._c, pools.n, block_tables.data_ptr(), tshape[1], seq_lens.data_ptr(), cu_q_lens.data_ptr(),
            tshape[0], path.data_ptr(), pshape[1], path_lens.data_ptr(), new_seq_lens.data_ptr(),
            None if status is None else status.data_ptr(), _raw_stream(gpu))
    if _current_device() == gpu:
        code = call(*args)
    else:
        with torch.cuda.device(gpu):
            code = call(*args)
    if code != PKV_OK:
        raise PkvError("paged_tree_commit", code)
    return new_seq_lens


def _latent_append_refuse(dev, dt, slot_mapping, latent_new, k_rope_new, positions, rope, q_rope, q_rope_out,
                          norm_weight, status, row):
    """The messages of paged_latent_append's checks."""
    _i32_dev(slot_mapping, "slot_mapping", dev)
    T = slot_mapping.shape[0] if slot_mapping.dim() == 1 else -1
    for t, name in ((latent_new, "latent_new"), (k_rope_new, "k_rope_new"), (q_rope, "q_rope"),
                    (q_rope_out, "q_rope_out"), (norm_weight, "norm_weight")):
        if t is not None:
            _on_device(t, name, dev)
            _require(t.dtype == dt, f"{name} matches the pool dtype")
            _require(t.numel() == 0 or t.shape[-1] == 1 or t.stride(-1) == 1, f"{name}'s rows are contiguous")
    _require(latent_new.dim() == 2 and k_rope_new.dim() == 2 and latent_new.shape[0] == T and
             k_rope_new.shape[0] == T and latent_new.shape[1] + k_rope_new.shape[1] == row,
             "latent_new [T, latent_dim] and k_rope_new [T, rope_dim] make up the pool's rows, one slot per token")
    _require(norm_weight is None or norm_weight.shape == latent_new.shape[1:], "norm_weight is [latent_dim]")
    _require(q_rope is not None or q_rope_out is None, "q_rope_out without q_rope")
    _require(q_rope is None or (q_rope.dim() == 3 and q_rope.shape[0] == T and q_rope.shape[2] == k_rope_new.shape[1]),
             "q_rope is [T, heads, rope_dim]")
    _require(q_rope_out is None or q_rope_out.shape == q_rope.shape, "q_rope_out matches q_rope")
    _require(positions.dtype == torch.int32 and positions.device == dev and
             (positions.shape == (rope.num_axes, T) or (rope.num_axes == 1 and positions.shape == (T,))) and
             (positions.stride(-1) == 1 or T <= 1),
             "positions are int32 [num_axes, T] (or [T]) on the pool's GPU, each axis contiguous")
    _status_ok(status, dev)


def paged_latent_append(pool: torch.Tensor, slot_mapping: torch.Tensor, latent_new: torch.Tensor,
                        k_rope_new: torch.Tensor, positions: torch.Tensor, rope: RopeDesc,
                        q_rope: Optional[torch.Tensor] = None, q_rope_out: Optional[torch.Tensor] = None,
                        norm_weight: Optional[torch.Tensor] = None, norm_eps: float = 1e-6,
                        status: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Write the rows [latent | rotated key] of ``latent_new`` [T, R] and ``k_rope_new``
    [T, Dr] into the latent ``pool`` [num_blocks, block_size, R + Dr] at
    ``slot_mapping`` [T], the latent normalised by its root mean square and
    ``norm_weight`` [R] where that is given; returns ``q_rope`` [T, H, Dr] rotated
    (``q_rope_out``, which may be ``q_rope`` or the tail of the absorbed queries).
    Token rows may be cut from wider tensors.  ``positions`` as for
    ``paged_kv_append_rope``; the descriptor's rotary_dim is Dr."""
    shape, dt, gpu, i32, rows = latent_new.shape, pool.dtype, pool.get_device(), torch.int32, pool.shape
    T, axes, kshape, pshape = slot_mapping.numel(), rope.num_axes, k_rope_new.shape, positions.shape
    cs, ks, ps = latent_new.stride(), k_rope_new.stride(), positions.stride()
    ok = (len(shape) == 2 and shape[0] == T and len(kshape) == 2 and kshape[0] == T and len(rows) == 3 and
          shape[1] + kshape[1] == rows[2] and slot_mapping.dtype is i32 and slot_mapping.ndim == 1 and
          slot_mapping.is_contiguous() and slot_mapping.get_device() == gpu and
          latent_new.dtype is dt and k_rope_new.dtype is dt and latent_new.get_device() == gpu and
          k_rope_new.get_device() == gpu and
          (T == 0 or ((cs[1] == 1 or shape[1] == 1) and (ks[1] == 1 or kshape[1] == 1))) and
          positions.dtype is i32 and positions.get_device() == gpu and
          (pshape[0] == T if axes == 1 and len(ps) == 1 else pshape == (axes, T)) and (ps[-1] == 1 or T <= 1) and
          (norm_weight is None or (norm_weight.dtype is dt and norm_weight.ndim == 1 and
                                   norm_weight.numel() == shape[1] and norm_weight.get_device() == gpu and
                                   norm_weight.is_contiguous())) and
          (status is None or _status_word(status, gpu)))
    H, qp, op, qs, qh, os_, oh = 0, None, None, 0, 0, 0, 0
    if ok:
        if q_rope is None:
            ok = q_rope_out is None
        else:
            qshape = q_rope.shape
            ok = len(qshape) == 3 and qshape[0] == T and qshape[2] == kshape[1] and q_rope.dtype is dt and \
                q_rope.get_device() == gpu and \
                (q_rope_out is None or (q_rope_out.shape == qshape and q_rope_out.dtype is dt and
                                        q_rope_out.get_device() == gpu))
            if ok:
                if q_rope_out is None:
                    q_rope_out = torch.empty(qshape, dtype=dt, device=q_rope.device)
                H, qp, op = qshape[1], q_rope.data_ptr(), q_rope_out.data_ptr()
                (qs, qh, qd), (os_, oh, od) = q_rope.stride(), q_rope_out.stride()
                if H == 1:
                    qh = oh = qshape[2]
                if T == 1:
                    qs, os_ = H * qh, H * oh
                ok = T == 0 or H == 0 or (qd == 1 and od == 1)
    if not ok:
        _latent_append_refuse(pool.device, dt, slot_mapping, latent_new, k_rope_new, positions, rope, q_rope,
                              q_rope_out, norm_weight, status, pool.shape[-1])
        raise ValueError("paged_latent_append: invalid arguments")
    c = _latent_pool(pool, shape[1], rows, dt, gpu)
    args = (ctypes.byref(c), slot_mapping.data_ptr(), T, latent_new.data_ptr(),
            cs[0] if T > 1 else shape[1], k_rope_new.data_ptr(),
            ks[0] if T > 1 else kshape[1], None if norm_weight is None else norm_weight.data_ptr(),
            norm_eps, qp, qs, qh, H, positions.data_ptr(), ps[0] if axes > 1 else T,
            ctypes.byref(rope._c), op, os_, oh, None if status is None else status.data_ptr(), _raw_stream(gpu))
    if _current_device() == gpu:
        code = _lib.paged_latent_append(*args)
    else:
        with torch.cuda.device(gpu):
            code = _lib.paged_latent_append(*args)
    if code != PKV_OK:
        raise PkvError("paged_latent_append", code)
    return q_rope_out


def latent_workspace_size(batch: int, num_q_heads: int, latent_dim: int, rope_dim: int, block_size: int,
                          max_q_len: int, max_seq_len: int) -> int:
    return int(_lib.paged_latent_workspace_size(batch, num_q_heads, latent_dim, rope_dim, block_size, max_q_len,
                                                max_seq_len))


def paged_latent_attention(q: torch.Tensor, pool: torch.Tensor, latent_dim: int, block_tables: torch.Tensor,
                           seq_lens: torch.Tensor, scale: float, cu_q_lens: Optional[torch.Tensor] = None,
                           max_q_len: Optional[int] = None, tree_masks: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                           max_seq_len: Optional[int] = None,
                           status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention over a latent ``pool`` [num_blocks, block_size, R + Dr] in the absorbed
    form: ``q`` [queries, H, R + Dr] against whole rows, weighted sums of the rows'
    latents into ``out`` [queries, H, R] (R = ``latent_dim``).

    One query per row (decode) without ``cu_q_lens``; with it [B+1] the last C
    positions of each row hold a chunk's queries, causally, or, with ``tree_masks``,
    a drafted tree's (as for ``paged_tree_attention``).  ``max_q_len`` bounds C; left
    out it is the number of queries, which no row passes (a tight bound leaves fewer
    empty items to look at; the result is the same)."""
    gpu, i32, dt, rows = pool.get_device(), torch.int32, pool.dtype, pool.shape
    qshape, tshape = q.shape, block_tables.shape
    c = _latent_pool(pool, latent_dim, rows, dt, gpu)
    if max_q_len is None:
        max_q_len = 1 if cu_q_lens is None else qshape[0] if tree_masks is None else min(qshape[0], MAX_TREE)
    if not (len(qshape) == 3 and qshape[2] == rows[2] and q.is_contiguous() and q.get_device() == gpu and
            q.dtype is dt and block_tables.dtype is i32 and block_tables.is_contiguous() and
            block_tables.get_device() == gpu and len(tshape) == 2 and seq_lens.dtype is i32 and
            seq_lens.is_contiguous() and seq_lens.get_device() == gpu and seq_lens.ndim == 1 and
            seq_lens.numel() == tshape[0] and
            (qshape[0] == tshape[0] and max_q_len == 1 if cu_q_lens is None else
             (cu_q_lens.dtype is i32 and cu_q_lens.is_contiguous() and cu_q_lens.get_device() == gpu and
              cu_q_lens.ndim == 1 and cu_q_lens.numel() == tshape[0] + 1)) and
            (tree_masks is None or (cu_q_lens is not None and tree_masks.dtype is torch.int64 and
                                    tree_masks.ndim == 1 and tree_masks.numel() == qshape[0] and
                                    tree_masks.is_contiguous() and
                                    tree_masks.get_device() == gpu)) and
            (out is None or (out.shape == (qshape[0], qshape[1], latent_dim) and out.dtype is dt and
                             out.is_contiguous() and out.get_device() == gpu)) and
            (workspace is None or (workspace.get_device() == gpu and workspace.is_contiguous())) and
            (status is None or _status_word(status, gpu))):
        dev = pool.device
        _require(q.dim() == 3 and q.shape[2] == pool.shape[2] and q.dtype == dt and q.is_contiguous() and
                 q.device == dev, "q is [queries, H, latent_dim + rope_dim], contiguous, pool dtype")
        _i32_dev(block_tables, "block_tables", dev)
        _i32_dev(seq_lens, "seq_lens", dev)
        _require(block_tables.dim() == 2 and seq_lens.shape == block_tables.shape[:1],
                 "block_tables [B, max_blocks], seq_lens [B]")
        if cu_q_lens is None:
            _require(q.shape[0] == block_tables.shape[0] and max_q_len == 1, "one query per row without cu_q_lens")
            _require(tree_masks is None, "tree_masks go with cu_q_lens")
        else:
            _i32_dev(cu_q_lens, "cu_q_lens", dev)
            _require(cu_q_lens.shape == (block_tables.shape[0] + 1,), "cu_q_lens [B+1]")
            _require(tree_masks is None or (tree_masks.dtype == torch.int64 and tree_masks.shape == q.shape[:1] and
                                            tree_masks.is_contiguous() and tree_masks.device == dev),
                     f"tree_masks are contiguous int64 [queries] on {dev}")
        _on_device(out, "out", dev)
        _on_device(workspace, "workspace", dev)
        _status_ok(status, dev)
        raise ValueError("out is [queries, H, latent_dim], contiguous, pool dtype")
    B, width = tshape
    H = qshape[1]
    if max_seq_len is None:
        max_seq_len = width * c.block_size
    if out is None:
        out = torch.empty((qshape[0], H, latent_dim), dtype=dt, device=q.device)
    if workspace is None:
        with torch.cuda.device(gpu):  # the plan reads the SM count of the current device
            workspace = alloc_workspace(
                latent_workspace_size(B, H, latent_dim, c.rope_dim, c.block_size, max_q_len, max_seq_len),
                q.device)
    args = (q.data_ptr(), qshape[0], None if cu_q_lens is None else cu_q_lens.data_ptr(),
            None if tree_masks is None else tree_masks.data_ptr(), H, ctypes.byref(c), block_tables.data_ptr(),
            width, seq_lens.data_ptr(), B, max_q_len, max_seq_len, scale, out.data_ptr(), workspace.data_ptr(),
            workspace.nbytes, None if status is None else status.data_ptr(), _raw_stream(gpu))
    if _current_device() == gpu:
        code = _lib.paged_latent_attention(*args)
    else:
        with torch.cuda.device(gpu):
            code = _lib.paged_latent_attention(*args)
    if code != PKV_OK:
        raise PkvError("paged_latent_attention", code)
    return out


def set_decode_split_blocks(n: int) -> int:
    """Diagnostic split-size override (0 = automatic); returns the previous value."""
    return int(_lib.pkv_set_decode_split_blocks(n))


def decode_plan(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
                max_seq_len: int, window: int = 0) -> Tuple[int, int]:
    """(splits per row, blocks per split) of the automatic plan on the current device."""
    c = ctypes.c_int32(0)
    n = _lib.pkv_decode_plan(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_seq_len,
                             window, ctypes.byref(c))
    return int(n), int(c.value)


def version() -> str:
    return _lib.pkv_version().decode()


def profile_enable(kinds=()) -> None:
    """Time every launch of the given kernel kinds with CUDA events on its stream."""
    mask = 0
    for k in kinds:
        mask |= 1 << k
    _check("pkv_profile_enable", _lib.pkv_profile_enable(mask))


def profile_mask(kinds=()) -> None:
    """Change which kernel kinds are timed, keeping the records so far."""
    mask = 0
    for k in kinds:
        mask |= 1 << k
    _check("pkv_profile_mask", _lib.pkv_profile_mask(mask))


def profile_read(kind: int) -> Tuple[int, float]:
    """(launches, summed device milliseconds) recorded for a kernel kind."""
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    _check("pkv_profile_read", _lib.pkv_profile_read(kind, ctypes.byref(n), ctypes.byref(ms)))
    return int(n.value), float(ms.value)


def profile_times(kind: int) -> list:
    """Device milliseconds of every recorded launch of a kernel kind, in launch order."""
    n = ctypes.c_int64(0)
    _check("pkv_profile_times", _lib.pkv_profile_times(kind, None, 0, ctypes.byref(n)))
    buf = (ctypes.c_float * max(int(n.value), 1))()
    _check("pkv_profile_times", _lib.pkv_profile_times(kind, buf, int(n.value), ctypes.byref(n)))
    return [float(buf[i]) for i in range(int(n.value))]


DRILL_WITHHOLD_FIRST_LOAD = 1
DRILL_LATE_CONSUMERS = 4
DRILL_LATE_PRODUCERS = 8


def set_wait_drill(wait_limit_ns: int = 0, flags: int = 0) -> None:
    """Diagnostic fail-closed drill for the launches that follow: the limit of
    each pipeline data wait (0 = the 2 s default) and, with
    DRILL_WITHHOLD_FIRST_LOAD, every pipeline's first load left unissued so
    that the wait for it runs out, or, with DRILL_LATE_CONSUMERS, the prefill's
    softmax warps late at each item's output, or, with DRILL_LATE_PRODUCERS, two of the
    latent attention's three loading warps late at everything they load.
    set_wait_drill() restores normal operation."""
    _check("pkv_set_wait_drill", _lib.pkv_set_wait_drill(int(wait_limit_ns), int(flags)))


def launch_count() -> int:
    """Kernels launched through the library by this process."""
    return int(_lib.pkv_launch_count())


@dataclass
class DecodeGroup:
    """One group of a fused decode: a paged_decode_attention call's own
    arguments (q [B, Hq, D], pools, tables, lengths, window, scale)."""
    q: torch.Tensor
    k_pool: torch.Tensor
    v_pool: torch.Tensor
    block_tables: torch.Tensor
    seq_lens: torch.Tensor
    window: int
    scale: float
    out: Optional[torch.Tensor] = None
    max_seq_len: Optional[int] = None
    k_scale: Optional[float] = None
    v_scale: Optional[float] = None
    sinks: int = 0


def _sinks_c(groups):
    return (ctypes.c_int32 * len(groups))(*[int(g.sinks) for g in groups])


def _group_c(g: DecodeGroup) -> _Group:
    pool = _pool(g.k_pool, g.v_pool, g.k_scale, g.v_scale)
    dev = g.k_pool.device
    _require(g.q.dim() == 3 and g.q.shape[2] == pool.head_dim and
             g.q.dtype == _act_dtype(g.k_pool.dtype) and g.q.is_contiguous() and g.q.device == dev,
             "q is [B, Hq, D], contiguous, pool dtype")
    B = g.q.shape[0]
    _i32_dev(g.block_tables, "block_tables", dev)
    _i32_dev(g.seq_lens, "seq_lens", dev)
    _require(g.block_tables.dim() == 2 and g.block_tables.shape[0] == B and g.seq_lens.shape == (B,),
             "block_tables [B, max_blocks], seq_lens [B]")
    if g.out is None:
        g.out = torch.empty_like(g.q)
    _require(g.out.shape == g.q.shape and g.out.dtype == g.q.dtype and g.out.is_contiguous(),
             "out matches q")
    _on_device(g.out, "out", dev)
    width = g.block_tables.shape[1]
    msl = g.max_seq_len if g.max_seq_len is not None else width * pool.block_size
    return _Group(g.q.data_ptr(), g.out.data_ptr(), pool, g.block_tables.data_ptr(), width,
                  g.seq_lens.data_ptr(), msl, int(g.window), float(g.scale))


def paged_decode_attention_groups(groups, workspace: Optional[torch.Tensor] = None,
                                  status: Optional[torch.Tensor] = None):
    """Several decode calls (groups of layers sharing the head shape: a full
    group and a sliding group, say) in one split launch and one merge launch.
    Returns the groups' outputs; each equals its own paged_decode_attention
    call bit for bit."""
    groups = list(groups)
    _require(1 <= len(groups) <= MAX_DECODE_GROUPS, f"1 .. {MAX_DECODE_GROUPS} groups")
    arr = (_Group * len(groups))(*[_group_c(g) for g in groups])
    B, hq = groups[0].q.shape[0], groups[0].q.shape[1]
    _require(all(g.q.shape[:2] == (B, hq) for g in groups), "every group has the same batch and q heads")
    dev = groups[0].k_pool.device
    _require(all(g.k_pool.device == dev for g in groups), "every group's pools on one GPU")
    _on_device(workspace, "workspace", dev)
    _status_ok(status, dev)
    with _on(dev):  # the plan reads the SM count of the current device
        sinks = _sinks_c(groups)
        if workspace is None:
            workspace = alloc_workspace(
                int(_lib.paged_decode_groups_sinks_workspace_size(arr, sinks, len(groups), B, hq)), dev)
        _check("paged_decode_attention_groups", _lib.paged_decode_attention_groups_sinks(
            arr, sinks, len(groups), B, hq, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _ptr(status), _stream(dev)))
    return [g.out for g in groups]


def decode_groups_workspace_size(groups) -> int:
    groups = list(groups)
    arr = (_Group * len(groups))(*[_group_c(g) for g in groups])
    return int(_lib.paged_decode_groups_sinks_workspace_size(arr, _sinks_c(groups), len(groups),
                                                             groups[0].q.shape[0], groups[0].q.shape[1]))


def paged_decode_attention_no_alloc(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                                    block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                    window: int, scale: float, out: torch.Tensor,
                                    max_seq_len: Optional[int] = None,
                                    prefix: Optional[PrefixDesc] = None,
                                    status: Optional[torch.Tensor] = None,
                                    k_scale: Optional[float] = None,
                                    v_scale: Optional[float] = None) -> torch.Tensor:
    """paged_decode_attention for callers that cannot allocate device memory.

    No workspace is passed and nothing is allocated: the library's fixed
    device scratch (``NO_ALLOC_SCRATCH_BYTES`` per GPU) is used, and ``out``
    must be given.  Calls on one device share that scratch, so calls that may
    overlap on the GPU must be ordered.  Sizes that need more scratch raise
    PkvError with PKV_ERR_WORKSPACE.
    """
    pool = _pool(k_pool, v_pool, k_scale, v_scale)
    dev = k_pool.device
    _require(q.dim() == 3 and q.shape[2] == pool.head_dim and q.dtype == _act_dtype(k_pool.dtype) and
             q.is_contiguous() and q.device == dev, "q is [B, Hq, D], contiguous, pool dtype")
    B, hq, _ = q.shape
    _i32_dev(block_tables, "block_tables", dev)
    _i32_dev(seq_lens, "seq_lens", dev)
    _require(block_tables.dim() == 2 and block_tables.shape[0] == B and seq_lens.shape == (B,),
             "block_tables [B, max_blocks], seq_lens [B]")
    _require(out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous(), "out matches q")
    _on_device(out, "out", dev)
    _status_ok(status, dev)
    _prefix_ok(prefix, dev)
    width = block_tables.shape[1]
    if max_seq_len is None:
        max_seq_len = width * pool.block_size
    px = ctypes.byref(prefix._c()) if prefix is not None else None
    # the pools' GPU is made current for the call: the library takes the
    # scratch of the current device and launches on this device's stream
    with _on(dev):
        code = _lib.paged_decode_attention_no_alloc(
            q.data_ptr(), hq, ctypes.byref(pool), block_tables.data_ptr(), width,
            seq_lens.data_ptr(), B, max_seq_len, window, float(scale), out.data_ptr(), px,
            _ptr(status), _stream(dev))
    if code == PKV_ERR_WORKSPACE:
        raise PkvError("paged_decode_attention_no_alloc (request exceeds the "
                       f"{NO_ALLOC_SCRATCH_BYTES >> 20} MiB static scratch)", code)
    _check("paged_decode_attention_no_alloc", code)
    return out


# ---------------------------------------------------------------------------
# host block allocator
# ---------------------------------------------------------------------------
class BlockAllocator:
    """The library's host block allocator (see ``include/pkv.h``): block ids of
    a pool of ``block_size``-token blocks, shared across requests by prefix
    hash, refcounted, with LRU eviction of cache-only blocks and
    grow-on-demand up to ``max_blocks``.  Token lists are int32 sequences."""

    def __init__(self, block_size: int, initial_blocks: int, max_blocks: int):
        self._a = _lib.pkv_allocator_create(block_size, initial_blocks, max_blocks)
        _require(bool(self._a), "block_size > 0 and 0 <= initial_blocks <= max_blocks")
        self.block_size = block_size

    def __del__(self):
        a = getattr(self, "_a", None)
        if a:
            _lib.pkv_allocator_destroy(a)
            self._a = None

    @staticmethod
    def _tokens(tokens):
        arr = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        return arr, (arr.ctypes.data if arr.size else None)

    @staticmethod
    def _keys(extra_keys):
        if extra_keys is None:
            return None, None
        arr = np.ascontiguousarray(np.asarray(extra_keys, dtype=np.uint64))
        return arr, arr.ctypes.data

    def begin(self) -> int:
        return int(_lib.pkv_allocator_begin(self._a))

    def find_cached_prefix(self, req: int, tokens, extra_keys=None) -> int:
        t, tp = self._tokens(tokens)
        k, kp = self._keys(extra_keys)
        n = ctypes.c_int32(0)
        _check("pkv_allocator_find_cached_prefix",
               _lib.pkv_allocator_find_cached_prefix(self._a, req, tp, t.size, kp, ctypes.byref(n)))
        return int(n.value)

    def reserve(self, req: int, n_tokens: int) -> None:
        _check("pkv_allocator_reserve", _lib.pkv_allocator_reserve(self._a, req, int(n_tokens)))

    def publish(self, req: int, tokens, extra_keys=None) -> None:
        t, tp = self._tokens(tokens)
        k, kp = self._keys(extra_keys)
        _check("pkv_allocator_publish", _lib.pkv_allocator_publish(self._a, req, tp, t.size, kp))

    def expire(self, req: int, first_live_token: int) -> None:
        """Drop the blocks wholly before ``first_live_token`` (a sliding
        window's start); their table entries become -1."""
        _check("pkv_allocator_expire", _lib.pkv_allocator_expire(self._a, req, int(first_live_token)))

    def expire_window(self, req: int, first_live_token: int, sinks: int) -> None:
        """``expire``, keeping the blocks that hold any of the first ``sinks`` tokens."""
        _check("pkv_allocator_expire_window", _lib.pkv_allocator_expire_window(
            self._a, req, int(first_live_token), int(sinks)))

    def fork(self, req: int, n_tokens: int):
        """A new request that shares ``req``'s first ``n_tokens`` tokens: its id and
        the page copy to make, ``(src, dst)``, or None when none is needed.  Inside
        a block that has expired it is refused (PKV_ERR_OUT_OF_BLOCKS)."""
        v = [ctypes.c_int32(-1) for _ in range(3)]
        _check("pkv_allocator_fork", _lib.pkv_allocator_fork(
            self._a, req, int(n_tokens), *[ctypes.byref(x) for x in v]))
        return int(v[0].value), (None if v[1].value < 0 else (int(v[1].value), int(v[2].value)))

    def truncate(self, req: int, n_tokens: int):
        """Roll ``req`` back to its first ``n_tokens`` tokens; the page copy to make,
        ``(src, dst)``, or None.  Into a block that has expired it is refused
        (PKV_ERR_OUT_OF_BLOCKS)."""
        v = [ctypes.c_int32(-1) for _ in range(2)]
        _check("pkv_allocator_truncate", _lib.pkv_allocator_truncate(
            self._a, req, int(n_tokens), *[ctypes.byref(x) for x in v]))
        return None if v[0].value < 0 else (int(v[0].value), int(v[1].value))

    def compact(self, num_blocks: int):
        """Shrink the pool to ``num_blocks`` blocks: the page copies to make, int32
        arrays ``(src, dst)``."""
        cap = self.stats()[0]
        src, dst = np.empty(max(cap, 1), np.int32), np.empty(max(cap, 1), np.int32)
        n = ctypes.c_int32(0)
        _check("pkv_allocator_compact", _lib.pkv_allocator_compact(
            self._a, int(num_blocks), src.ctypes.data, dst.ctypes.data, cap, ctypes.byref(n)))
        return src[:n.value].copy(), dst[:n.value].copy()

    def release(self, req: int) -> None:
        _check("pkv_allocator_release", _lib.pkv_allocator_release(self._a, req))

    def table(self, req: int) -> np.ndarray:
        n = ctypes.c_int32(0)
        _check("pkv_allocator_table", _lib.pkv_allocator_table(self._a, req, None, 0, ctypes.byref(n)))
        out = np.empty(n.value, dtype=np.int32)
        if n.value:
            _check("pkv_allocator_table", _lib.pkv_allocator_table(
                self._a, req, out.ctypes.data, n.value, ctypes.byref(n)))
        return out

    def refcount(self, block: int) -> int:
        return int(_lib.pkv_allocator_refcount(self._a, block))

    def stats(self):
        """(num_blocks, free_blocks, cached_blocks, grows)."""
        v = [ctypes.c_int32(0) for _ in range(4)]
        _check("pkv_allocator_stats", _lib.pkv_allocator_stats(self._a, *[ctypes.byref(x) for x in v]))
        return tuple(int(x.value) for x in v)
