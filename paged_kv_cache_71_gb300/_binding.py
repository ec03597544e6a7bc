"""ctypes binding of libpkv.so: argument marshalling only.

Every function here has the name of the C entry point it calls and does
nothing but turn tensors into pointers and sizes, pick the current CUDA
stream, call the library and raise on a non-OK status.  All computation
happens in the library's CUDA kernels.  There is no fallback: without a
built libpkv.so these functions raise.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libpkv.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "pkv.h")

PKV_F32, PKV_BF16, PKV_FP8_E4M3, PKV_INT8 = 0, 1, 2, 3
PKV_OK = 0
STATUS_NAMES = {0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_UNSUPPORTED", 3: "PKV_ERR_OUT_OF_RANGE",
                4: "PKV_ERR_WORKSPACE", 5: "PKV_ERR_CUDA"}
DEVERR_BAD_SLOT, DEVERR_BAD_BLOCK, DEVERR_BAD_LENGTH, DEVERR_TIMEOUT = 0x1, 0x2, 0x4, 0x8
DEVERR_Q_RANGE = 0x10

_DTYPE_CODE = {torch.float32: PKV_F32, torch.bfloat16: PKV_BF16, torch.uint8: PKV_FP8_E4M3,
               torch.float8_e4m3fn: PKV_FP8_E4M3, torch.int8: PKV_INT8}


class PkvError(RuntimeError):
    def __init__(self, status: int, func: str, detail: str):
        self.status = status
        super().__init__(f"{func}: {STATUS_NAMES.get(status, status)}: {detail}")


class CacheDesc(ctypes.Structure):
    """Mirror of pkv_cache_desc."""
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float), ("k_head_scales", ctypes.c_void_p), ("v_head_scales", ctypes.c_void_p)]

    @classmethod
    def for_cache(cls, k_cache: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0, k_head_scales=None,
                  v_head_scales=None) -> "CacheDesc":
        """Descriptor of a [NB][S][Hkv][D] cache; the optional per-head scales are fp32 device tensors [Hkv]
        (kept alive by the caller)."""
        NB, S, Hkv, D = k_cache.shape
        return cls(NB, S, Hkv, D, _DTYPE_CODE[k_cache.dtype], float(k_scale), float(v_scale),
                   _ptr(k_head_scales), _ptr(v_head_scales))


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libpkv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libpkv.so is not built ({LIB_PATH}); run __graft_entry__.build() or "
                           "python -m paged_kv_cache_71_gb300.build")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    D = ctypes.POINTER(CacheDesc)
    L.pkv_reshape_and_cache.argtypes = [P, P, i32, P, i32, P, P, D, P, P]
    L.pkv_paged_attention_workspace_size.argtypes = [D, i32, i32, i32, ctypes.POINTER(sz)]
    L.pkv_paged_attention_decode.argtypes = [P, P, i32, P, P, D, P, i32, P, i32, i32, f32, i32, i32, P, sz, P, P]
    L.pkv_paged_attention_decode_shared.argtypes = L.pkv_paged_attention_decode.argtypes
    L.pkv_copy_blocks.argtypes = [P, P, D, P, i32, P, P]
    L.pkv_paged_attention_decode_static_scratch.argtypes = [P, P, i32, P, P, D, P, i32, P, i32, i32, f32, i32, i32,
                                                            P, P]
    L.pkv_paged_prefill_chunk.argtypes = [P, P, i32, i32, i32, P, P, D, P, i32, i32, f32, P, P]
    L.pkv_paged_prefill_varlen.argtypes = [P, P, i32, i32, P, P, P, P, P, D, P, i32, i32, i32, f32, P, P]
    L.pkv_paged_attention_mixed.argtypes = [P, P, i32, i32, P, P, P, P, P, D, P, i32, i32, i32, i32, f32, P, sz,
                                            P, P]
    L.pkv_paged_attention_mixed_workspace_size.argtypes = [D, i32, i32, ctypes.POINTER(sz)]
    L.pkv_swap_blocks.argtypes = [P, P, i32, P, P, i32, D, P, i32, P, P]
    L.pkv_block_hashes.argtypes = [P, P, i32, i32, P, P, ctypes.c_int64, P, P]
    L.pkv_extend_sequences.argtypes = [P, i32, P, P, i32, i32, P, P, i32, P, P, P, i32, P, P, P, P]
    L.pkv_release_sequences.argtypes = [P, i32, P, P, P, i32, i32, P, P, i32, P, P, P, P]
    L.pkv_paged_attention_decode_prefix.argtypes = [P, P, i32, P, P, D, P, i32, P, i32, i32, f32, P, P, i32, P, sz,
                                                    P, P]
    L.pkv_paged_attention_decode_prefix_workspace_size.argtypes = [D, i32, i32, ctypes.POINTER(sz)]
    L.pkv_paged_cross_attention.argtypes = [P, P, i32, i32, P, P, P, P, D, P, i32, i32, i32, f32, P, sz, P, P]
    L.pkv_paged_cross_attention_workspace_size.argtypes = [D, i32, i32, i32, ctypes.POINTER(sz)]
    i64 = ctypes.c_int64
    L.pkv_rope_and_cache.argtypes = [P, P, P, P, i32, i64, i64, i64, i64, P, P, i32, i32, P, i32, i32, f32, P, P, D, P, P]
    L.pkv_paged_attention_tree.argtypes = [P, P, i32, i32, P, P, P, i32, P, P, D, P, i32, i32, i32, f32, P, sz, P, P]
    L.pkv_paged_attention_tree_workspace_size.argtypes = [D, i32, i32, i32, ctypes.POINTER(sz)]
    L.pkv_commit_tree.argtypes = [P, P, i32, D, P, i32, P, P, P, P, P, i32, i32, P, P, P, P, P, P, P]
    for name in ("pkv_reshape_and_cache", "pkv_paged_attention_workspace_size", "pkv_paged_attention_decode",
                 "pkv_copy_blocks", "pkv_paged_attention_decode_static_scratch", "pkv_paged_prefill_chunk",
                 "pkv_paged_prefill_varlen", "pkv_swap_blocks", "pkv_block_hashes", "pkv_extend_sequences",
                 "pkv_release_sequences", "pkv_paged_attention_decode_prefix",
                 "pkv_paged_attention_decode_prefix_workspace_size", "pkv_paged_cross_attention",
                 "pkv_paged_cross_attention_workspace_size", "pkv_rope_and_cache", "pkv_paged_attention_tree",
                 "pkv_paged_attention_tree_workspace_size", "pkv_commit_tree"):
        getattr(L, name).restype = ctypes.c_int
    L.pkv_status_string.argtypes = [ctypes.c_int]
    L.pkv_status_string.restype = ctypes.c_char_p
    L.pkv_last_error.argtypes = []
    L.pkv_last_error.restype = ctypes.c_char_p
    L.pkv_abi_version.argtypes = []
    L.pkv_abi_version.restype = ctypes.c_int32
    _lib = L
    return L


def declared_entry_points() -> list[str]:
    """Names of the functions declared in include/pkv.h."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:pkv_status|const char\*|int32_t)\s+(pkv_\w+)\s*\(", text, re.M)))


def _check(status: int, func: str) -> None:
    if status != PKV_OK:
        raise PkvError(status, func, (lib().pkv_last_error() or b"").decode())


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream, device: int | None = None) -> int | None:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device is None else device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype(t: torch.Tensor) -> int:
    return _DTYPE_CODE[t.dtype]


# ---------------------------------------------------------------- entry points

def pkv_reshape_and_cache(k_new, v_new, slot_mapping, k_cache, v_cache, cache: CacheDesc, device_error=None,
                          stream=None) -> None:
    _check(lib().pkv_reshape_and_cache(_ptr(k_new), _ptr(v_new), _dtype(k_new), _ptr(slot_mapping),
                                       int(slot_mapping.shape[0]), _ptr(k_cache), _ptr(v_cache),
                                       ctypes.byref(cache), _ptr(device_error), _stream(stream)),
           "pkv_reshape_and_cache")


def pkv_paged_attention_workspace_size(cache: CacheDesc, num_seqs: int, num_q_heads: int, num_splits: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().pkv_paged_attention_workspace_size(ctypes.byref(cache), int(num_seqs), int(num_q_heads),
                                                    int(num_splits), ctypes.byref(out)),
           "pkv_paged_attention_workspace_size")
    return int(out.value)


def pkv_paged_attention_decode(out, q, k_cache, v_cache, cache: CacheDesc, block_tables, context_lens,
                               scale: float, num_splits: int = 0, max_context_len: int = 0, workspace=None,
                               device_error=None, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().pkv_paged_attention_decode(_ptr(out), _ptr(q), _dtype(q), _ptr(k_cache), _ptr(v_cache),
                                            ctypes.byref(cache), _ptr(block_tables), int(block_tables.shape[1]),
                                            _ptr(context_lens), int(q.shape[0]), int(q.shape[1]), float(scale),
                                            int(num_splits), int(max_context_len), _ptr(workspace), ws_bytes,
                                            _ptr(device_error), _stream(stream)),
           "pkv_paged_attention_decode")


def pkv_paged_attention_decode_shared(out, q, k_cache, v_cache, cache: CacheDesc, block_tables, context_lens,
                                      scale: float, num_splits: int = 0, max_context_len: int = 0, workspace=None,
                                      device_error=None, stream=None) -> None:
    """pkv_paged_attention_decode for a batch whose tables share physical blocks (same arguments)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().pkv_paged_attention_decode_shared(_ptr(out), _ptr(q), _dtype(q), _ptr(k_cache), _ptr(v_cache),
                                                   ctypes.byref(cache), _ptr(block_tables),
                                                   int(block_tables.shape[1]), _ptr(context_lens), int(q.shape[0]),
                                                   int(q.shape[1]), float(scale), int(num_splits),
                                                   int(max_context_len), _ptr(workspace), ws_bytes,
                                                   _ptr(device_error), _stream(stream)),
           "pkv_paged_attention_decode_shared")


def pkv_paged_attention_decode_static_scratch(out, q, k_cache, v_cache, cache: CacheDesc, block_tables,
                                              context_lens, scale: float, num_splits: int = 0,
                                              max_context_len: int = 0, device_error=None, stream=None) -> None:
    """pkv_paged_attention_decode without a workspace argument: the library's static scratch is used."""
    _check(lib().pkv_paged_attention_decode_static_scratch(
        _ptr(out), _ptr(q), _dtype(q), _ptr(k_cache), _ptr(v_cache), ctypes.byref(cache), _ptr(block_tables),
        int(block_tables.shape[1]), _ptr(context_lens), int(q.shape[0]), int(q.shape[1]), float(scale),
        int(num_splits), int(max_context_len), _ptr(device_error), _stream(stream)),
        "pkv_paged_attention_decode_static_scratch")


def pkv_paged_prefill_chunk(out, q, q_start: int, k_cache, v_cache, cache: CacheDesc, block_table, kv_len: int,
                            scale: float, device_error=None, stream=None) -> None:
    _check(lib().pkv_paged_prefill_chunk(_ptr(out), _ptr(q), _dtype(q), int(q.shape[0]), int(q_start),
                                         _ptr(k_cache), _ptr(v_cache), ctypes.byref(cache), _ptr(block_table),
                                         int(kv_len), int(q.shape[1]), float(scale), _ptr(device_error),
                                         _stream(stream)),
           "pkv_paged_prefill_chunk")


def pkv_paged_attention_mixed_workspace_size(cache: CacheDesc, num_decode: int, num_q_heads: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().pkv_paged_attention_mixed_workspace_size(ctypes.byref(cache), int(num_decode), int(num_q_heads),
                                                          ctypes.byref(out)),
           "pkv_paged_attention_mixed_workspace_size")
    return int(out.value)


def pkv_paged_attention_mixed(out, q, cu_q, q_starts, kv_lens, k_cache, v_cache, cache: CacheDesc, block_tables,
                              num_decode: int, scale: float, workspace=None, device_error=None, stream=None) -> None:
    """A mixed step in one launch: chunks [0, num_decode) are decode tokens, the rest prefill chunks (varlen arrays
    on the device, q/out [total_q_tokens][Hq][128])."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().pkv_paged_attention_mixed(_ptr(out), _ptr(q), _dtype(q), int(q.shape[0]), _ptr(cu_q),
                                           _ptr(q_starts), _ptr(kv_lens), _ptr(k_cache), _ptr(v_cache),
                                           ctypes.byref(cache), _ptr(block_tables), int(block_tables.shape[1]),
                                           int(kv_lens.shape[0]), int(num_decode), int(q.shape[1]), float(scale),
                                           _ptr(workspace), ws_bytes, _ptr(device_error), _stream(stream)),
           "pkv_paged_attention_mixed")


def pkv_paged_prefill_varlen(out, q, cu_q, q_starts, kv_lens, k_cache, v_cache, cache: CacheDesc, block_tables,
                             scale: float, device_error=None, stream=None) -> None:
    """Several prefill chunks in one launch; q/out are [total_q_tokens][Hq][128], the index arrays on the device."""
    _check(lib().pkv_paged_prefill_varlen(_ptr(out), _ptr(q), _dtype(q), int(q.shape[0]), _ptr(cu_q),
                                          _ptr(q_starts), _ptr(kv_lens), _ptr(k_cache), _ptr(v_cache),
                                          ctypes.byref(cache), _ptr(block_tables), int(block_tables.shape[1]),
                                          int(kv_lens.shape[0]), int(q.shape[1]), float(scale),
                                          _ptr(device_error), _stream(stream)),
           "pkv_paged_prefill_varlen")


STATIC_SCRATCH_BYTES = 12 * 1024 * 1024  # PKV_STATIC_SCRATCH_BYTES in include/pkv.h


def pkv_copy_blocks(k_cache, v_cache, cache: CacheDesc, block_mapping, device_error=None, stream=None) -> None:
    _check(lib().pkv_copy_blocks(_ptr(k_cache), _ptr(v_cache), ctypes.byref(cache), _ptr(block_mapping),
                                 int(block_mapping.shape[0]), _ptr(device_error), _stream(stream)),
           "pkv_copy_blocks")


def pkv_swap_blocks(src_k, src_v, dst_k, dst_v, cache: CacheDesc, block_mapping, device_error=None,
                    stream=None) -> None:
    """Whole-block copies between two pools (device or pinned host memory)."""
    _check(lib().pkv_swap_blocks(_ptr(src_k), _ptr(src_v), int(src_k.shape[0]), _ptr(dst_k), _ptr(dst_v),
                                 int(dst_k.shape[0]), ctypes.byref(cache), _ptr(block_mapping),
                                 int(block_mapping.shape[0]), _ptr(device_error), _stream(stream)),
           "pkv_swap_blocks")


def pkv_block_hashes(token_ids, cu_tokens, block_size: int, out_offsets, hashes, device_error=None,
                     stream=None) -> None:
    """Chained FNV-1a-64 content hashes of every full block (hashes: int64/uint64 device tensor)."""
    _check(lib().pkv_block_hashes(_ptr(token_ids), _ptr(cu_tokens), int(cu_tokens.shape[0]) - 1, int(block_size),
                                  _ptr(out_offsets), _ptr(hashes), int(hashes.numel()), _ptr(device_error),
                                  _stream(stream)),
           "pkv_block_hashes")


def _device() -> int:
    """The current CUDA device; a number that no tensor's device has, where CUDA has not been used."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -2


def _here(t) -> int:
    """The current CUDA device, which t must be on (-2: it is on none, and CUDA may not have been used)."""
    return torch._C._cuda_getDevice() if t.get_device() >= 0 else -2


def _extra(t, device: int) -> bool:
    """A workspace or error word: a tensor must be on the device; None and raw pointers pass."""
    return t is None or isinstance(t, int) or t.get_device() == device


def _word(t, device: int) -> bool:
    """An error word: None, a raw pointer, or a tensor on the device whose elements have room for it."""
    return t is None or isinstance(t, int) or (t.element_size() >= 4 and t.get_device() == device)


def _room(t, device: int) -> bool:
    """A workspace: None, or a contiguous tensor on the device (a raw pointer has no size)."""
    return t is None or (not isinstance(t, int) and t.get_device() == device and t.is_contiguous())


def _dims(func: str, **tensors) -> None:
    """name=(tensor, its number of dimensions), for the shapes that sizes are taken from."""
    for name, (t, n) in tensors.items():
        if t.dim() != n:
            raise PkvError(1, func, f"{name} has shape {tuple(t.shape)}, expected {n} dimension{'s' if n > 1 else ''}")


def _fits(t, dtype, shape, device: int) -> bool:
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device


def _refuse(func: str, device: int, device_error=None, workspace=None, **tensors) -> None:
    """Say what is wrong with tensors that the pointers alone would not tell from good ones: name=(tensor or None, dtypes,
    shape).  Layouts must be contiguous, and every tensor on the current CUDA device."""
    tensors = {name: x for name, x in tensors.items() if x[0] is not None}
    for name, (t, dtypes, shape) in tensors.items():
        if t.dtype not in dtypes:
            raise PkvError(1, func, f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
        if t.shape != shape:
            raise PkvError(1, func, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise PkvError(1, func, f"{name} must be contiguous")
    for name, (t, _, _) in tensors.items():
        if t.get_device() != device:
            raise PkvError(1, func, f"{name} is on {t.device}, not on the current CUDA device")
    if isinstance(workspace, int):
        raise PkvError(4, func, "workspace must be a tensor: a raw pointer has no size")
    for name, t in (("device_error", device_error), ("workspace", workspace)):
        if not _extra(t, device):
            raise PkvError(1, func, f"{name} is on {t.device}, not on the current CUDA device")
    if not _word(device_error, device):
        raise PkvError(1, func, f"device_error has dtype {device_error.dtype}, expected torch.int32")
    if not _room(workspace, device):
        raise PkvError(4, func, "workspace must be contiguous")


_I32, _I64, _FLAG = (torch.int32,), (torch.int64,), (torch.bool, torch.uint8)
_FLOATS = (torch.float32, torch.bfloat16)
_MASK = (torch.int64, torch.uint64)


def _cache_dtypes(cache: CacheDesc) -> tuple:
    """The tensor types that a cache of the descriptor's type may have."""
    return tuple(t for t, code in _DTYPE_CODE.items() if code == cache.dtype)


def pkv_extend_sequences(block_tables, past_lens, new_lens, block_size: int, free_blocks, free_count, seq_lens,
                         new_free_count, slot_mapping, cu_q=None, q_starts=None, device_error=None,
                         stream=None) -> None:
    """Block tables, lengths and slot map of a step from the request lengths, on the GPU.  seq_lens may be past_lens and
    new_free_count may be free_count (in place); free_blocks has one entry per block of the pool."""
    L, shape, rows, i32, dev = lib(), past_lens.shape, block_tables.shape, torch.int32, _here(past_lens)
    if len(shape) != 1 or len(rows) != 2:
        _dims("pkv_extend_sequences", past_lens=(past_lens, 1), block_tables=(block_tables, 2))
    (n,), width, nb, cap = shape, rows[-1], free_blocks.numel(), slot_mapping.numel()
    if not (block_tables.dtype is past_lens.dtype is new_lens.dtype is free_blocks.dtype is free_count.dtype
            is seq_lens.dtype is new_free_count.dtype is i32 and slot_mapping.dtype is torch.int64
            and rows == (n, width) and new_lens.shape == shape == seq_lens.shape
            and free_count.numel() == new_free_count.numel() == free_blocks.dim() == slot_mapping.dim() == 1
            and block_tables.is_contiguous() and past_lens.is_contiguous() and new_lens.is_contiguous()
            and free_blocks.is_contiguous() and seq_lens.is_contiguous() and slot_mapping.is_contiguous()
            and block_tables.get_device() == past_lens.get_device() == new_lens.get_device() == free_blocks.get_device()
            == free_count.get_device() == seq_lens.get_device() == new_free_count.get_device()
            == slot_mapping.get_device() == dev and _word(device_error, dev)
            and (cu_q is None or _fits(cu_q, i32, (n + 1,), dev)) and (q_starts is None or _fits(q_starts, i32, shape, dev))):
        _refuse("pkv_extend_sequences", _device(), device_error, block_tables=(block_tables, _I32, (n, width)), past_lens=(past_lens, _I32, (n,)),
                new_lens=(new_lens, _I32, (n,)), free_blocks=(free_blocks, _I32, (nb,)), free_count=(free_count, _I32, (1,)),
                seq_lens=(seq_lens, _I32, (n,)), new_free_count=(new_free_count, _I32, (1,)),
                slot_mapping=(slot_mapping, _I64, (cap,)), cu_q=(cu_q, _I32, (n + 1,)), q_starts=(q_starts, _I32, (n,)))
    status = L.pkv_extend_sequences(block_tables.data_ptr(), width, past_lens.data_ptr(), new_lens.data_ptr(), n,
                                    int(block_size), free_blocks.data_ptr(), free_count.data_ptr(), nb, seq_lens.data_ptr(),
                                    new_free_count.data_ptr(), slot_mapping.data_ptr(), cap, _ptr(cu_q), _ptr(q_starts),
                                    _ptr(device_error), _stream(stream, dev))
    if status:
        _check(status, "pkv_extend_sequences")


def pkv_release_sequences(block_tables, past_lens, finished, block_size: int, free_blocks, free_count, seq_lens,
                          new_free_count, keep_blocks=None, device_error=None, stream=None) -> None:
    """Finished sequences hand their blocks back to the free stack, on the GPU (finished: bool or uint8 [num_seqs])."""
    L, shape, rows, i32, dev = lib(), past_lens.shape, block_tables.shape, torch.int32, _here(past_lens)
    if len(shape) != 1 or len(rows) != 2:
        _dims("pkv_release_sequences", past_lens=(past_lens, 1), block_tables=(block_tables, 2))
    (n,), width, nb = shape, rows[-1], free_blocks.numel()
    if not (block_tables.dtype is past_lens.dtype is free_blocks.dtype is free_count.dtype is seq_lens.dtype
            is new_free_count.dtype is i32 and finished.dtype in _FLAG
            and rows == (n, width) and finished.shape == shape == seq_lens.shape
            and free_count.numel() == new_free_count.numel() == free_blocks.dim() == 1
            and block_tables.is_contiguous() and past_lens.is_contiguous() and finished.is_contiguous()
            and free_blocks.is_contiguous() and seq_lens.is_contiguous()
            and block_tables.get_device() == past_lens.get_device() == finished.get_device() == free_blocks.get_device()
            == free_count.get_device() == seq_lens.get_device() == new_free_count.get_device() == dev
            and _word(device_error, dev) and (keep_blocks is None or _fits(keep_blocks, i32, shape, dev))):
        _refuse("pkv_release_sequences", _device(), device_error, block_tables=(block_tables, _I32, (n, width)),
                past_lens=(past_lens, _I32, (n,)), finished=(finished, _FLAG, (n,)), free_blocks=(free_blocks, _I32, (nb,)),
                free_count=(free_count, _I32, (1,)), seq_lens=(seq_lens, _I32, (n,)),
                new_free_count=(new_free_count, _I32, (1,)), keep_blocks=(keep_blocks, _I32, (n,)))
    status = L.pkv_release_sequences(block_tables.data_ptr(), width, past_lens.data_ptr(), finished.data_ptr(),
                                     _ptr(keep_blocks), n, int(block_size), free_blocks.data_ptr(), free_count.data_ptr(), nb,
                                     seq_lens.data_ptr(), new_free_count.data_ptr(), _ptr(device_error),
                                     _stream(stream, dev))
    if status:
        _check(status, "pkv_release_sequences")


def pkv_paged_attention_decode_prefix_workspace_size(cache: CacheDesc, num_seqs: int, num_q_heads: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().pkv_paged_attention_decode_prefix_workspace_size(ctypes.byref(cache), int(num_seqs),
                                                                  int(num_q_heads), ctypes.byref(out)),
           "pkv_paged_attention_decode_prefix_workspace_size")
    return int(out.value)


def pkv_paged_attention_decode_prefix(out, q, k_cache, v_cache, cache: CacheDesc, block_tables, context_lens,
                                      cu_groups, prefix_lens, scale: float, workspace=None, device_error=None,
                                      stream=None) -> None:
    """Decode attention for groups of sequences (cu_groups) that share their first prefix_lens tokens' blocks: a group's
    prefix is computed once for all of its sequences."""
    L, dev = lib(), _here(q)
    if q.dim() != 3 or block_tables.dim() != 2:
        _dims("pkv_paged_attention_decode_prefix", q=(q, 3), block_tables=(block_tables, 2))
    n, heads, D = q.shape
    caches, groups, width = (cache.num_blocks, cache.block_size, cache.num_kv_heads, D), prefix_lens.numel(), block_tables.shape[-1]
    if not (D == cache.head_dim and q.dtype in _FLOATS and _DTYPE_CODE.get(k_cache.dtype) == cache.dtype and _room(workspace, dev)
            and _word(device_error, dev)
            and _fits(q, out.dtype, out.shape, dev) and out.is_contiguous() and out.get_device() == dev
            and _fits(k_cache, v_cache.dtype, caches, dev) and _fits(v_cache, k_cache.dtype, caches, dev)
            and _fits(block_tables, torch.int32, (n, width), dev) and _fits(context_lens, torch.int32, (n,), dev)
            and _fits(cu_groups, torch.int32, (groups + 1,), dev) and _fits(prefix_lens, torch.int32, (groups,), dev)):
        caches = (*caches[:3], cache.head_dim)
        _refuse("pkv_paged_attention_decode_prefix", _device(), device_error, workspace, q=(q, _FLOATS, (n, heads, cache.head_dim)),
                out=(out, (q.dtype,), (n, heads, D)), k_cache=(k_cache, _cache_dtypes(cache), caches),
                v_cache=(v_cache, (k_cache.dtype,), caches), block_tables=(block_tables, _I32, (n, width)),
                context_lens=(context_lens, _I32, (n,)), cu_groups=(cu_groups, _I32, (groups + 1,)),
                prefix_lens=(prefix_lens, _I32, (groups,)))
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    status = L.pkv_paged_attention_decode_prefix(out.data_ptr(), q.data_ptr(), _DTYPE_CODE[q.dtype], k_cache.data_ptr(),
                                                 v_cache.data_ptr(), ctypes.byref(cache), block_tables.data_ptr(), width,
                                                 context_lens.data_ptr(), n, heads, float(scale), cu_groups.data_ptr(),
                                                 prefix_lens.data_ptr(), groups, ws, ws_bytes, _ptr(device_error),
                                                 _stream(stream, dev))
    if status:
        _check(status, "pkv_paged_attention_decode_prefix")


def pkv_paged_cross_attention_workspace_size(cache: CacheDesc, total_q_tokens: int, num_seqs: int,
                                             num_q_heads: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().pkv_paged_cross_attention_workspace_size(ctypes.byref(cache), int(total_q_tokens), int(num_seqs),
                                                          int(num_q_heads), ctypes.byref(out)),
           "pkv_paged_cross_attention_workspace_size")
    return int(out.value)


def pkv_paged_cross_attention(out, q, cu_q, kv_lens, k_cache, v_cache, cache: CacheDesc, block_tables, scale: float,
                              workspace=None, device_error=None, stream=None) -> None:
    """Decoder queries against paged encoder states, without a mask: sequence s owns query tokens
    [cu_q[s], cu_q[s + 1]) of q (cu_q None: one token a sequence) and kv_lens[s] states."""
    L, n, dev = lib(), kv_lens.numel(), _here(q)
    if q.dim() != 3 or block_tables.dim() != 2:
        _dims("pkv_paged_cross_attention", q=(q, 3), block_tables=(block_tables, 2))
    tokens, heads, D = q.shape
    caches, width = (cache.num_blocks, cache.block_size, cache.num_kv_heads, D), block_tables.shape[-1]
    if not (D == cache.head_dim and q.dtype in _FLOATS and _DTYPE_CODE.get(k_cache.dtype) == cache.dtype and _room(workspace, dev)
            and _word(device_error, dev)
            and _fits(q, out.dtype, out.shape, dev) and out.is_contiguous() and out.get_device() == dev
            and _fits(k_cache, v_cache.dtype, caches, dev) and _fits(v_cache, k_cache.dtype, caches, dev)
            and _fits(block_tables, torch.int32, (n, width), dev) and _fits(kv_lens, torch.int32, (n,), dev)
            and (cu_q is None or _fits(cu_q, torch.int32, (n + 1,), dev))):
        caches = (*caches[:3], cache.head_dim)
        _refuse("pkv_paged_cross_attention", _device(), device_error, workspace, q=(q, _FLOATS, (tokens, heads, cache.head_dim)),
                out=(out, (q.dtype,), (tokens, heads, D)), kv_lens=(kv_lens, _I32, (n,)), k_cache=(k_cache, _cache_dtypes(cache), caches),
                v_cache=(v_cache, (k_cache.dtype,), caches), block_tables=(block_tables, _I32, (n, width)),
                cu_q=(cu_q, _I32, (n + 1,)))
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    status = L.pkv_paged_cross_attention(out.data_ptr(), q.data_ptr(), _DTYPE_CODE[q.dtype], tokens, _ptr(cu_q),
                                         kv_lens.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ctypes.byref(cache),
                                         block_tables.data_ptr(), width, n, heads, float(scale), ws, ws_bytes,
                                         _ptr(device_error), _stream(stream, dev))
    if status:
        _check(status, "pkv_paged_cross_attention")


def _refuse_rows(func: str, name: str, t, dtypes, shape) -> None:
    if t.dtype not in dtypes:
        raise PkvError(1, func, f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.shape != shape:
        raise PkvError(1, func, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.numel() and not _apart(t.stride(), shape):
        raise PkvError(1, func, f"{name} must have contiguous, separate tokens (strides {t.stride()})")


def _apart(strides, shape) -> bool:
    """[tokens][heads][D] whose tokens may be further apart than a token is long (parts of a fused projection's rows)."""
    tokens, heads, D = shape
    return strides[2] == 1 and (strides[1] == D or heads == 1) and (tokens < 2 or strides[0] >= heads * D)


def pkv_rope_and_cache(q_out, q, k_new, v_new, positions, slot_mapping, inv_freq, k_cache, v_cache, cache: CacheDesc,
                       interleaved: bool = False, rope_scale: float = 1.0, device_error=None, stream=None) -> None:
    """Rotary positions on the queries (q_out may be q) and keys, keys and values written to their slots, in one pass.
    inv_freq: fp32, one per pair of rotated elements (rotary_frequencies makes it).  q and q_out None: keys and values only;
    k_new and v_new None: queries only."""
    func, L, dev, D = "pkv_rope_and_cache", lib(), _here(positions), cache.head_dim
    some = q if q is not None else k_new
    if some is None or (q is None) != (q_out is None) or (k_new is None) != (v_new is None):
        raise PkvError(1, func, "q comes with q_out, k_new with v_new, and one of the pairs is needed")
    if positions.dim() != 1 or inv_freq.dim() != 1 or some.dim() != 3:
        _dims(func, positions=(positions, 1), inv_freq=(inv_freq, 1), **{"k_new" if q is None else "q": (some, 3)})
    src, i32, f32 = some.dtype, torch.int32, torch.float32
    n, hkv, pairs = positions.shape[0], cache.num_kv_heads, inv_freq.shape[0]
    heads = 0 if q is None else q.shape[1]
    good = (src in _FLOATS and positions.dtype is i32 and inv_freq.dtype is f32 and positions.is_contiguous()
            and inv_freq.is_contiguous() and inv_freq.get_device() == dev and _word(device_error, dev)
            and (slot_mapping is None or _fits(slot_mapping, torch.int64, (n,), dev)))
    q_stride = q_out_stride = k_stride = v_stride = 0
    kc = vc = None
    if good and q is not None:
        shape, s0, s1 = (n, heads, D), q.stride(), q_out.stride()
        good = (q_out.dtype is src and q.shape == shape == q_out.shape and _apart(s0, shape) and (s1 == s0 or _apart(s1, shape))
                and q.get_device() == dev == q_out.get_device())
        q_stride, q_out_stride = (s0[0], s1[0]) if n > 1 else (heads * D, heads * D)  # (a single token's stride may be anything)
    if good and k_new is not None:
        shape, s0, s1, caches = (n, hkv, D), k_new.stride(), v_new.stride(), (cache.num_blocks, cache.block_size, hkv, D)
        kind = k_cache.dtype
        good = (slot_mapping is not None and k_new.dtype is src is v_new.dtype and k_new.shape == shape == v_new.shape
                and _apart(s0, shape) and (s1 == s0 or _apart(s1, shape)) and _DTYPE_CODE.get(kind) == cache.dtype
                and v_cache.dtype is kind and k_cache.shape == caches == v_cache.shape and k_cache.is_contiguous()
                and v_cache.is_contiguous()
                and k_new.get_device() == dev == v_new.get_device() == k_cache.get_device() == v_cache.get_device())
        k_stride, v_stride = (s0[0], s1[0]) if n > 1 else (hkv * D, hkv * D)
        kc, vc = k_cache.data_ptr(), v_cache.data_ptr()
    if not good:
        if k_new is not None and slot_mapping is None:
            raise PkvError(1, func, "k_new and v_new need slot_mapping")
        for name, t, h in (("q", q, heads), ("q_out", q_out, heads), ("k_new", k_new, hkv), ("v_new", v_new, hkv)):
            if t is not None:
                _refuse_rows(func, name, t, _FLOATS if t is some else (src,), (n, h, D))
        caches = (cache.num_blocks, cache.block_size, hkv, D)
        pools = {} if k_new is None else dict(k_cache=(k_cache, _cache_dtypes(cache), caches), v_cache=(v_cache, (k_cache.dtype,), caches))
        _refuse(func, _device(), device_error, positions=(positions, _I32, (n,)), slot_mapping=(slot_mapping, _I64, (n,)),
                inv_freq=(inv_freq, (f32,), (pairs,)), **pools)
        for name, t in (("q", q), ("q_out", q_out), ("k_new", k_new), ("v_new", v_new)):
            if t is not None and t.get_device() != _device():
                raise PkvError(1, func, f"{name} is on {t.device}, not on the current CUDA device")
    if n == 0:
        return
    status = L.pkv_rope_and_cache(_ptr(q_out), _ptr(q), _ptr(k_new), _ptr(v_new), _DTYPE_CODE[src], q_out_stride, q_stride, k_stride,
                                  v_stride, positions.data_ptr(), _ptr(slot_mapping), n, heads, inv_freq.data_ptr(), 2 * pairs,
                                  1 if interleaved else 0, float(rope_scale), kc, vc, ctypes.byref(cache), _ptr(device_error),
                                  _stream(stream, dev))
    if status:
        _check(status, func)


def pkv_paged_attention_tree_workspace_size(cache: CacheDesc, total_q_tokens: int, num_seqs: int, num_q_heads: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().pkv_paged_attention_tree_workspace_size(ctypes.byref(cache), int(total_q_tokens), int(num_seqs),
                                                         int(num_q_heads), ctypes.byref(out)),
           "pkv_paged_attention_tree_workspace_size")
    return int(out.value)


def pkv_paged_attention_tree(out, q, cu_q, kv_lens, tree_mask, k_cache, v_cache, cache: CacheDesc, block_tables,
                             scale: float, workspace=None, device_error=None, stream=None) -> None:
    """Attention of runs of drafted tokens, the last of their sequence's keys: each sees all keys before the run and those of
    the run that its row of tree_mask (int64 or uint64 [total_q_tokens][words], bit j: token j of the run) names; tree_mask
    None: runs are chains.  draft_tree_masks makes the masks of trees of a fixed shape."""
    func, L, n, dev = "pkv_paged_attention_tree", lib(), kv_lens.numel(), _here(q)
    if q.dim() != 3 or block_tables.dim() != 2 or (tree_mask is not None and tree_mask.dim() != 2):
        _dims(func, q=(q, 3), block_tables=(block_tables, 2), **({} if tree_mask is None else dict(tree_mask=(tree_mask, 2))))
    tokens, heads, D = q.shape
    caches, width = (cache.num_blocks, cache.block_size, cache.num_kv_heads, D), block_tables.shape[-1]
    words = 0 if tree_mask is None else tree_mask.shape[1]
    if tree_mask is not None and words == 0:
        raise PkvError(1, func, "tree_mask has no words (a chain has no mask: None)")
    if not (D == cache.head_dim and q.dtype in _FLOATS and _DTYPE_CODE.get(k_cache.dtype) == cache.dtype and _room(workspace, dev)
            and _word(device_error, dev)
            and _fits(q, out.dtype, out.shape, dev) and out.is_contiguous() and out.get_device() == dev
            and _fits(k_cache, v_cache.dtype, caches, dev) and _fits(v_cache, k_cache.dtype, caches, dev)
            and _fits(block_tables, torch.int32, (n, width), dev) and _fits(kv_lens, torch.int32, (n,), dev)
            and _fits(cu_q, torch.int32, (n + 1,), dev)
            and (tree_mask is None or (tree_mask.dtype in _MASK and _fits(tree_mask, tree_mask.dtype, (tokens, words), dev)))):
        caches = (*caches[:3], cache.head_dim)
        _refuse(func, _device(), device_error, workspace, q=(q, _FLOATS, (tokens, heads, cache.head_dim)),
                out=(out, (q.dtype,), (tokens, heads, D)), kv_lens=(kv_lens, _I32, (n,)), k_cache=(k_cache, _cache_dtypes(cache), caches),
                v_cache=(v_cache, (k_cache.dtype,), caches), block_tables=(block_tables, _I32, (n, width)),
                cu_q=(cu_q, _I32, (n + 1,)), tree_mask=(tree_mask, _MASK, (tokens, words)))
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    status = L.pkv_paged_attention_tree(out.data_ptr(), q.data_ptr(), _DTYPE_CODE[q.dtype], tokens, cu_q.data_ptr(),
                                        kv_lens.data_ptr(), _ptr(tree_mask), words if tokens else 0, k_cache.data_ptr(), v_cache.data_ptr(),
                                        ctypes.byref(cache), block_tables.data_ptr(), width, n, heads, float(scale), ws, ws_bytes,
                                        _ptr(device_error), _stream(stream, dev))
    if status:
        _check(status, func)


class LayerCaches:
    """The K and V pools of all layers of a model, checked once: alike in shape and type, contiguous, on one device."""

    def __init__(self, k_caches, v_caches):
        k_caches, v_caches = list(k_caches), list(v_caches)
        if not k_caches or len(k_caches) != len(v_caches):
            raise PkvError(1, "LayerCaches", f"{len(k_caches)} K and {len(v_caches)} V pools, expected as many, one or more")
        first = k_caches[0]
        _dims("LayerCaches", k_cache=(first, 4))
        if first.dtype not in _DTYPE_CODE:
            raise PkvError(1, "LayerCaches", f"pools have dtype {first.dtype}, expected a cache type")
        for t in k_caches + v_caches:
            if t.dtype is not first.dtype or t.shape != first.shape or t.device != first.device or not t.is_contiguous():
                raise PkvError(1, "LayerCaches", "the layers' pools must be contiguous, of one shape, type and device")
        if len({t.data_ptr() for t in k_caches + v_caches}) < 2 * len(k_caches):
            raise PkvError(1, "LayerCaches", "two of the layers' pools are the same memory")
        self.tensors = k_caches, v_caches  # kept alive
        self.device = first.get_device()
        self.num_layers = len(k_caches)
        self.desc = CacheDesc.for_cache(first)
        array = ctypes.c_void_p * self.num_layers
        self.k_pointers, self.v_pointers = array(*(t.data_ptr() for t in k_caches)), array(*(t.data_ptr() for t in v_caches))


def pkv_commit_tree(layers: LayerCaches, block_tables, cu_q, past_lens, parents, draft_tokens, target_tokens, accepted,
                    num_accepted, seq_lens, next_tokens, keep_blocks=None, device_error=None, stream=None) -> None:
    """The accepted path of each sequence's draft tree (accepted, num_accepted, seq_lens, next_tokens, keep_blocks are written),
    its K/V moved to consecutive slots in all layers."""
    func, L, dev, i32 = "pkv_commit_tree", lib(), _here(past_lens), torch.int32
    if past_lens.dim() != 1 or block_tables.dim() != 2 or parents.dim() != 1:
        _dims(func, past_lens=(past_lens, 1), block_tables=(block_tables, 2), parents=(parents, 1))
    shape, runs, width = past_lens.shape, parents.shape, block_tables.shape[1]
    n, tokens = shape[0], runs[0]
    if not (block_tables.dtype is cu_q.dtype is past_lens.dtype is parents.dtype is draft_tokens.dtype is target_tokens.dtype
            is accepted.dtype is num_accepted.dtype is seq_lens.dtype is next_tokens.dtype is i32
            and block_tables.shape[0] == n and cu_q.dim() == 1 and cu_q.shape[0] == n + 1
            and draft_tokens.shape == runs == target_tokens.shape and accepted.shape == runs
            and num_accepted.shape == shape == seq_lens.shape and next_tokens.shape == shape
            and block_tables.is_contiguous() and cu_q.is_contiguous() and past_lens.is_contiguous() and parents.is_contiguous()
            and draft_tokens.is_contiguous() and target_tokens.is_contiguous() and accepted.is_contiguous()
            and num_accepted.is_contiguous() and seq_lens.is_contiguous() and next_tokens.is_contiguous()
            and layers.device == block_tables.get_device() == cu_q.get_device() == past_lens.get_device() == parents.get_device()
            == draft_tokens.get_device() == target_tokens.get_device() == accepted.get_device() == num_accepted.get_device()
            == seq_lens.get_device() == next_tokens.get_device() == dev and _word(device_error, dev)
            and (keep_blocks is None or _fits(keep_blocks, i32, shape, dev))):
        _refuse(func, _device(), device_error, past_lens=(past_lens, _I32, (n,)), block_tables=(block_tables, _I32, (n, width)),
                cu_q=(cu_q, _I32, (n + 1,)), parents=(parents, _I32, (tokens,)), draft_tokens=(draft_tokens, _I32, (tokens,)),
                target_tokens=(target_tokens, _I32, (tokens,)), accepted=(accepted, _I32, (tokens,)),
                num_accepted=(num_accepted, _I32, (n,)), seq_lens=(seq_lens, _I32, (n,)), next_tokens=(next_tokens, _I32, (n,)),
                keep_blocks=(keep_blocks, _I32, (n,)))
        raise PkvError(1, func, f"the layers' pools are on device {layers.device}, not on the current CUDA device")
    status = L.pkv_commit_tree(layers.k_pointers, layers.v_pointers, layers.num_layers, ctypes.byref(layers.desc),
                               block_tables.data_ptr(), width, cu_q.data_ptr(), past_lens.data_ptr(), parents.data_ptr(),
                               draft_tokens.data_ptr(), target_tokens.data_ptr(), tokens, n, accepted.data_ptr(),
                               num_accepted.data_ptr(), seq_lens.data_ptr(), next_tokens.data_ptr(), _ptr(keep_blocks),
                               _ptr(device_error), _stream(stream, dev))
    if status:
        _check(status, func)


def pkv_status_string(status: int) -> str:
    return lib().pkv_status_string(int(status)).decode()


def pkv_last_error() -> str:
    return (lib().pkv_last_error() or b"").decode()


def pkv_abi_version() -> int:
    return int(lib().pkv_abi_version())
