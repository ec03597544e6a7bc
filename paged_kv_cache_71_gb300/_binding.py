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
    for name in ("pkv_reshape_and_cache", "pkv_paged_attention_workspace_size", "pkv_paged_attention_decode",
                 "pkv_copy_blocks", "pkv_paged_attention_decode_static_scratch", "pkv_paged_prefill_chunk",
                 "pkv_paged_prefill_varlen", "pkv_swap_blocks", "pkv_block_hashes", "pkv_extend_sequences",
                 "pkv_release_sequences", "pkv_paged_attention_decode_prefix",
                 "pkv_paged_attention_decode_prefix_workspace_size", "pkv_paged_cross_attention",
                 "pkv_paged_cross_attention_workspace_size"):
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


def pkv_status_string(status: int) -> str:
    return lib().pkv_status_string(int(status)).decode()


def pkv_last_error() -> str:
    return (lib().pkv_last_error() or b"").decode()


def pkv_abi_version() -> int:
    return int(lib().pkv_abi_version())
