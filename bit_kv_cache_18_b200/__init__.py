"""Python binding of libkvq.so, the B200 (sm_100a) quantized paged KV cache.

Argument marshalling only: every step of the write and read paths runs in the
library's CUDA kernels.  The names mirror include/kvq.h.  Torch is used for
device memory, dtypes and streams.  There is no fallback: if libkvq.so is
missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libkvq.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "kvq.h")

KVQ_OK = 0
KVQ_ERR_INVALID = -1
KVQ_ERR_UNSUPPORTED = -2
KVQ_ERR_CUDA = -3
KVQ_ERR_POOL_EXHAUSTED = -4
KVQ_ERR_OUT_OF_RANGE = -5
KVQ_ERR_DEVICE_TIMEOUT = -6
KVQ_ERR_WORKSPACE = -7

KVQ_F16, KVQ_BF16, KVQ_F32 = 0, 1, 2

HEAD_DIM = 128
BLOCK_SIZE = 16
SEGMENT_BYTES = 1664

_lock = threading.Lock()
_lib = None


class KvqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {kvq_error_string(status)} ({status})")


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("k_bits", ctypes.c_int32), ("v_bits", ctypes.c_int32), ("group", ctypes.c_int32),
                ("pool", ctypes.c_void_p)]


class WindowDesc(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_seqs", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("sink", ctypes.c_int32), ("recent", ctypes.c_int32)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("original_len", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double)]


class ScoreOpts(ctypes.Structure):
    _fields_ = [("softmax_scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("alibi_slopes", ctypes.c_void_p)]


def lib():
    """Load libkvq.so (raises if it is absent: there is no other path)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing; build it with python -m bit_kv_cache_18_b200.build")
            L = ctypes.CDLL(LIB_PATH)
            i32, i64, u64, sz, vp, f32 = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_size_t,
                                          ctypes.c_void_p, ctypes.c_float)
            dp = ctypes.POINTER(CacheDesc)
            sig = {
                "kvq_parse_dtype": (ctypes.c_int, [ctypes.c_char_p, vp, vp, vp]),
                "kvq_cache_bytes": (sz, [dp]),
                "kvq_block_table": (ctypes.c_int, [i32, i32, vp, i32, i32, u64, vp, vp]),
                "kvq_slot_mapping": (ctypes.c_int, [vp, i32, vp, vp, i32, i32, vp]),
                "kvq_quantize_append": (ctypes.c_int, [dp, vp, vp, ctypes.c_int, i32, i64, vp, vp]),
                "kvq_decode_workspace_bytes": (sz, [dp, i32, i32, i32]),
                "kvq_decode_workspace_bytes_ex": (sz, [dp, i32, i32, i32, i32]),
                "kvq_decode_attention": (ctypes.c_int, [dp, vp, ctypes.c_int, i32, i32, vp, i32, vp, i32, f32, vp,
                                                        ctypes.c_int, vp, sz, vp]),
                "kvq_decode_attention_ex": (ctypes.c_int, [dp, vp, ctypes.c_int, i32, i32, vp, i32, vp, i32, f32,
                                                           vp, ctypes.c_int, vp, sz, i32, vp]),
                "kvq_decode_attention_noalloc": (ctypes.c_int, [dp, vp, ctypes.c_int, i32, i32, vp, i32, vp, i32, f32,
                                                                vp, ctypes.c_int, vp]),
                "kvq_append_decode_attention": (ctypes.c_int, [dp, vp, vp, ctypes.c_int, i64, vp, ctypes.c_int, i32,
                                                               i32, vp, i32, vp, i32, f32, vp, ctypes.c_int, vp, sz,
                                                               vp]),
                "kvq_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint32, vp, vp]),
                "kvq_window_bytes": (sz, [ctypes.POINTER(WindowDesc)]),
                "kvq_window_append": (ctypes.c_int, [ctypes.POINTER(WindowDesc), vp, vp, i64, vp, vp, i32, vp]),
                "kvq_decode_window_workspace_bytes": (sz, [dp, i32, i32, i32]),
                "kvq_decode_attention_window": (ctypes.c_int, [dp, ctypes.POINTER(WindowDesc), vp, ctypes.c_int, i32,
                                                               i32, vp, i32, vp, i32, f32, vp, ctypes.c_int, vp, sz,
                                                               vp]),
                "kvq_update_tables": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, vp, vp, vp,
                                                     vp]),
                "kvq_rope_table": (ctypes.c_int, [ctypes.POINTER(RopeDesc), vp, vp]),
                "kvq_rope": (ctypes.c_int, [ctypes.POINTER(RopeDesc), vp, f32, vp, i32, vp, i64, vp, i64, i32, vp,
                                            i64, vp, i64, i32, ctypes.c_int, vp]),
                "kvq_prefill_attention": (ctypes.c_int, [ctypes.POINTER(ScoreOpts), vp, i64, vp, i64, vp, i64, vp, i64,
                                                         i32, i32, i32, vp, i32, vp, ctypes.c_int, vp]),
                "kvq_decode_scored_workspace_bytes": (sz, [dp, i32, i32, i32, i32]),
                "kvq_decode_attention_scored": (ctypes.c_int, [dp, ctypes.POINTER(ScoreOpts), vp, ctypes.c_int, i32,
                                                               i32, vp, i32, vp, i32, vp, ctypes.c_int, vp, sz, vp]),
                "kvq_last_device_status": (ctypes.c_int, [vp]),
                "kvq_error_string": (ctypes.c_char_p, [ctypes.c_int]),
            }
            for name, (res, args) in sig.items():
                f = getattr(L, name)
                f.restype, f.argtypes = res, args
            _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/kvq.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(kvq_[a-z_]+)\s*\(", text)))


def kvq_error_string(status: int) -> str:
    return lib().kvq_error_string(status).decode()


def _check(rc: int, what: str):
    if rc != KVQ_OK:
        raise KvqError(rc, what)


def _stream_ptr(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t) -> int:
    import torch
    return {torch.float16: KVQ_F16, torch.bfloat16: KVQ_BF16, torch.float32: KVQ_F32}[t.dtype]


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


# ---- host-only helpers -------------------------------------------------------

def kvq_parse_dtype(s: str):
    kb, vb, g = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    rc = lib().kvq_parse_dtype(s.encode(), ctypes.byref(kb), ctypes.byref(vb), ctypes.byref(g))
    return rc, (kb.value, vb.value, g.value)


# The cache presets the library builds, as (key bits, value bits); the first
# is the pages' default, kvarn_k4v2_g128.
PRESETS = ((4, 2), (4, 4), (2, 2), (8, 4))


def make_desc(num_blocks: int, num_kv_heads: int, pool=None, preset=(4, 2)) -> CacheDesc:
    return CacheDesc(num_blocks, BLOCK_SIZE, num_kv_heads, HEAD_DIM, preset[0], preset[1], HEAD_DIM,
                     pool.data_ptr() if pool is not None else None)


def kvq_cache_bytes(desc: CacheDesc) -> int:
    return lib().kvq_cache_bytes(ctypes.byref(desc))


def kvq_block_table(num_blocks, seq_lens, max_blocks_per_seq, shuffle_seed=0, block_size=BLOCK_SIZE):
    """-> (block_table int32 numpy [batch, max_blocks_per_seq], blocks_used)"""
    import numpy as np
    lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
    out = np.empty((lens.size, max_blocks_per_seq), dtype=np.int32)
    used = ctypes.c_int32()
    _check(lib().kvq_block_table(num_blocks, block_size, lens.ctypes.data, lens.size, max_blocks_per_seq,
                                 shuffle_seed, out.ctypes.data, ctypes.byref(used)), "kvq_block_table")
    return out, used.value


def kvq_slot_mapping(block_table, positions, seq_ids, block_size=BLOCK_SIZE):
    import numpy as np
    bt = np.ascontiguousarray(block_table, dtype=np.int32)
    pos = np.ascontiguousarray(positions, dtype=np.int32)
    sid = np.ascontiguousarray(seq_ids, dtype=np.int32)
    out = np.empty(pos.size, dtype=np.int32)
    _check(lib().kvq_slot_mapping(bt.ctypes.data, bt.shape[1], pos.ctypes.data, sid.ctypes.data, pos.size,
                                  block_size, out.ctypes.data), "kvq_slot_mapping")
    return out


# ---- device calls ------------------------------------------------------------

def new_pool(num_blocks: int, num_kv_heads: int, device="cuda", preset=(4, 2)):
    """A caller-owned pool tensor (uint8) sized by kvq_cache_bytes."""
    import torch
    nbytes = kvq_cache_bytes(make_desc(num_blocks, num_kv_heads, preset=preset))
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def kvq_quantize_append(pool, num_blocks, num_kv_heads, k, v, slot_mapping, stream=None, token_stride=None,
                        preset=(4, 2)):
    """k, v: [n_tokens, ..., Hkv*128 elements per row] fp16/bf16 device tensors
    with stride(0) = token_stride; slot_mapping: int32 device [n_tokens]."""
    desc = make_desc(num_blocks, num_kv_heads, pool, preset)
    n = int(slot_mapping.numel())
    ts = k.stride(0) if token_stride is None else token_stride
    rc = lib().kvq_quantize_append(ctypes.byref(desc), _ptr(k), _ptr(v), _dtype_code(k), n, ts, _ptr(slot_mapping),
                                   _stream_ptr(stream))
    _check(rc, "kvq_quantize_append")


def kvq_decode_workspace_bytes(num_blocks, num_kv_heads, batch, num_q_heads, max_seq_len, blocks_per_split=0,
                               preset=(4, 2)):
    desc = make_desc(num_blocks, num_kv_heads, preset=preset)
    return lib().kvq_decode_workspace_bytes_ex(ctypes.byref(desc), batch, num_q_heads, max_seq_len,
                                               blocks_per_split)


def new_workspace(num_blocks, num_kv_heads, batch, num_q_heads, max_seq_len, blocks_per_split=0, device="cuda",
                  preset=(4, 2)):
    import torch
    n = kvq_decode_workspace_bytes(num_blocks, num_kv_heads, batch, num_q_heads, max_seq_len, blocks_per_split,
                                   preset)
    if n == 0:
        raise KvqError(KVQ_ERR_UNSUPPORTED, "kvq_decode_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def kvq_decode_attention(pool, num_blocks, num_kv_heads, q, block_table, seq_lens, max_seq_len, out, workspace,
                         softmax_scale=0.0, blocks_per_split=0, stream=None, preset=(4, 2)):
    """q: [batch, Hq, 128] device; block_table int32 [batch, max_blocks]; seq_lens int32 [batch];
    out: [batch, Hq, 128] device (fp32/bf16/fp16); workspace from new_workspace()."""
    desc = make_desc(num_blocks, num_kv_heads, pool, preset)
    batch, hq, _ = q.shape
    rc = lib().kvq_decode_attention_ex(ctypes.byref(desc), _ptr(q), _dtype_code(q), batch, hq, _ptr(block_table),
                                       block_table.shape[1], _ptr(seq_lens), max_seq_len, softmax_scale, _ptr(out),
                                       _dtype_code(out), _ptr(workspace), workspace.numel(), blocks_per_split,
                                       _stream_ptr(stream))
    _check(rc, "kvq_decode_attention")


def kvq_append_decode_attention(pool, num_blocks, num_kv_heads, k_new, v_new, q, block_table, seq_lens, max_seq_len,
                                out, workspace, softmax_scale=0.0, stream=None, token_stride=None, preset=(4, 2)):
    """One fused decode step: the new token of each sequence (k_new, v_new:
    [batch, ..., Hkv*128] fp16/bf16 rows) is quantized into position
    seq_lens[b] - 1, then decode attention runs over the grown cache."""
    desc = make_desc(num_blocks, num_kv_heads, pool, preset)
    batch, hq, _ = q.shape
    ts = k_new.stride(0) if token_stride is None else token_stride
    rc = lib().kvq_append_decode_attention(ctypes.byref(desc), _ptr(k_new), _ptr(v_new), _dtype_code(k_new), ts,
                                           _ptr(q), _dtype_code(q), batch, hq, _ptr(block_table),
                                           block_table.shape[1], _ptr(seq_lens), max_seq_len, softmax_scale,
                                           _ptr(out), _dtype_code(out), _ptr(workspace), workspace.numel(),
                                           _stream_ptr(stream))
    _check(rc, "kvq_append_decode_attention")


def kvq_decode_attention_noalloc(pool, num_blocks, num_kv_heads, q, block_table, seq_lens, max_seq_len, out,
                                 softmax_scale=0.0, stream=None, preset=(4, 2)):
    """kvq_decode_attention with the library's fixed device scratch instead of
    a caller workspace (for callers that cannot allocate at call time)."""
    desc = make_desc(num_blocks, num_kv_heads, pool, preset)
    batch, hq, _ = q.shape
    rc = lib().kvq_decode_attention_noalloc(ctypes.byref(desc), _ptr(q), _dtype_code(q), batch, hq,
                                            _ptr(block_table), block_table.shape[1], _ptr(seq_lens), max_seq_len,
                                            softmax_scale, _ptr(out), _dtype_code(out), _stream_ptr(stream))
    _check(rc, "kvq_decode_attention_noalloc")


# ---- bf16 window of sink and recent tokens -------------------------------------

def make_window(num_seqs, num_kv_heads, sink, recent, data=None) -> WindowDesc:
    return WindowDesc(data.data_ptr() if data is not None else None, num_seqs, num_kv_heads, sink, recent)


def kvq_window_bytes(num_seqs, num_kv_heads, sink, recent) -> int:
    return lib().kvq_window_bytes(ctypes.byref(make_window(num_seqs, num_kv_heads, sink, recent)))


def new_window(num_seqs, num_kv_heads, sink, recent, device="cuda"):
    """A zeroed window buffer: bf16 [num_seqs, Hkv, sink + recent, 2, 128]."""
    import torch
    if kvq_window_bytes(num_seqs, num_kv_heads, sink, recent) == 0 and num_seqs * (sink + recent) > 0:
        raise KvqError(KVQ_ERR_INVALID, "kvq_window_bytes")
    return torch.zeros((num_seqs, num_kv_heads, sink + recent, 2, HEAD_DIM), dtype=torch.bfloat16, device=device)


def kvq_window_append(window, sink, recent, k, v, seq_ids, positions, stream=None, token_stride=None):
    """k, v: [n, ..., Hkv*128] bf16 rows; seq_ids, positions: int32 [n] device."""
    num_seqs, hkv = window.shape[0], window.shape[1]
    w = make_window(num_seqs, hkv, sink, recent, window)
    ts = k.stride(0) if token_stride is None else token_stride
    rc = lib().kvq_window_append(ctypes.byref(w), _ptr(k), _ptr(v), ts, _ptr(seq_ids), _ptr(positions),
                                 seq_ids.numel(), _stream_ptr(stream))
    _check(rc, "kvq_window_append")


def new_window_workspace(num_blocks, num_kv_heads, batch, num_q_heads, max_seq_len, device="cuda", preset=(4, 2)):
    import torch
    desc = make_desc(num_blocks, num_kv_heads, preset=preset)
    n = lib().kvq_decode_window_workspace_bytes(ctypes.byref(desc), batch, num_q_heads, max_seq_len)
    if n == 0:
        raise KvqError(KVQ_ERR_UNSUPPORTED, "kvq_decode_window_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def kvq_decode_attention_window(pool, num_blocks, num_kv_heads, window, sink, recent, q, block_table, seq_lens,
                                max_seq_len, out, workspace, softmax_scale=0.0, stream=None, preset=(4, 2)):
    """kvq_decode_attention with the window's raw rows at the sink and recent
    positions; workspace from new_window_workspace()."""
    desc = make_desc(num_blocks, num_kv_heads, pool, preset)
    w = make_window(window.shape[0], window.shape[1], sink, recent, window)
    batch, hq, _ = q.shape
    rc = lib().kvq_decode_attention_window(ctypes.byref(desc), ctypes.byref(w), _ptr(q), _dtype_code(q), batch, hq,
                                           _ptr(block_table), block_table.shape[1], _ptr(seq_lens), max_seq_len,
                                           softmax_scale, _ptr(out), _dtype_code(out), _ptr(workspace),
                                           workspace.numel(), _stream_ptr(stream))
    _check(rc, "kvq_decode_attention_window")


# ---- a serving step around the cache --------------------------------------------
# These calls are short on the device (a few microseconds for a decode step), so
# their checks are kept to a handful of attribute reads, without generators,
# imports or formatted messages on the way of a call that is right.

_torch = None
_codes = {}


def _need_torch():
    global _torch, _codes
    if _torch is None:
        import torch
        _codes = {torch.float16: KVQ_F16, torch.bfloat16: KVQ_BF16, torch.float32: KVQ_F32}
        _torch = torch
    return _torch


def _refuse(what: str, why: str):
    """Argument rules that only the tensors show (shape, type, layout, device):
    refused like the library's own, before anything is launched."""
    raise KvqError(KVQ_ERR_INVALID, f"{what}: {why}")


def _on_device(what: str, *tensors) -> int:
    """The current CUDA device, where the launch goes and every tensor has to be."""
    dev = (_torch or _need_torch())._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _refuse(what, "a tensor is not on the current CUDA device")
    return dev


def _all_int32(what: str, *tensors):
    i32 = _torch.int32
    for t in tensors:
        if t is not None and not (t.dtype is i32 and t.is_contiguous()):
            _refuse(what, "tables and lengths are contiguous int32 tensors")


def _rows(what: str, t):
    """[n, heads, 128] with contiguous heads -> n, heads, elements from one
    token's row to the next (any value does for a single row)."""
    try:
        n, heads, d = t.shape
    except ValueError:
        d = 0
    if d != HEAD_DIM:
        _refuse(what, "rows are [tokens, heads, 128]")
    if t.is_contiguous():
        return n, heads, heads * HEAD_DIM
    row, head, one = t.stride()
    if one != 1 or (heads > 1 and head != HEAD_DIM):
        _refuse(what, "rows are [tokens, heads, 128] with contiguous heads")
    return n, heads, row if n > 1 else heads * HEAD_DIM


def _addr(t):
    return t.data_ptr() if t is not None else None


def _stream_of(stream, dev: int):
    return _torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def kvq_update_tables(ring, state_in, state_out, seq_lens, target_lens, lens_out, block_table, cu_seqlens, positions,
                      seq_ids, slots, stream=None):
    """Block tables and slot maps of a step from its request lengths: int32
    device tensors ring [capacity], state_in and state_out [4] (head, count,
    two words that are zero at first; they may be one tensor), seq_lens,
    target_lens and lens_out [batch], block_table [batch, max_blocks],
    cu_seqlens [batch + 1], positions, seq_ids and slots [max_tokens]."""
    what = "kvq_update_tables"
    every = (ring, state_in, state_out, seq_lens, target_lens, lens_out, block_table, cu_seqlens, positions, seq_ids,
             slots)
    dev, i32 = (_torch or _need_torch())._C._cuda_getDevice(), _torch.int32
    for t in every:
        if t.get_device() != dev or t.dtype is not i32 or not t.is_contiguous():
            _on_device(what, t)
            _all_int32(what, t)
    batch, n = seq_lens.numel(), positions.numel()
    if not (state_in.numel() >= 4 and state_out.numel() >= 4 and target_lens.numel() == batch and
            lens_out.numel() == batch and block_table.dim() == 2 and block_table.shape[0] == batch and
            cu_seqlens.numel() == batch + 1 and seq_ids.numel() == n and slots.numel() == n):
        _refuse(what, "buffer sizes")
    rc = (_lib or lib()).kvq_update_tables(ring.data_ptr(), ring.numel(), state_in.data_ptr(), state_out.data_ptr(),
                                           seq_lens.data_ptr(), target_lens.data_ptr(), lens_out.data_ptr(), batch,
                                           block_table.data_ptr(), block_table.shape[1], cu_seqlens.data_ptr(), n,
                                           positions.data_ptr(), seq_ids.data_ptr(), slots.data_ptr(),
                                           _stream_of(stream, dev))
    if rc:
        raise KvqError(rc, what)


ROPE_SCALINGS = ("none", "linear", "ntk", "bands", "yarn")


def make_rope(rotary_dim=HEAD_DIM, base=10000.0, interleaved=False, scaling="none", factor=1.0, original_len=0,
              low=0.0, high=0.0) -> RopeDesc:
    if scaling not in ROPE_SCALINGS:
        _refuse("make_rope", "scaling")
    return RopeDesc(rotary_dim, int(interleaved), ROPE_SCALINGS.index(scaling), original_len, base, factor, low, high)


def kvq_rope_table(desc: RopeDesc):
    """-> (uint64 numpy [rotary_dim / 2]: turns per position in units of 2^-64, magnitude)"""
    import numpy as np
    turns = np.zeros(max(desc.rotary_dim // 2, 1), dtype=np.uint64)
    mag = ctypes.c_float()
    _check(lib().kvq_rope_table(ctypes.byref(desc), turns.ctypes.data, ctypes.byref(mag)), "kvq_rope_table")
    return turns, mag.value


def new_rope_table(desc: RopeDesc, device="cuda"):
    """-> (the table on the device, as int64, magnitude)"""
    import numpy as np
    import torch
    turns, mag = kvq_rope_table(desc)
    return torch.from_numpy(turns.view(np.int64)).to(device), mag


def kvq_rope(desc, table, magnitude, positions, q, k=None, q_out=None, k_out=None, stream=None):
    """Rotate q [n, Hq, 128] and k [n, Hkv, 128] (fp16 or bf16) by positions
    (int32 [n]) into q_out and k_out, in place where those are None."""
    what = "kvq_rope"
    if k is None and k_out is not None:
        _refuse(what, "k_out without k")
    dev = _on_device(what, table, positions, q, k, q_out, k_out)
    _all_int32(what, positions)
    if not (table.dtype is _torch.int64 and table.is_contiguous() and table.numel() == desc.rotary_dim // 2):
        _refuse(what, "a table of another descriptor")
    n, dtype = positions.numel(), q.dtype
    nq, hq, qs = _rows(what, q)
    qos, hk, ks, kos = qs, 0, 0, 0
    ok = nq == n and dtype in _codes
    if q_out is None:
        q_out = q
    else:
        no, ho, qos = _rows(what, q_out)
        ok = ok and no == n and ho == hq and q_out.dtype is dtype
    if k is not None:
        nk, hk, ks = _rows(what, k)
        kos = ks
        ok = ok and nk == n and k.dtype is dtype
        if k_out is None:
            k_out = k
        else:
            no, ho, kos = _rows(what, k_out)
            ok = ok and no == n and ho == hk and k_out.dtype is dtype
    if not ok:
        _refuse(what, "shapes and types")
    rc = (_lib or lib()).kvq_rope(ctypes.byref(desc), table.data_ptr(), magnitude, positions.data_ptr(), n,
                                  q.data_ptr(), qs, q_out.data_ptr(), qos, hq, _addr(k), ks, _addr(k_out), kos, hk,
                                  _codes[dtype], _stream_of(stream, dev))
    if rc:
        raise KvqError(rc, what)


def make_score_opts(softmax_scale=0.0, softcap=0.0, window=0, alibi_slopes=None) -> ScoreOpts:
    """alibi_slopes: fp32 device tensor [num_q_heads], kept alive by the options."""
    if alibi_slopes is not None:
        if not (alibi_slopes.is_cuda and alibi_slopes.dtype is _need_torch().float32 and alibi_slopes.is_contiguous()):
            _refuse("make_score_opts", "alibi_slopes is a contiguous fp32 device tensor")
    if not 0 <= window < 2 ** 31:
        _refuse("make_score_opts", "window")
    o = ScoreOpts(softmax_scale, softcap, window, _addr(alibi_slopes))
    o.slopes_tensor = alibi_slopes
    return o


def _slopes_of(what: str, opts, num_q_heads: int):
    """The options' slopes (None without), one per query head."""
    slopes = getattr(opts, "slopes_tensor", None)
    if slopes is not None and slopes.numel() != num_q_heads:
        _refuse(what, "one slope per query head")
    return slopes


def kvq_prefill_attention(q, k, v, cu_seqlens, out, opts=None, prefix_lens=None, stream=None):
    """Attention of whole prompts over their own rows, with no history in the
    cache: q and out [n, Hq, 128],
    k and v [n, Hkv, 128] (fp16 or bf16; slices of a fused projection do),
    cu_seqlens int32 [batch + 1], prefix_lens int32 [batch] or None, opts from
    make_score_opts."""
    what = "kvq_prefill_attention"
    nq, hq, qs = _rows(what, q)
    dev = _on_device(what, q, k, v, out, cu_seqlens, prefix_lens, _slopes_of(what, opts, hq))
    _all_int32(what, cu_seqlens, prefix_lens)
    nk, hk, ks = _rows(what, k)
    nv, hv, vs = _rows(what, v)
    no, ho, os_ = _rows(what, out)
    batch, dtype = cu_seqlens.numel() - 1, q.dtype
    if not (batch >= 0 and nq == nk == nv == no and ho == hq and hv == hk and dtype in _codes and k.dtype is dtype and
            v.dtype is dtype and out.dtype is dtype and (prefix_lens is None or prefix_lens.numel() == batch)):
        _refuse(what, "shapes and types")
    rc = (_lib or lib()).kvq_prefill_attention(ctypes.byref(opts) if opts is not None else None, q.data_ptr(), qs,
                                               k.data_ptr(), ks, v.data_ptr(), vs, out.data_ptr(), os_, nq, hq, hk,
                                               cu_seqlens.data_ptr(), batch, _addr(prefix_lens), _codes[dtype],
                                               _stream_of(stream, dev))
    if rc:
        raise KvqError(rc, what)


def kvq_decode_scored_workspace_bytes(num_blocks, num_kv_heads, batch, num_q_heads, max_seq_len, window=0,
                                      preset=(4, 2)) -> int:
    desc = make_desc(num_blocks, num_kv_heads, preset=preset)
    return lib().kvq_decode_scored_workspace_bytes(ctypes.byref(desc), batch, num_q_heads, max_seq_len, window)


def new_scored_workspace(num_blocks, num_kv_heads, batch, num_q_heads, max_seq_len, window=0, device="cuda",
                         preset=(4, 2)):
    import torch
    n = kvq_decode_scored_workspace_bytes(num_blocks, num_kv_heads, batch, num_q_heads, max_seq_len, window, preset)
    if n == 0 and batch > 0:
        raise KvqError(KVQ_ERR_UNSUPPORTED, "kvq_decode_scored_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=64)
def _desc_image(num_blocks: int, num_kv_heads: int, preset):
    """A cache descriptor without a pool, as bytes to copy (a few times cheaper
    than its fields one by one), and the size of its pool."""
    desc = make_desc(num_blocks, num_kv_heads, preset=preset)
    return bytes(desc), lib().kvq_cache_bytes(ctypes.byref(desc))


def kvq_decode_attention_scored(pool, num_blocks, num_kv_heads, q, block_table, seq_lens, max_seq_len, out, workspace,
                                opts=None, stream=None, preset=(4, 2)):
    """kvq_decode_attention with score options (make_score_opts); q[b] is
    sequence b's query: packed row cu_seqlens[b] of a step whose tables
    kvq_update_tables made; workspace from new_scored_workspace() with the same
    window."""
    what = "kvq_decode_attention_scored"
    if q.dim() != 3:
        _refuse(what, "q is [batch, heads, 128]")
    batch, hq, d = q.shape
    image, pool_bytes = _desc_image(num_blocks, num_kv_heads, tuple(preset))
    desc = CacheDesc.from_buffer_copy(image)
    desc.pool = pool.data_ptr()
    dev = _on_device(what, pool, q, block_table, seq_lens, out, workspace, _slopes_of(what, opts, hq))
    _all_int32(what, block_table, seq_lens)
    if not (d == HEAD_DIM and q.is_contiguous() and out.is_contiguous() and out.shape == q.shape and
            q.dtype in _codes and out.dtype in _codes and block_table.dim() == 2 and block_table.shape[0] == batch and
            seq_lens.numel() == batch and workspace.is_contiguous()):
        _refuse(what, "shapes, types and layout")
    # (a pool of an unsupported preset has no size: the library refuses it below)
    if not pool.is_contiguous() or pool.numel() * pool.element_size() < pool_bytes:
        _refuse(what, "pool too small")
    rc = (_lib or lib()).kvq_decode_attention_scored(ctypes.byref(desc),
                                                     ctypes.byref(opts) if opts is not None else None, q.data_ptr(),
                                                     _codes[q.dtype], batch, hq, block_table.data_ptr(),
                                                     block_table.shape[1], seq_lens.data_ptr(), max_seq_len,
                                                     out.data_ptr(), _codes[out.dtype], workspace.data_ptr(),
                                                     workspace.numel() * workspace.element_size(),
                                                     _stream_of(stream, dev))
    if rc:
        raise KvqError(rc, what)


def kvq_selftest_wait_timeout(limit_us: int, elapsed_ns=None, stream=None):
    """Launch the bounded-wait self-test (a wait that must give up after
    limit_us microseconds); elapsed_ns: optional int64 device tensor of one
    element."""
    rc = lib().kvq_selftest_wait_timeout(limit_us, _ptr(elapsed_ns), _stream_ptr(stream))
    _check(rc, "kvq_selftest_wait_timeout")


def kvq_last_device_status(stream=None) -> int:
    return lib().kvq_last_device_status(_stream_ptr(stream))
