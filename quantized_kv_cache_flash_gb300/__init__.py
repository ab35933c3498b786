"""Quantized-KV decode attention for GB300: Python binding of libtq.so.

Argument marshalling only.  Every step of the path (encode/append, decode,
split combine, inverse rotation) runs in the CUDA kernels of ``libtq.so``; the
functions here turn torch tensors into device pointers and call the C ABI of
``include/tq.h`` under the same names.  There is no CPU fallback: if the
library cannot be loaded every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtq.so")

TQ_OK = 0
TQ_ERR_INVALID_ARG = -1
TQ_ERR_UNSUPPORTED = -2
TQ_ERR_CAPACITY = -3
TQ_ERR_CUDA = -4
TQ_ERR_NOMEM = -5

TQ_TURBO4_ASYM = 0
TQ_TURBO3 = 1
TQ_TURBO4 = 2
TQ_TURBO3_ASYM = 3
TQ_TURBO4K_3V = 4
TQ_TURBO3_TABLE = 5
MODES = {"turbo4_asym": TQ_TURBO4_ASYM, "turbo3": TQ_TURBO3, "turbo4": TQ_TURBO4,
         "turbo3_asym": TQ_TURBO3_ASYM, "turbo4k_3v": TQ_TURBO4K_3V,
         "turbo3_table": TQ_TURBO3_TABLE}
MODE_BITS = {TQ_TURBO4_ASYM: (16, 4), TQ_TURBO3: (3, 3), TQ_TURBO4: (4, 4),
             TQ_TURBO3_ASYM: (16, 3), TQ_TURBO4K_3V: (4, 3), TQ_TURBO3_TABLE: (3, 3)}
# modes whose 64-byte records carry the centroid x norm table (no norm arrays)
TABLE_MODES = {TQ_TURBO3_TABLE}
TABLE_RECORD_BYTES = 64

TQ_STATUS_CAPACITY = 1
TQ_STATUS_NORM_OVERFLOW = 2
TQ_STATUS_SHORT_CONTEXT = 4
TQ_STATUS_PIPELINE_STALL = 8
TQ_STATUS_BAD_INDEX = 16

TQ_MAX_TREE_NODES = 256

# every entry point declared in include/tq.h: name -> (restype, argtypes)
_c = ctypes
_SIGS = {
    "tq_encode_append": (_c.c_int, [_c.POINTER(_c.c_void_p), _c.c_void_p, _c.c_void_p,
                                    _c.c_void_p, _c.c_int32, _c.c_void_p]),
    "tq_decode_attention": (_c.c_int, [_c.POINTER(_c.c_void_p), _c.c_void_p, _c.c_void_p,
                                       _c.c_int32, _c.c_int32, _c.c_int32, _c.c_float,
                                       _c.c_void_p, _c.c_void_p]),
    "tq_prefill_attention": (_c.c_int, [_c.POINTER(_c.c_void_p), _c.c_void_p, _c.c_void_p,
                                        _c.c_int32, _c.c_int32, _c.c_int32, _c.c_float,
                                        _c.c_void_p, _c.c_void_p]),
    "tq_decode_attention_sparse_v": (_c.c_int, [_c.POINTER(_c.c_void_p), _c.c_void_p,
                                                _c.c_void_p, _c.c_int32, _c.c_int32, _c.c_int32,
                                                _c.c_float, _c.c_float, _c.c_void_p,
                                                _c.c_void_p]),
    "tq_decode_attention_noalloc": (_c.c_int, [_c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_int32,
                                               _c.c_int32, _c.c_float, _c.c_void_p, _c.c_void_p,
                                               _c.c_void_p]),
    "tq_encode_append_packed": (_c.c_int, [_c.POINTER(_c.c_void_p), _c.c_void_p, _c.c_void_p,
                                           _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_void_p]),
    "tq_prefill_attention_packed": (_c.c_int, [_c.POINTER(_c.c_void_p), _c.c_void_p, _c.c_void_p,
                                               _c.c_int32, _c.c_void_p, _c.c_int32, _c.c_int32,
                                               _c.c_float, _c.c_void_p, _c.c_void_p]),
    "tq_tree_attention": (_c.c_int, [_c.POINTER(_c.c_void_p), _c.c_void_p, _c.c_void_p, _c.c_int32,
                                     _c.c_int32, _c.c_int32, _c.c_float, _c.c_void_p, _c.c_int32,
                                     _c.c_void_p, _c.c_void_p]),
    "tq_tree_mask": (_c.c_int, [_c.POINTER(_c.c_int32), _c.c_int32, _c.POINTER(_c.c_uint32)]),
    "tq_cache_compact": (_c.c_int, [_c.POINTER(_c.c_void_p), _c.c_void_p, _c.c_void_p, _c.c_int32,
                                    _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_void_p]),
    "tq_cache_copy": (_c.c_int, [_c.POINTER(_c.c_void_p), _c.c_void_p, _c.c_void_p, _c.c_void_p,
                                 _c.c_void_p, _c.c_void_p, _c.c_int32, _c.c_int32, _c.c_void_p]),
    "tq_selftest_bounded_wait": (_c.c_int, [_c.POINTER(_c.c_void_p), _c.c_int32, _c.c_void_p]),
    "tq_free": (None, [_c.c_void_p]),
    "tq_get_status": (_c.c_int, [_c.c_void_p, _c.POINTER(_c.c_uint32)]),
    "tq_lloyd_max_codebook": (_c.c_int, [_c.c_int32, _c.POINTER(_c.c_float)]),
    "tq_record_bytes": (_c.c_int, [_c.c_int32]),
    "tq_plan_splits": (_c.c_int, [_c.c_int32, _c.c_int32, _c.c_int32, _c.c_int32, _c.c_int32,
                                  _c.POINTER(_c.c_int32), _c.POINTER(_c.c_int32)]),
    "tq_get_sparse_v_tiles": (_c.c_int, [_c.c_void_p, _c.POINTER(_c.c_uint64),
                                         _c.POINTER(_c.c_uint64)]),
    "tq_set_kernel_timing": (_c.c_int, [_c.c_void_p, _c.c_int32]),
    "tq_get_kernel_time": (_c.c_int, [_c.c_void_p, _c.POINTER(_c.c_float),
                                      _c.POINTER(_c.c_int32)]),
    "tq_error_string": (_c.c_char_p, [_c.c_int32]),
}


class TqError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {error_string(code)} ({code})")


class tq_cache(ctypes.Structure):
    """Mirror of ``tq_cache`` in include/tq.h."""

    _fields_ = [
        ("mode", _c.c_int32), ("batch", _c.c_int32), ("num_kv_heads", _c.c_int32),
        ("head_dim", _c.c_int32), ("capacity", _c.c_int32),
        ("k_data", _c.c_void_p), ("k_norm", _c.c_void_p),
        ("v_data", _c.c_void_p), ("v_norm", _c.c_void_p),
        ("lengths", _c.c_void_p),
        ("codebook_k", _c.POINTER(_c.c_float)), ("codebook_k_size", _c.c_int32),
        ("codebook_v", _c.POINTER(_c.c_float)), ("codebook_v_size", _c.c_int32),
        ("rot_seed", _c.c_uint64), ("v_rescale", _c.c_float),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libtq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m quantized_kv_cache_flash_gb300.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib = h
    return _lib


def error_string(code: int) -> str:
    return lib().tq_error_string(code).decode()


def _check(code: int, where: str) -> None:
    if code != TQ_OK:
        raise TqError(code, where)


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


# What the calls on packed sequences, trees and moves need of torch, bound by the first
# cache (an import statement and torch.cuda's wrappers take 0.5 us of a call's 5.7).
_F16 = _I32 = _current_device = _current_stream = None


def _bind_torch() -> None:
    global _F16, _I32, _current_device, _current_stream
    import torch
    _F16, _I32 = torch.float16, torch.int32
    _current_device = getattr(torch._C, "_cuda_getDevice", None)
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    return int(getattr(stream, "cuda_stream", stream))


class Context:
    """Owner of a ``tq_ctx*`` (created lazily by the first call)."""

    def __init__(self):
        self.ptr = ctypes.c_void_p(None)
        self.ref = ctypes.byref(self.ptr)

    def free(self) -> None:
        if self.ptr.value:
            tq_free(self)
            self.ptr.value = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def tq_lloyd_max_codebook(bits: int):
    """The library's Lloyd-Max codebook of N(0, 1/128) (list of fp32 floats)."""
    n = 1 << bits
    buf = (ctypes.c_float * n)()
    _check(lib().tq_lloyd_max_codebook(bits, buf), "tq_lloyd_max_codebook")
    return [float(v) for v in buf]


def tq_record_bytes(bits: int) -> int:
    r = lib().tq_record_bytes(bits)
    if r < 0:
        raise TqError(r, "tq_record_bytes")
    return r


def tq_plan_splits(mode: int, batch: int, num_kv_heads: int, rows_per_kv_head: int,
                   max_len_hint: int):
    st, ns = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().tq_plan_splits(mode, batch, num_kv_heads, rows_per_kv_head, max_len_hint,
                                ctypes.byref(st), ctypes.byref(ns)), "tq_plan_splits")
    return st.value, ns.value


class Cache:
    """Device tensors of one packed cache plus the ``tq_cache`` struct that
    points at them.  Allocation is torch's; layout is the library's."""

    def __init__(self, mode: int, batch: int, num_kv_heads: int, capacity: int, device,
                 codebook_k=None, codebook_v=None, rot_seed: int = 42, v_rescale: float = 1.0):
        import torch
        if _F16 is None:
            _bind_torch()
        kb, vb = MODE_BITS[mode]
        self.mode, self.batch, self.num_kv_heads, self.capacity = mode, batch, num_kv_heads, capacity
        table = mode in TABLE_MODES
        if kb == 16:
            self.k_data = torch.zeros(batch, num_kv_heads, capacity, 128, dtype=torch.float16,
                                      device=device)
            self.k_norm = None
        elif table:
            self.k_data = torch.zeros(batch, num_kv_heads, capacity, TABLE_RECORD_BYTES,
                                      dtype=torch.uint8, device=device)
            self.k_norm = None
        else:
            self.k_data = torch.zeros(batch, num_kv_heads, capacity, tq_record_bytes(kb),
                                      dtype=torch.uint8, device=device)
            self.k_norm = torch.zeros(batch, num_kv_heads, capacity, dtype=torch.float16,
                                      device=device)
        self.v_data = torch.zeros(batch, num_kv_heads, capacity,
                                  TABLE_RECORD_BYTES if table else tq_record_bytes(vb),
                                  dtype=torch.uint8, device=device)
        self.v_norm = None if table else torch.zeros(batch, num_kv_heads, capacity,
                                                     dtype=torch.float16, device=device)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device=device)
        cbk = codebook_k if codebook_k is not None else (
            tq_lloyd_max_codebook(kb) if kb != 16 else [])
        cbv = codebook_v if codebook_v is not None else tq_lloyd_max_codebook(vb)
        self._cbk = (ctypes.c_float * max(len(cbk), 1))(*cbk)
        self._cbv = (ctypes.c_float * len(cbv))(*cbv)
        self.codebook_k = list(cbk)
        self.codebook_v = list(cbv)
        self.device = self.v_data.device
        self.device_index = self.v_data.get_device()   # (-1: not on a CUDA device)
        self.struct = tq_cache(
            mode, batch, num_kv_heads, 128, capacity,
            _ptr(self.k_data), _ptr(self.k_norm), _ptr(self.v_data), _ptr(self.v_norm),
            _ptr(self.lengths),
            ctypes.cast(self._cbk, ctypes.POINTER(ctypes.c_float)), len(cbk),
            ctypes.cast(self._cbv, ctypes.POINTER(ctypes.c_float)), len(cbv),
            rot_seed, v_rescale)
        self.ref = ctypes.byref(self.struct)

    def set_v_rescale(self, v: float) -> None:
        self.struct.v_rescale = v


def tq_encode_append(ctx: Context, cache: Cache, k_new, v_new, stream=None) -> None:
    """Append k_new/v_new fp16 [B, Hkv, T, 128] at lengths[b]; lengths += T (on device)."""
    import torch
    for t in (k_new, v_new):
        if t.dtype != torch.float16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("k_new/v_new must be contiguous fp16 [B, Hkv, T, 128]")
    t_new = int(k_new.shape[2])
    _check(lib().tq_encode_append(ctypes.byref(ctx.ptr), ctypes.byref(cache.struct),
                                  _ptr(k_new), _ptr(v_new), t_new, _stream(stream)),
           "tq_encode_append")


def tq_decode_attention(ctx: Context, cache: Cache, q, out, max_len_hint: int,
                        scale: float = 0.0, stream=None) -> None:
    """out[B, Hq, Tq, 128] = decode attention of q[B, Hq, Tq, 128] over the cache."""
    import torch
    if q.dtype != torch.float16 or not q.is_contiguous() or q.dim() != 4:
        raise ValueError("q must be contiguous fp16 [B, Hq, Tq, 128]")
    if out.dtype != torch.float16 or not out.is_contiguous() or out.shape != q.shape:
        raise ValueError("out must be contiguous fp16 shaped like q")
    _check(lib().tq_decode_attention(ctypes.byref(ctx.ptr), ctypes.byref(cache.struct),
                                     _ptr(q), int(q.shape[1]), int(q.shape[2]),
                                     int(max_len_hint), float(scale), _ptr(out),
                                     _stream(stream)), "tq_decode_attention")


def tq_prefill_attention(ctx: Context, cache: Cache, q, out, max_len_hint: int,
                         scale: float = 0.0, stream=None) -> None:
    """Attention of a block of many queries q[B, Hq, Tq, 128] (a prefill chunk
    already appended to the cache) on the tcgen05 tensor cores."""
    import torch
    if q.dtype != torch.float16 or not q.is_contiguous() or q.dim() != 4:
        raise ValueError("q must be contiguous fp16 [B, Hq, Tq, 128]")
    if out.dtype != torch.float16 or not out.is_contiguous() or out.shape != q.shape:
        raise ValueError("out must be contiguous fp16 shaped like q")
    _check(lib().tq_prefill_attention(ctypes.byref(ctx.ptr), ctypes.byref(cache.struct),
                                      _ptr(q), int(q.shape[1]), int(q.shape[2]),
                                      int(max_len_hint), float(scale), _ptr(out),
                                      _stream(stream)), "tq_prefill_attention")


def tq_decode_attention_sparse_v(ctx: Context, cache: Cache, q, out, max_len_hint: int,
                                 tau: float, scale: float = 0.0, stream=None) -> None:
    """Decode with the V of tokens whose softmax weight is below `tau` skipped."""
    import torch
    if q.dtype != torch.float16 or not q.is_contiguous() or q.dim() != 4:
        raise ValueError("q must be contiguous fp16 [B, Hq, Tq, 128]")
    if out.dtype != torch.float16 or not out.is_contiguous() or out.shape != q.shape:
        raise ValueError("out must be contiguous fp16 shaped like q")
    _check(lib().tq_decode_attention_sparse_v(ctypes.byref(ctx.ptr), ctypes.byref(cache.struct),
                                              _ptr(q), int(q.shape[1]), int(q.shape[2]),
                                              int(max_len_hint), float(scale), float(tau),
                                              _ptr(out), _stream(stream)),
           "tq_decode_attention_sparse_v")


def tq_decode_attention_noalloc(cache: Cache, q, out, max_len_hint: int, scale: float = 0.0,
                                status=None, stream=None) -> None:
    """Decode without a context and without any device allocation: the split-K
    scratch is the library's fixed device array (shared by all calls; serialise
    calls that could overlap on the GPU).  `status` is an optional int32/uint32
    device tensor of one element that the kernels OR status bits into."""
    import torch
    if q.dtype != torch.float16 or not q.is_contiguous() or q.dim() != 4:
        raise ValueError("q must be contiguous fp16 [B, Hq, Tq, 128]")
    if out.dtype != torch.float16 or not out.is_contiguous() or out.shape != q.shape:
        raise ValueError("out must be contiguous fp16 shaped like q")
    _check(lib().tq_decode_attention_noalloc(ctypes.byref(cache.struct), _ptr(q), int(q.shape[1]),
                                             int(q.shape[2]), int(max_len_hint), float(scale),
                                             _ptr(out), _ptr(status), _stream(stream)),
           "tq_decode_attention_noalloc")


def _tensor(name: str, t, dtype, shape, cache) -> None:
    """A contiguous tensor of this type and shape on the cache's device;
    ValueError otherwise."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == cache.device_index:
        return
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}"
                         + ("" if t.is_contiguous() else " (strided)"))
    if t.device != cache.device:
        raise ValueError(f"{name} is on {t.device}, the cache on {cache.device}")


def _int32(name: str, x) -> int:
    """x as the C call's 32-bit integer (ctypes would cut a larger one off)."""
    x = int(x)
    if not -0x80000000 <= x <= 0x7FFFFFFF:
        raise ValueError(f"{name} is past 32 bits: {x}")
    return x


def _launch_stream(cache, stream) -> int:
    """The stream handle of a call on this cache: the given one or the current
    one of the cache's device, which has to be the current device."""
    dev = cache.device_index
    if dev < 0 or dev != _current_device():
        raise ValueError(f"the cache is on {cache.device}, which is not the current CUDA device")
    if stream is None:
        return _current_stream(dev)
    return int(getattr(stream, "cuda_stream", stream))


def tq_encode_append_packed(ctx: Context, cache: Cache, k_new, v_new, cu_seqlens, stream=None) -> None:
    """Append packed k_new/v_new fp16 [total, Hkv, 128]: rows cu_seqlens[b] ..
    cu_seqlens[b + 1] - 1 (int32 [B + 1] on the device) go to sequence b."""
    shape = (k_new.shape[0], cache.num_kv_heads, 128)
    _tensor("k_new", k_new, _F16, shape, cache)
    _tensor("v_new", v_new, _F16, shape, cache)
    _tensor("cu_seqlens", cu_seqlens, _I32, (cache.batch + 1,), cache)
    _check(lib().tq_encode_append_packed(ctx.ref, cache.ref,
                                         k_new.data_ptr(), v_new.data_ptr(), cu_seqlens.data_ptr(),
                                         shape[0], _launch_stream(cache, stream)),
           "tq_encode_append_packed")


def tq_prefill_attention_packed(ctx: Context, cache: Cache, q, out, cu_seqlens, max_len_hint: int,
                                scale: float = 0.0, stream=None) -> None:
    """Causal attention of packed query blocks q[total, Hq, 128] (already
    appended to the cache): rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 belong
    to sequence b.  Output rows of no sequence are left as they were."""
    if q.dim() != 3:
        raise ValueError("q must be [total, Hq, 128]")
    total, hq, _ = q.shape
    _tensor("q", q, _F16, (total, hq, 128), cache)
    _tensor("out", out, _F16, q.shape, cache)
    _tensor("cu_seqlens", cu_seqlens, _I32, (cache.batch + 1,), cache)
    _check(lib().tq_prefill_attention_packed(ctx.ref, cache.ref,
                                             _ptr(q), int(q.shape[1]), _ptr(cu_seqlens),
                                             int(q.shape[0]), _int32("max_len_hint", max_len_hint), float(scale),
                                             _ptr(out), _launch_stream(cache, stream)),
           "tq_prefill_attention_packed")


def tq_tree_attention(ctx: Context, cache: Cache, q, out, tree_mask, max_len_hint: int,
                      scale: float = 0.0, stream=None) -> None:
    """Attention of a tree of drafted tokens q[B, Hq, Tq, 128], the last Tq
    tokens of every sequence.  tree_mask: int32 [1 or B, Tq, ceil(Tq / 32)]
    words (``tq_tree_mask``), bit i of row j set where node j sees node i."""
    if q.dim() != 4 or tree_mask.dim() != 3:
        raise ValueError("q must be [B, Hq, Tq, 128] and tree_mask [1 or B, Tq, ceil(Tq / 32)]")
    _, hq, n, _ = q.shape
    per_seq = tree_mask.shape[0]
    _tensor("q", q, _F16, (cache.batch, hq, n, 128), cache)
    _tensor("out", out, _F16, q.shape, cache)
    _tensor("tree_mask", tree_mask, _I32,
            (1 if per_seq == 1 else cache.batch, n, (n + 31) // 32), cache)
    _check(lib().tq_tree_attention(ctx.ref, cache.ref, q.data_ptr(),
                                   hq, n, _int32("max_len_hint", max_len_hint), float(scale),
                                   tree_mask.data_ptr(), per_seq, out.data_ptr(),
                                   _launch_stream(cache, stream)), "tq_tree_attention")


def tq_tree_mask(parents):
    """The int32 mask words [N, ceil(N / 32)] (a CPU tensor) of a tree whose
    node i follows node parents[i], or the context where that is -1."""
    import torch
    n = len(parents)
    words = (n + 31) // 32
    buf = (ctypes.c_uint32 * max(n * words, 1))()
    _check(lib().tq_tree_mask((ctypes.c_int32 * max(n, 1))(*[max(-2, min(int(x), n)) for x in parents]), n, buf),
           "tq_tree_mask")
    return torch.frombuffer(bytearray(buf), dtype=torch.int32).reshape(n, words)


def tq_cache_compact(ctx: Context, cache: Cache, start, keep, num_keep, num_drafted: int,
                     stream=None) -> None:
    """Keep tokens start[b] + keep[b, :num_keep[b]] of the drafted block
    [start[b], start[b] + num_drafted) as start[b], start[b] + 1, ... and cut
    the sequence off behind them (all int32 on the device)."""
    _tensor("start", start, _I32, (cache.batch,), cache)
    if keep.dim() != 2:
        raise ValueError("keep must be [B, max_keep]")
    _tensor("keep", keep, _I32, (cache.batch, keep.shape[1]), cache)
    _tensor("num_keep", num_keep, _I32, (cache.batch,), cache)
    _check(lib().tq_cache_compact(ctx.ref, cache.ref, start.data_ptr(),
                                  _int32("num_drafted", num_drafted), keep.data_ptr(), num_keep.data_ptr(), keep.shape[1],
                                  _launch_stream(cache, stream)), "tq_cache_compact")


def tq_cache_copy(ctx: Context, dst: Cache, src: Cache, dst_seq, src_seq, max_len_hint: int,
                  num_tokens=None, stream=None) -> None:
    """Sequence dst_seq[m] of `dst` becomes the first num_tokens[m] tokens (None:
    all) of sequence src_seq[m] of `src`, which may be the same cache."""
    m = dst_seq.numel()
    _tensor("dst_seq", dst_seq, _I32, (m,), dst)
    _tensor("src_seq", src_seq, _I32, (m,), dst)
    if num_tokens is not None:
        _tensor("num_tokens", num_tokens, _I32, (m,), dst)
    if src.device != dst.device:
        raise ValueError("the two caches are on different devices")
    _check(lib().tq_cache_copy(ctx.ref, dst.ref,
                               src.ref, dst_seq.data_ptr(), src_seq.data_ptr(),
                               _ptr(num_tokens), m, _int32("max_len_hint", max_len_hint), _launch_stream(dst, stream)),
           "tq_cache_copy")


def tq_selftest_bounded_wait(ctx: Context, limit_us: int, stream=None) -> None:
    """Make one bounded in-kernel wait run out (failure-path self-test)."""
    _check(lib().tq_selftest_bounded_wait(ctypes.byref(ctx.ptr), int(limit_us), _stream(stream)),
           "tq_selftest_bounded_wait")


def tq_free(ctx: Context) -> None:
    lib().tq_free(ctx.ptr)


def tq_get_status(ctx: Context) -> int:
    """Return and clear the device status bits (waits for the context's latest stream)."""
    s = ctypes.c_uint32()
    _check(lib().tq_get_status(ctx.ptr, ctypes.byref(s)), "tq_get_status")
    return s.value


def tq_get_sparse_v_tiles(ctx: Context):
    """(skipped, judged) 16-token tiles of the sparse-V decode since the last read."""
    a, b = ctypes.c_uint64(), ctypes.c_uint64()
    _check(lib().tq_get_sparse_v_tiles(ctx.ptr, ctypes.byref(a), ctypes.byref(b)),
           "tq_get_sparse_v_tiles")
    return a.value, b.value


def tq_set_kernel_timing(ctx: Context, enable: bool) -> None:
    _check(lib().tq_set_kernel_timing(ctx.ptr, 1 if enable else 0), "tq_set_kernel_timing")


def tq_get_kernel_time(ctx: Context):
    ms, n = ctypes.c_float(), ctypes.c_int32()
    _check(lib().tq_get_kernel_time(ctx.ptr, ctypes.byref(ms), ctypes.byref(n)),
           "tq_get_kernel_time")
    return ms.value, n.value
