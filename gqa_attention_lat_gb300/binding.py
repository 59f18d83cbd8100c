"""ctypes binding of the lat_attn C ABI (include/lat_attn.h).

Argument marshalling only: every function forwards to the CUDA library under the same
name and argument order, by way of the C extension that the build writes out from the
signatures below, or by ctypes where there is none or the library is not the one beside it
(sizes and names always by ctypes).  Pointer arguments accept a torch tensor (its data_ptr),
an int address or None (NULL); ``stream`` accepts a torch.cuda.Stream, an int handle or None
(torch's current stream when CUDA is up, else the legacy default stream).  Either way a wrong
type raises TypeError (AttributeError for a pointer), a whole number past its argument's range
OverflowError, and a non-OK status LatError.  There is no CPU fallback: if the library is not
built, the first call raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import operator
import os
import sys
import threading
import types

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblat_attn.so")
# (the suffix names the interpreter: an extension of another one is not taken for this one's)
CALLER_PATH = os.path.join(HERE, "_lat_call" + importlib.machinery.EXTENSION_SUFFIXES[0])

LAT_F32, LAT_BF16 = 0, 1
STATUS_NAMES = {0: "LAT_OK", 1: "LAT_ERR_INVALID_ARG", 2: "LAT_ERR_UNSUPPORTED",
                3: "LAT_ERR_WORKSPACE", 4: "LAT_ERR_CUDA", 5: "LAT_ERR_BOUNDS",
                6: "LAT_ERR_TIMEOUT"}
(LAT_OK, LAT_ERR_INVALID_ARG, LAT_ERR_UNSUPPORTED, LAT_ERR_WORKSPACE, LAT_ERR_CUDA,
 LAT_ERR_BOUNDS, LAT_ERR_TIMEOUT) = range(7)


class LatError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s" % (where, STATUS_NAMES.get(status, str(status))))


_lock = threading.Lock()
_lib = None
_caller = None

_P, _I64, _I32, _F32, _SZ, _U64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                   ctypes.c_float, ctypes.c_size_t, ctypes.c_uint64)
_SIGNATURES = {
    "lat_status_string": (ctypes.c_char_p, [_I32]),
    "lat_attn_prefill": (_I32, [_I32, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P,
                                _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P, _P]),
    "lat_attn_prefill_cached": (_I32, [_I32, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I64, _P,
                                       _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P,
                                       _P]),
    "lat_attn_prefill_softcap": (_I32, [_I32, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P,
                                        _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _F32,
                                        _F32, _P, _P]),
    "lat_attn_decode_softcap": (_I32, [_I32, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I32, _P,
                                       _I64, _P, _I32, _I32, _I32, _I32, _I32, _F32, _F32, _P,
                                       _SZ, _P, _P]),
    "lat_attn_decode_ring": (_I32, [_I32, _P, _I64, _P, _P, _I64, _I64, _I64, _I32, _P, _I32,
                                    _P, _I64, _P, _I32, _I32, _I32, _I32, _I32, _F32, _P, _SZ,
                                    _P, _P]),
    "lat_kv_append_ring": (_I32, [_I32, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _I64, _P, _I32,
                                  _I32, _I32, _I32, _P, _P]),
    "lat_qkv_norm_rope_append": (_I32, [_I32, _P, _I64, _P, _P, _F32, ctypes.c_double, _I32,
                                        _P, _I64, _P, _P, _I64, _I64, _I64, _I32, _P, _I32,
                                        _I32, _I32, _I32, _I32, _P, _P]),
    "lat_attn_decode_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "lat_attn_decode": (_I32, [_I32, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I32, _P, _I64,
                               _P, _I32, _I32, _I32, _I32, _I32, _F32, _P, _SZ, _P, _P]),
    "lat_attn_decode_static": (_I32, [_I32, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I32, _P,
                                      _I64, _P, _I32, _I32, _I32, _I32, _I32, _F32, _P, _P]),
    "lat_kv_append": (_I32, [_I32, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _I64, _P, _I32,
                             _I32, _I32, _I32, _P, _P]),
    "lat_kv_q4_row_bytes": (_I32, [_I32]),
    "lat_kv_append_q4": (_I32, [_I32, _P, _I64, _I64, _I64, _I32, _P, _P, _I64, _P, _I32, _I32,
                                _I32, _I32, _P, _P]),
    "lat_kv_expand_q4": (_I32, [_I32, _P, _I64, _I64, _I64, _I32, _P, _P, _I64, _P, _I32, _I32,
                                _I32, _I32, _P, _P]),
    "lat_attn_decode_q4_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    "lat_attn_decode_q4": (_I32, [_I32, _P, _I64, _P, _I64, _I64, _I64, _P, _I32, _P, _I64, _P,
                                  _I32, _I32, _I32, _I32, _I32, _F32, _F32, _P, _SZ, _P, _P]),
    "lat_kv_block_bounds": (_I32, [_I32, _P, _I64, _I64, _I64, _I32, _P, _I64, _I64, _I64, _I32,
                                   _P, _I32, _I32, _I32, _I32, _P, _P]),
    "lat_attn_select_blocks_workspace_size": (_SZ, [_I32, _I32, _I32, _I32]),
    "lat_attn_select_blocks": (_I32, [_I32, _P, _I64, _P, _I64, _I64, _I64, _I32, _P, _I32, _P,
                                      _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P, _SZ, _P,
                                      _P]),
    "lat_attn_decode_blocks_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "lat_attn_decode_blocks": (_I32, [_I32, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I32, _I32,
                                      _P, _I32, _P, _I64, _P, _I32, _I32, _I32, _I32, _F32,
                                      _F32, _P, _SZ, _P, _P]),
    "lat_test_prefill_timeout": (_I32, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I32, _I32,
                                        _I32, _I32, _I32, _U64, _P, _P]),
    "lat_test_decode_timeout": (_I32, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _I32, _P, _I64,
                                       _I32, _I32, _I32, _I32, _P, _SZ, _U64, _P, _P]),
    "lat_test_decode_q4_timeout": (_I32, [_I32, _P, _I64, _P, _I64, _I64, _I64, _P, _I32, _P, _I64,
                                          _I32, _I32, _I32, _I32, _P, _SZ, _U64, _P, _P]),
    "lat_test_decode_blocks_timeout": (_I32, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _I32, _I32,
                                              _P, _I32, _P, _I64, _I32, _I32, _I32, _I32, _P, _SZ,
                                              _U64, _P, _P]),
    "lat_test_capped_scores": (_I32, [_P, _I64, _F32, _F32, _P, _P]),
}


def library(path: str = LIB_PATH) -> ctypes.CDLL:
    """The loaded CUDA library (raises if it has not been built).  The first call decides which
    one that is, for sizes and launches alike."""
    global _lib, _caller
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError("lat_attn CUDA library missing at %s; build it with "
                                   "`python -m gqa_attention_lat_gb300.build`" % path)
            lib = ctypes.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            # the extension is linked to the library beside it and to no other
            ours = os.path.realpath(path) == os.path.realpath(LIB_PATH)
            _caller = (_extension() if ours else None) or _ctypes_calls(lib)
            _lib = lib
    return _lib


def _extension():
    """The C extension's module; None where it was not built for this interpreter."""
    spec = importlib.util.spec_from_file_location(__package__ + "._lat_call", CALLER_PATH)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError:
        return None
    return module if all(hasattr(module, name) for name in _status_calls()) else None


def _status_calls():
    """The names of the calls that return a status (the others are not on a hot path)."""
    return [name for name, (res, args) in _SIGNATURES.items() if res is _I32 and len(args) > 1]


def _ptr(x):
    return x if x is None or isinstance(x, int) else x.data_ptr()


_RANGES = {_I32: (-1 << 31, 1 << 31), _I64: (-1 << 63, 1 << 63), _SZ: (0, 1 << 64), _U64: (0, 1 << 64)}


def _whole(x, t):  # (ctypes would take x modulo its argument's width)
    x = operator.index(x)
    lo, hi = _RANGES[t]
    if not lo <= x < hi:
        raise OverflowError("%d exceeds its argument" % x)
    return x


def _ctypes_call(name, fn, args):
    def call(*values):
        if len(values) != len(args):
            raise TypeError("%s takes %d arguments, got %d" % (name, len(args), len(values)))
        return fn(*[_ptr(v) if t is _P else _whole(v, t) if t in _RANGES else float(v)
                    for v, t in zip(values, args)])
    return call


def _ctypes_calls(lib):
    return types.SimpleNamespace(**{name: _ctypes_call(name, getattr(lib, name), _SIGNATURES[name][1])
                                    for name in _status_calls()})


def _calls():
    """The calls that return a status, by name."""
    if _caller is None:
        library()  # raises if nothing has been built
    return _caller


def _stream(s):
    if s is None:
        torch = sys.modules.get("torch")  # CUDA cannot be up in a torch that was never imported
        if torch is None or not torch.cuda.is_initialized():
            return None
        try:  # torch.cuda.current_stream().cuda_stream without the Stream object (3 us a call)
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:  # a torch that has no such functions
            return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(st: int, where: str):
    if st != LAT_OK:
        raise LatError(st, where)


def lat_status_string(status: int) -> str:
    return library().lat_status_string(status).decode()


def lat_attn_prefill(dt, q, q_rs, k, k_rs, v, v_rs, out, out_rs, lse, batch, seq_len, kv_len,
                     n_heads, n_kv_heads, head_dim, causal, window, scale, status=None,
                     stream=None):
    _check(_calls().lat_attn_prefill(
        dt, q, q_rs, k, k_rs, v, v_rs, out, out_rs, lse, batch,
        seq_len, kv_len, n_heads, n_kv_heads, head_dim, int(bool(causal)), window, scale,
        status, _stream(stream)), "lat_attn_prefill")


def lat_attn_prefill_softcap(dt, q, q_rs, k, k_rs, v, v_rs, out, out_rs, lse, batch, seq_len,
                             kv_len, n_heads, n_kv_heads, head_dim, causal, window, scale,
                             softcap, status=None, stream=None):
    _check(_calls().lat_attn_prefill_softcap(
        dt, q, q_rs, k, k_rs, v, v_rs, out, out_rs, lse, batch,
        seq_len, kv_len, n_heads, n_kv_heads, head_dim, int(bool(causal)), window, scale,
        softcap, status, _stream(stream)), "lat_attn_prefill_softcap")


def lat_attn_decode_softcap(dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                            cache_seq_stride, kv_lens, max_kv_len, out, out_rs, lse, batch,
                            n_heads, n_kv_heads, head_dim, window, scale, softcap, workspace,
                            workspace_bytes, status=None, stream=None):
    _check(_calls().lat_attn_decode_softcap(
        dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
        cache_seq_stride, kv_lens, max_kv_len, out, out_rs, lse, batch,
        n_heads, n_kv_heads, head_dim, window, scale, softcap, workspace,
        workspace_bytes, status, _stream(stream)), "lat_attn_decode_softcap")


def lat_attn_decode_ring(dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                         cache_seq_stride, ring_capacity, kv_lens, max_kv_len, out, out_rs, lse,
                         batch, n_heads, n_kv_heads, head_dim, window, scale, workspace,
                         workspace_bytes, status=None, stream=None):
    _check(_calls().lat_attn_decode_ring(
        dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
        cache_seq_stride, ring_capacity, kv_lens, max_kv_len, out, out_rs,
        lse, batch, n_heads, n_kv_heads, head_dim, window, scale, workspace,
        workspace_bytes, status, _stream(stream)), "lat_attn_decode_ring")


def lat_kv_append_ring(dt, k_cache, v_cache, cache_rs, cache_head_stride, cache_seq_stride,
                       ring_capacity, k_new, v_new, new_rs, pos, n_new, batch, n_kv_heads,
                       head_dim, status=None, stream=None):
    _check(_calls().lat_kv_append_ring(
        dt, k_cache, v_cache, cache_rs, cache_head_stride, cache_seq_stride,
        ring_capacity, k_new, v_new, new_rs, pos, n_new, batch, n_kv_heads,
        head_dim, status, _stream(stream)), "lat_kv_append_ring")


def lat_qkv_norm_rope_append(dt, qkv, qkv_rs, q_norm_w, k_norm_w, eps, rope_base, v_unit_norm,
                             q_out, q_out_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                             cache_seq_stride, capacity, pos, n_new, batch, n_heads, n_kv_heads,
                             head_dim, status=None, stream=None):
    _check(_calls().lat_qkv_norm_rope_append(
        dt, qkv, qkv_rs, q_norm_w, k_norm_w, eps, rope_base,
        int(bool(v_unit_norm)), q_out, q_out_rs, k_cache, v_cache, cache_rs,
        cache_head_stride, cache_seq_stride, capacity, pos, n_new, batch, n_heads,
        n_kv_heads, head_dim, status, _stream(stream)), "lat_qkv_norm_rope_append")


def lat_attn_prefill_cached(dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                            cache_seq_stride, out, out_rs, lse, batch, seq_len, kv_len, n_heads,
                            n_kv_heads, head_dim, causal, window, scale, status=None,
                            stream=None):
    _check(_calls().lat_attn_prefill_cached(
        dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
        cache_seq_stride, out, out_rs, lse, batch, seq_len, kv_len, n_heads,
        n_kv_heads, head_dim, int(bool(causal)), window, scale, status, _stream(stream)),
        "lat_attn_prefill_cached")


def lat_attn_decode_workspace_size(dt, batch, n_heads, n_kv_heads, head_dim, max_kv_len) -> int:
    return library().lat_attn_decode_workspace_size(dt, batch, n_heads, n_kv_heads, head_dim,
                                                    max_kv_len)


def lat_attn_decode(dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                    cache_seq_stride, kv_lens, max_kv_len, out, out_rs, lse, batch, n_heads,
                    n_kv_heads, head_dim, window, scale, workspace, workspace_bytes,
                    status=None, stream=None):
    _check(_calls().lat_attn_decode(
        dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
        cache_seq_stride, kv_lens, max_kv_len, out, out_rs, lse, batch,
        n_heads, n_kv_heads, head_dim, window, scale, workspace, workspace_bytes,
        status, _stream(stream)), "lat_attn_decode")


def lat_attn_decode_static(dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                           cache_seq_stride, kv_lens, max_kv_len, out, out_rs, lse, batch,
                           n_heads, n_kv_heads, head_dim, window, scale, status=None,
                           stream=None):
    """lat_attn_decode with the library's own fixed device scratch (no workspace)."""
    _check(_calls().lat_attn_decode_static(
        dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
        cache_seq_stride, kv_lens, max_kv_len, out, out_rs, lse, batch,
        n_heads, n_kv_heads, head_dim, window, scale, status, _stream(stream)),
        "lat_attn_decode_static")


def lat_kv_append(dt, k_cache, v_cache, cache_rs, cache_head_stride, cache_seq_stride,
                  capacity, k_new, v_new, new_rs, pos, n_new, batch, n_kv_heads, head_dim,
                  status=None, stream=None):
    _check(_calls().lat_kv_append(
        dt, k_cache, v_cache, cache_rs, cache_head_stride, cache_seq_stride,
        capacity, k_new, v_new, new_rs, pos, n_new, batch, n_kv_heads,
        head_dim, status, _stream(stream)), "lat_kv_append")


def lat_kv_q4_row_bytes(head_dim) -> int:
    """Bytes of one 4-bit cache row (a token's K and V of one head); 0 if not built."""
    return library().lat_kv_q4_row_bytes(head_dim)


def lat_kv_append_q4(dt, cache, cache_rs, cache_head_stride, cache_seq_stride, capacity, k_new,
                     v_new, new_rs, pos, n_new, batch, n_kv_heads, head_dim, status=None,
                     stream=None):
    """Quantise new K/V rows into a 4-bit cache (cache strides in bytes)."""
    _check(_calls().lat_kv_append_q4(
        dt, cache, cache_rs, cache_head_stride, cache_seq_stride, capacity, k_new,
        v_new, new_rs, pos, n_new, batch, n_kv_heads, head_dim, status,
        _stream(stream)), "lat_kv_append_q4")


def lat_kv_expand_q4(dt, cache, cache_rs, cache_head_stride, cache_seq_stride, capacity, k_out,
                     v_out, out_rs, pos, n_rows, batch, n_kv_heads, head_dim, status=None,
                     stream=None):
    """Read rows of a 4-bit cache back as K and V rows."""
    _check(_calls().lat_kv_expand_q4(
        dt, cache, cache_rs, cache_head_stride, cache_seq_stride, capacity, k_out,
        v_out, out_rs, pos, n_rows, batch, n_kv_heads, head_dim, status,
        _stream(stream)), "lat_kv_expand_q4")


def lat_attn_decode_q4_workspace_size(dt, batch, n_heads, n_kv_heads, head_dim,
                                      max_kv_len) -> int:
    return library().lat_attn_decode_q4_workspace_size(dt, batch, n_heads, n_kv_heads, head_dim,
                                                       max_kv_len)


def lat_attn_decode_q4(dt, q, q_rs, cache, cache_rs, cache_head_stride, cache_seq_stride,
                       kv_lens, max_kv_len, out, out_rs, lse, batch, n_heads, n_kv_heads,
                       head_dim, window, scale, softcap, workspace, workspace_bytes,
                       status=None, stream=None):
    """Decode over a 4-bit cache (cache strides in bytes)."""
    _check(_calls().lat_attn_decode_q4(
        dt, q, q_rs, cache, cache_rs, cache_head_stride, cache_seq_stride,
        kv_lens, max_kv_len, out, out_rs, lse, batch, n_heads, n_kv_heads,
        head_dim, window, scale, softcap, workspace, workspace_bytes, status,
        _stream(stream)), "lat_attn_decode_q4")


def lat_kv_block_bounds(dt, k_cache, cache_rs, cache_head_stride, cache_seq_stride, capacity,
                        bounds, bounds_rs, bounds_head_stride, bounds_seq_stride, block_size,
                        pos, n_new, batch, n_kv_heads, head_dim, status=None, stream=None):
    """Bring the bounds of the blocks that hold the newly appended keys up to date."""
    _check(_calls().lat_kv_block_bounds(
        dt, k_cache, cache_rs, cache_head_stride, cache_seq_stride, capacity, bounds,
        bounds_rs, bounds_head_stride, bounds_seq_stride, block_size, pos, n_new, batch,
        n_kv_heads, head_dim, status, _stream(stream)), "lat_kv_block_bounds")


def lat_attn_select_blocks_workspace_size(batch, n_kv_heads, block_size, max_kv_len) -> int:
    return library().lat_attn_select_blocks_workspace_size(batch, n_kv_heads, block_size,
                                                           max_kv_len)


def lat_attn_select_blocks(dt, q, q_rs, bounds, bounds_rs, bounds_head_stride,
                           bounds_seq_stride, block_size, kv_lens, max_kv_len, blocks, n_sel,
                           n_first, n_last, batch, n_heads, n_kv_heads, head_dim, workspace,
                           workspace_bytes, status=None, stream=None):
    """Choose the blocks that each KV head keeps, into int32 blocks [batch, n_kv_heads, n_sel]."""
    _check(_calls().lat_attn_select_blocks(
        dt, q, q_rs, bounds, bounds_rs, bounds_head_stride, bounds_seq_stride,
        block_size, kv_lens, max_kv_len, blocks, n_sel, n_first, n_last, batch,
        n_heads, n_kv_heads, head_dim, workspace, workspace_bytes, status,
        _stream(stream)), "lat_attn_select_blocks")


def lat_attn_decode_blocks_workspace_size(dt, batch, n_heads, n_kv_heads, head_dim, block_size,
                                          n_sel) -> int:
    return library().lat_attn_decode_blocks_workspace_size(dt, batch, n_heads, n_kv_heads,
                                                           head_dim, block_size, n_sel)


def lat_attn_decode_blocks(dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                           cache_seq_stride, kv_lens, max_kv_len, block_size, blocks, n_sel,
                           out, out_rs, lse, batch, n_heads, n_kv_heads, head_dim, scale,
                           softcap, workspace, workspace_bytes, status=None, stream=None):
    """Decode over the listed blocks of the cache alone."""
    _check(_calls().lat_attn_decode_blocks(
        dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
        cache_seq_stride, kv_lens, max_kv_len, block_size, blocks, n_sel, out,
        out_rs, lse, batch, n_heads, n_kv_heads, head_dim, scale, softcap,
        workspace, workspace_bytes, status, _stream(stream)),
        "lat_attn_decode_blocks")


def lat_test_prefill_timeout(q, q_rs, k, k_rs, v, v_rs, out, out_rs, batch, seq_len, n_heads,
                             n_kv_heads, head_dim, timeout_ns, status, stream=None):
    _check(_calls().lat_test_prefill_timeout(
        q, q_rs, k, k_rs, v, v_rs, out, out_rs, batch, seq_len,
        n_heads, n_kv_heads, head_dim, timeout_ns, status, _stream(stream)),
        "lat_test_prefill_timeout")


def lat_test_decode_timeout(q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                            cache_seq_stride, kv_lens, max_kv_len, out, out_rs, batch, n_heads,
                            n_kv_heads, head_dim, workspace, workspace_bytes, timeout_ns, status,
                            stream=None):
    _check(_calls().lat_test_decode_timeout(
        q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
        cache_seq_stride, kv_lens, max_kv_len, out, out_rs, batch, n_heads,
        n_kv_heads, head_dim, workspace, workspace_bytes, timeout_ns, status,
        _stream(stream)), "lat_test_decode_timeout")


def lat_test_decode_q4_timeout(dt, q, q_rs, cache, cache_rs, cache_head_stride, cache_seq_stride,
                               kv_lens, max_kv_len, out, out_rs, batch, n_heads, n_kv_heads,
                               head_dim, workspace, workspace_bytes, timeout_ns, status,
                               stream=None):
    _check(_calls().lat_test_decode_q4_timeout(
        dt, q, q_rs, cache, cache_rs, cache_head_stride, cache_seq_stride, kv_lens, max_kv_len,
        out, out_rs, batch, n_heads, n_kv_heads, head_dim, workspace, workspace_bytes,
        timeout_ns, status, _stream(stream)), "lat_test_decode_q4_timeout")


def lat_test_decode_blocks_timeout(q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                                   cache_seq_stride, kv_lens, max_kv_len, block_size, blocks,
                                   n_sel, out, out_rs, batch, n_heads, n_kv_heads, head_dim,
                                   workspace, workspace_bytes, timeout_ns, status, stream=None):
    _check(_calls().lat_test_decode_blocks_timeout(
        q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride, cache_seq_stride, kv_lens,
        max_kv_len, block_size, blocks, n_sel, out, out_rs, batch, n_heads, n_kv_heads, head_dim,
        workspace, workspace_bytes, timeout_ns, status, _stream(stream)),
        "lat_test_decode_blocks_timeout")


def lat_test_capped_scores(raw, n, scale, softcap, out, stream=None):
    _check(_calls().lat_test_capped_scores(raw, n, scale, softcap, out,
                                            _stream(stream)), "lat_test_capped_scores")
