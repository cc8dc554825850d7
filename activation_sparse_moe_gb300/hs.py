"""ctypes binding of libhs (include/hs.h): argument marshalling only.

Every function here has the name of the C entry point it calls.  Tensors are
torch tensors already on the device; they are passed as raw pointers.  No
computation of the path happens in Python, and nothing falls back to the CPU:
if libhs.so is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes as C
import os
import re

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libhs.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "hs.h")

HS_OK = 0
HS_ERR_INVALID_ARG = -1
HS_ERR_MISALIGNED = -2
HS_ERR_UNSUPPORTED_SHAPE = -3
HS_ERR_WORKSPACE = -4
HS_ERR_CUDA = -5
HS_ERR_TIMEOUT = -6
HS_FORCE_DENSE = 0x1
HS_BATCH_EXPERT_UNION = 0x2
HS_DOWN_ROW_SCALES = 0x4
HS_PREFILL_ROW_GATHER = 0x8


class HsError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({hs_status_string(status)})")


class hs_w4(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("sb", C.c_void_p)]


class hs_expert(C.Structure):
    _fields_ = [("up", hs_w4), ("down_nm", hs_w4), ("up_offset", C.c_void_p), ("neurons", C.c_int)]


class hs_moe_layer(C.Structure):
    _fields_ = [("routed", C.POINTER(hs_expert)), ("n_routed", C.c_int), ("shared", C.POINTER(hs_expert)),
                ("hidden", C.c_int), ("top_k", C.c_int)]


class hs_decode_debug(C.Structure):
    _fields_ = [("topk_idx", C.c_void_p), ("topk_w", C.c_void_p), ("h", C.c_void_p), ("live_rows", C.c_void_p),
                ("live_groups", C.c_void_p), ("live_mask", C.c_void_p)]


class hs_prefill_debug(C.Structure):
    _fields_ = [("topk_idx", C.c_void_p), ("topk_w", C.c_void_p), ("tiles", C.c_void_p), ("work", C.c_void_p),
                ("live_mask", C.c_void_p), ("tile_live", C.c_void_p)]


class hs_kv4_cache(C.Structure):
    _fields_ = [("pool", C.c_void_p), ("n_pages", C.c_int), ("page_tokens", C.c_int), ("n_kv_heads", C.c_int),
                ("head_dim", C.c_int)]

    @property
    def ref(self):
        r = self.__dict__.get("_ref")
        if r is None:
            r = self.__dict__["_ref"] = C.byref(self)
        return r


class hs_kv8_cache(C.Structure):
    _fields_ = hs_kv4_cache._fields_
    ref = hs_kv4_cache.ref


_lib = None

_SIGS = {
    "hs_status_string": (C.c_char_p, [C.c_int]),
    "hs_device_status": (C.c_int, [C.POINTER(C.c_int)]),
    "hs_selftest_bounded_wait": (C.c_int, [C.c_longlong, C.c_void_p]),
    "hs_repack_down_nm": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_void_p,
                                    C.c_void_p]),
    "hs_pack_sb": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_void_p]),
    "hs_expert_down_sparse_workspace_size": (C.c_size_t, [C.c_int, C.c_int]),
    "hs_expert_down_sparse": (C.c_int, [C.c_void_p, C.POINTER(hs_w4), C.c_int, C.c_int, C.c_void_p, C.c_void_p,
                                        C.c_void_p, C.c_void_p, C.c_uint, C.c_void_p, C.c_size_t, C.c_void_p]),
    "hs_expert_down_sparse_noalloc": (C.c_int, [C.c_void_p, C.POINTER(hs_w4), C.c_int, C.c_int, C.c_void_p,
                                                C.c_void_p, C.c_void_p, C.c_void_p, C.c_uint, C.c_void_p]),
    "hs_moe_layer_decode_workspace_size": (C.c_size_t, [C.POINTER(hs_moe_layer), C.c_int]),
    "hs_moe_layer_decode": (C.c_int, [C.POINTER(hs_moe_layer), C.c_void_p, C.c_void_p, C.c_int, C.c_void_p,
                                      C.c_void_p, C.c_uint, C.POINTER(hs_decode_debug), C.c_void_p, C.c_size_t,
                                      C.c_void_p]),
    "hs_requant_down_rowscale": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p,
                                           C.c_void_p, C.c_void_p]),
    "hs_router_logits": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p]),
    "hs_moe_prefill_workspace_size": (C.c_size_t, [C.POINTER(hs_moe_layer), C.c_int]),
    "hs_moe_prefill": (C.c_int, [C.POINTER(hs_moe_layer), C.c_void_p, C.c_void_p, C.c_int, C.c_void_p, C.c_void_p,
                                 C.c_uint, C.POINTER(hs_prefill_debug), C.c_void_p, C.c_size_t, C.c_void_p]),
    "hs_kv4_pool_bytes": (C.c_size_t, [C.POINTER(hs_kv4_cache)]),
    "hs_kv4_plan": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_void_p,
                              C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                              C.c_void_p, C.c_void_p, C.c_void_p]),
    "hs_kv4_append": (C.c_int, [C.POINTER(hs_kv4_cache), C.c_void_p, C.c_longlong, C.c_longlong, C.c_void_p,
                                C.c_longlong, C.c_longlong, C.c_void_p, C.c_int, C.c_void_p]),
    "hs_kv4_read": (C.c_int, [C.POINTER(hs_kv4_cache), C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p,
                              C.c_void_p, C.c_void_p]),
    "hs_kv4_attention_workspace_size": (C.c_size_t, [C.POINTER(hs_kv4_cache), C.c_int, C.c_int]),
    "hs_kv4_attention": (C.c_int, [C.POINTER(hs_kv4_cache), C.c_void_p, C.c_longlong, C.c_longlong, C.c_void_p,
                                   C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int, C.c_float,
                                   C.c_int, C.c_void_p, C.c_longlong, C.c_longlong, C.c_void_p, C.c_size_t, C.c_void_p]),
    "hs_kv8_pool_bytes": (C.c_size_t, [C.POINTER(hs_kv8_cache)]),
    "hs_kv8_append": (C.c_int, [C.POINTER(hs_kv8_cache), C.c_void_p, C.c_longlong, C.c_longlong, C.c_void_p,
                                C.c_longlong, C.c_longlong, C.c_void_p, C.c_int, C.c_void_p]),
    "hs_kv8_read": (C.c_int, [C.POINTER(hs_kv8_cache), C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p,
                              C.c_void_p, C.c_void_p]),
    "hs_kv8_attention_workspace_size": (C.c_size_t, [C.POINTER(hs_kv8_cache), C.c_int, C.c_int]),
    "hs_kv8_attention": (C.c_int, [C.POINTER(hs_kv8_cache), C.c_void_p, C.c_longlong, C.c_longlong, C.c_void_p,
                                   C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int, C.c_float,
                                   C.c_int, C.c_void_p, C.c_longlong, C.c_longlong, C.c_void_p, C.c_size_t, C.c_void_p]),
    "hs_kv_pages_workspace_size": (C.c_size_t, [C.c_int]),
    "hs_kv_fork": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p,
                             C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                             C.c_void_p, C.c_void_p, C.c_void_p]),
    "hs_kv_copy_pages": (C.c_int, [C.c_void_p, C.c_int, C.c_longlong, C.c_int, C.c_void_p, C.c_void_p, C.c_int, C.c_void_p]),
    "hs_kv_release": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_void_p,
                                C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "hs_kv_compact": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p,
                                C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                C.c_size_t, C.c_void_p]),
}


def lib() -> C.CDLL:
    """The loaded libhs.so.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libhs.so is not built ({LIB_PATH}); run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            if hasattr(L, name):
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
        _lib = L
    return _lib


def declared_functions() -> list[str]:
    """Names of the functions include/hs.h declares for export (its static
    inline helpers are compiled into the caller and are not exported)."""
    txt = open(HEADER).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    txt = re.sub(r"^\s*static\s+inline\b.*$", "", txt, flags=re.M)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][\w\s\*]*?\b(hs_\w+)\s*\(", txt, flags=re.M)))


def hs_row_sb_words(out_dim: int) -> int:
    """Words per neuron row of a row-scale (scale, bias) array (the header's
    inline helper of the same name): one per 64 outputs, padded to 16 bytes."""
    return ((out_dim // 64) + 3) & ~3


def _p(t) -> int | None:
    """Raw device pointer of a tensor (None for None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, st: int):
    if st != HS_OK:
        raise HsError(fn, st)


def hs_status_string(status: int) -> str:
    return lib().hs_status_string(status).decode()


def hs_device_status() -> int:
    v = C.c_int(0)
    _check("hs_device_status", lib().hs_device_status(C.byref(v)))
    return v.value


def hs_selftest_bounded_wait(limit_cycles, stream=None):
    _check("hs_selftest_bounded_wait", lib().hs_selftest_bounded_wait(int(limit_cycles), _stream(stream)))


def hs_repack_down_nm(codes_om, scale_om, bias_om, out_dim, neurons, codes_nm, sb_nm, stream=None):
    _check("hs_repack_down_nm", lib().hs_repack_down_nm(_p(codes_om), _p(scale_om), _p(bias_om), out_dim, neurons,
                                                        _p(codes_nm), _p(sb_nm), _stream(stream)))


def hs_pack_sb(scale, bias, rows, groups, sb, stream=None):
    _check("hs_pack_sb", lib().hs_pack_sb(_p(scale), _p(bias), rows, groups, _p(sb), _stream(stream)))


def hs_expert_down_sparse_workspace_size(neurons, out_dim) -> int:
    return lib().hs_expert_down_sparse_workspace_size(neurons, out_dim)


def hs_expert_down_sparse(h, down_codes, down_sb, neurons, out_dim, y_bf16, y_f32=None, live_count=None, flags=0,
                          workspace=None, workspace_bytes=None, stream=None, live_idx=None):
    """One expert's sparse down projection.  The workspace must be zero-filled
    before its first use (the call leaves it so)."""
    w = hs_w4(_p(down_codes), _p(down_sb))
    nb = workspace_bytes if workspace_bytes is not None else (workspace.numel() * workspace.element_size()
                                                              if workspace is not None else 0)
    _check("hs_expert_down_sparse", lib().hs_expert_down_sparse(
        _p(h), C.byref(w), neurons, out_dim, _p(y_bf16), _p(y_f32), _p(live_idx), _p(live_count), flags,
        _p(workspace), nb, _stream(stream)))


def hs_expert_down_sparse_noalloc(h, down_codes, down_sb, neurons, out_dim, y_bf16, y_f32=None, live_count=None,
                                  flags=0, stream=None, live_idx=None):
    """hs_expert_down_sparse with the library's built-in scratch (no workspace)."""
    w = hs_w4(_p(down_codes), _p(down_sb))
    _check("hs_expert_down_sparse_noalloc", lib().hs_expert_down_sparse_noalloc(
        _p(h), C.byref(w), neurons, out_dim, _p(y_bf16), _p(y_f32), _p(live_idx), _p(live_count), flags,
        _stream(stream)))


def make_expert(up_codes, up_sb, down_codes, down_sb, offset, neurons) -> hs_expert:
    return hs_expert(hs_w4(_p(up_codes), _p(up_sb)), hs_w4(_p(down_codes), _p(down_sb)), _p(offset), neurons)


class Layer:
    """Host descriptor of one MoE layer (hs_moe_layer) built from device tensors.

    routed: list of hs_expert; shared: hs_expert or None.  Keeps the ctypes
    arrays alive for as long as the descriptor is used."""

    def __init__(self, routed: list, shared, hidden: int, top_k: int):
        self._routed = (hs_expert * len(routed))(*routed)
        self._shared = shared
        self.c = hs_moe_layer(self._routed, len(routed),
                              C.pointer(shared) if shared is not None else None, hidden, top_k)

    @property
    def ref(self):
        return C.byref(self.c)


def hs_moe_layer_decode_workspace_size(layer: Layer, batch: int) -> int:
    return lib().hs_moe_layer_decode_workspace_size(layer.ref, batch)


def hs_moe_layer_decode(layer: Layer, x_bf16, logits, batch, y_bf16, y_f32=None, flags=0, debug=None,
                        workspace=None, workspace_bytes=None, stream=None):
    nb = workspace_bytes if workspace_bytes is not None else (workspace.numel() * workspace.element_size()
                                                              if workspace is not None else 0)
    dbg = None
    if debug is not None:
        dbg = C.byref(hs_decode_debug(_p(debug.get("topk_idx")), _p(debug.get("topk_w")), _p(debug.get("h")),
                                      _p(debug.get("live_rows")), _p(debug.get("live_groups")),
                                      _p(debug.get("live_mask"))))
    _check("hs_moe_layer_decode", lib().hs_moe_layer_decode(
        layer.ref, _p(x_bf16), _p(logits), batch, _p(y_bf16), _p(y_f32), flags, dbg, _p(workspace), nb,
        _stream(stream)))


def hs_requant_down_rowscale(codes_om, scale_om, bias_om, out_dim, neurons, codes_nm, sb_row, stream=None):
    _check("hs_requant_down_rowscale", lib().hs_requant_down_rowscale(
        _p(codes_om), _p(scale_om), _p(bias_om), out_dim, neurons, _p(codes_nm), _p(sb_row), _stream(stream)))


def hs_router_logits(x_bf16, w_router, batch, hidden, n_experts, logits, stream=None):
    _check("hs_router_logits", lib().hs_router_logits(_p(x_bf16), _p(w_router), batch, hidden, n_experts,
                                                      _p(logits), _stream(stream)))


def hs_moe_prefill_workspace_size(layer: Layer, tokens: int) -> int:
    return lib().hs_moe_prefill_workspace_size(layer.ref, tokens)


def hs_moe_prefill(layer: Layer, x_bf16, logits, tokens, y_bf16, y_f32=None, flags=0, debug=None, workspace=None,
                   workspace_bytes=None, stream=None):
    nb = workspace_bytes if workspace_bytes is not None else (workspace.numel() * workspace.element_size()
                                                              if workspace is not None else 0)
    dbg = None
    if debug is not None:
        dbg = C.byref(hs_prefill_debug(_p(debug.get("topk_idx")), _p(debug.get("topk_w")), _p(debug.get("tiles")),
                                       _p(debug.get("work")), _p(debug.get("live_mask")),
                                       _p(debug.get("tile_live"))))
    _check("hs_moe_prefill", lib().hs_moe_prefill(
        layer.ref, _p(x_bf16), _p(logits), tokens, _p(y_bf16), _p(y_f32), flags, dbg, _p(workspace), nb,
        _stream(stream)))


def make_kv4_cache(pool, n_pages, page_tokens, n_kv_heads, head_dim) -> hs_kv4_cache:
    """Descriptor of a 4-bit key/value cache; pool is a device tensor (or
    address, or None where only sizes are asked for) that the caller keeps."""
    return hs_kv4_cache(_p(pool), n_pages, page_tokens, n_kv_heads, head_dim)


def hs_kv4_pool_bytes(cache: hs_kv4_cache) -> int:
    return lib().hs_kv4_pool_bytes(cache.ref)


# The key/value cache's calls are made for every layer of every token, so their
# marshalling is kept short (as called they take as long as the smallest steps do
# on the GPU): pointers and strides straight from the tensors, and one look at
# what the pointers would not tell the library: shapes against the cache and the
# sizes, the slots' type, rows that do not follow one another.
_current = None   # torch's own lookups of the current device and its raw stream
_i64 = None       # torch.int64
_i32 = _b16 = _f32 = None  # and its int32, bfloat16 and float32


def _kv4_stream(stream):
    global _current
    if stream is None:
        if _current is None:
            import torch
            torch.cuda.init()
            _current = (torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
        return _current[1](_current[0]())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _kv4_refuse(fn):
    """The first call of a process looks at the tensors' types before they are known: True to look again."""
    global _i64, _i32, _b16, _f32
    if _i64 is not None:
        raise HsError(fn, HS_ERR_INVALID_ARG)
    import torch
    _i64, _i32, _b16, _f32 = torch.int64, torch.int32, torch.bfloat16, torch.float32
    return True


def hs_kv4_plan(cached_len, new_len, n_seqs, page_tokens, n_pages, table_in, table_width, ring, counters_in,
                max_tokens, table_out, seq_len, q_start, slot, position, counters_out, short, stream=None):
    """Tensors of the header's types and sizes, each contiguous; position may be None."""
    if not (table_in.is_contiguous() and table_out.is_contiguous() and slot.dtype is _i64):
        if _kv4_refuse("hs_kv4_plan"):
            return hs_kv4_plan(cached_len, new_len, n_seqs, page_tokens, n_pages, table_in, table_width, ring, counters_in, max_tokens,
                               table_out, seq_len, q_start, slot, position, counters_out, short, stream)
    st = (_lib or lib()).hs_kv4_plan(
        cached_len.data_ptr(), new_len.data_ptr(), n_seqs, page_tokens, n_pages, table_in.data_ptr(), table_width,
        ring.data_ptr(), counters_in.data_ptr(), max_tokens, table_out.data_ptr(), seq_len.data_ptr(),
        q_start.data_ptr(), slot.data_ptr(), None if position is None else position.data_ptr(), counters_out.data_ptr(),
        short.data_ptr(), _current[1](_current[0]()) if stream is None and _current else _kv4_stream(stream))
    if st:
        raise HsError("hs_kv4_plan", st)


def hs_kv4_append(cache: hs_kv4_cache, k, v, slots, n_tokens, stream=None):
    """k, v: bf16 [tokens][kv heads][head_dim], any token and head strides;
    slots: int64, contiguous; n_tokens of each at least."""
    (kt, kh, kc), (vt, vh, vc), shape = k.stride(), v.stride(), k.shape
    rows, heads, dim = shape
    if (kc != 1 or vc != 1 or dim != cache.head_dim or heads != cache.n_kv_heads or rows < n_tokens or v.shape != shape
            or slots.dtype is not _i64 or not slots.is_contiguous() or slots.numel() < n_tokens):
        if _kv4_refuse("hs_kv4_append"):
            return hs_kv4_append(cache, k, v, slots, n_tokens, stream)
    st = (_lib or lib()).hs_kv4_append(cache, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, slots.data_ptr(), n_tokens,
                                       _current[1](_current[0]()) if stream is None and _current else _kv4_stream(stream))
    if st:
        raise HsError("hs_kv4_append", st)


def hs_kv4_read(cache: hs_kv4_cache, slots, n_tokens, k_bf16=None, v_bf16=None, k_f32=None, v_f32=None, stream=None):
    """slots: int64, contiguous; outputs contiguous, n_tokens rows of [kv heads][head_dim] at least."""
    n = n_tokens * cache.n_kv_heads * cache.head_dim
    if (slots.dtype is not _i64 or not slots.is_contiguous() or slots.numel() < n_tokens
            or (k_bf16 is not None and (k_bf16.numel() < n or not k_bf16.is_contiguous()))
            or (v_bf16 is not None and (v_bf16.numel() < n or not v_bf16.is_contiguous()))
            or (k_f32 is not None and (k_f32.numel() < n or not k_f32.is_contiguous()))
            or (v_f32 is not None and (v_f32.numel() < n or not v_f32.is_contiguous()))):
        if _kv4_refuse("hs_kv4_read"):
            return hs_kv4_read(cache, slots, n_tokens, k_bf16, v_bf16, k_f32, v_f32, stream)
    st = (_lib or lib()).hs_kv4_read(
        cache, slots.data_ptr(), n_tokens, k_bf16 if k_bf16 is None else k_bf16.data_ptr(),
        v_bf16 if v_bf16 is None else v_bf16.data_ptr(), k_f32 if k_f32 is None else k_f32.data_ptr(),
        v_f32 if v_f32 is None else v_f32.data_ptr(),
        _current[1](_current[0]()) if stream is None and _current else _kv4_stream(stream))
    if st:
        raise HsError("hs_kv4_read", st)


def hs_kv4_attention_workspace_size(cache: hs_kv4_cache, n_seqs, n_q_heads) -> int:
    return lib().hs_kv4_attention_workspace_size(cache.ref, n_seqs, n_q_heads)


def hs_kv4_attention(cache: hs_kv4_cache, q, q_start, seq_len, table, n_seqs, max_new, scale, window, out,
                     workspace=None, workspace_bytes=None, stream=None):
    """q, out: bf16 [tokens][query heads][head_dim], any token and head
    strides; table: int32 [n_seqs][table_width] contiguous; q_start and seq_len:
    int32, contiguous, n_seqs + 1 and n_seqs at least."""
    (qt, qh, qc), (ot, oh, oc), shape, (rows, width) = q.stride(), out.stride(), q.shape, table.shape
    tokens, heads, dim = shape
    if (qc != 1 or oc != 1 or dim != cache.head_dim or out.shape != shape or rows < n_seqs or not table.is_contiguous()
            or q_start.numel() <= n_seqs or seq_len.numel() < n_seqs):
        raise HsError("hs_kv4_attention", HS_ERR_INVALID_ARG)
    if workspace is None:
        ws, nb = None, 0
    else:
        ws, nb = workspace.data_ptr(), workspace.nbytes if workspace_bytes is None else workspace_bytes
    st = (_lib or lib()).hs_kv4_attention(
        cache, q.data_ptr(), qt, qh, q_start.data_ptr(), seq_len.data_ptr(), table.data_ptr(), width,
        n_seqs, tokens, heads, max_new, scale, window, out.data_ptr(), ot, oh, ws, nb,
        _current[1](_current[0]()) if stream is None and _current else _kv4_stream(stream))
    if st:
        raise HsError("hs_kv4_attention", st)


def make_kv8_cache(pool, n_pages, page_tokens, n_kv_heads, head_dim) -> hs_kv8_cache:
    """Descriptor of an 8-bit key/value cache, as make_kv4_cache."""
    return hs_kv8_cache(_p(pool), n_pages, page_tokens, n_kv_heads, head_dim)


def hs_kv8_pool_bytes(cache: hs_kv8_cache) -> int:
    return lib().hs_kv8_pool_bytes(cache.ref)


def hs_kv8_append(cache: hs_kv8_cache, k, v, slots, n_tokens, stream=None):
    """As hs_kv4_append; the tokens of a block of 16 next to one another."""
    (kt, kh, kc), (vt, vh, vc), shape = k.stride(), v.stride(), k.shape
    rows, heads, dim = shape
    if (kc != 1 or vc != 1 or dim != cache.head_dim or heads != cache.n_kv_heads or rows < n_tokens or v.shape != shape
            or slots.dtype is not _i64 or not slots.is_contiguous() or slots.numel() < n_tokens or k.dtype is not _b16
            or v.dtype is not _b16):
        if _kv4_refuse("hs_kv8_append"):
            return hs_kv8_append(cache, k, v, slots, n_tokens, stream)
    st = (_lib or lib()).hs_kv8_append(cache, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, slots.data_ptr(), n_tokens,
                                       _current[1](_current[0]()) if stream is None and _current else _kv4_stream(stream))
    if st:
        raise HsError("hs_kv8_append", st)


def hs_kv8_read(cache: hs_kv8_cache, slots, n_tokens, k_bf16=None, v_bf16=None, k_f32=None, v_f32=None, stream=None):
    """As hs_kv4_read; outputs of the types that their names say."""
    n = n_tokens * cache.n_kv_heads * cache.head_dim
    if (slots.dtype is not _i64 or not slots.is_contiguous() or slots.numel() < n_tokens
            or (k_bf16 is not None and (k_bf16.numel() < n or k_bf16.dtype is not _b16 or not k_bf16.is_contiguous()))
            or (v_bf16 is not None and (v_bf16.numel() < n or v_bf16.dtype is not _b16 or not v_bf16.is_contiguous()))
            or (k_f32 is not None and (k_f32.numel() < n or k_f32.dtype is not _f32 or not k_f32.is_contiguous()))
            or (v_f32 is not None and (v_f32.numel() < n or v_f32.dtype is not _f32 or not v_f32.is_contiguous()))):
        if _kv4_refuse("hs_kv8_read"):
            return hs_kv8_read(cache, slots, n_tokens, k_bf16, v_bf16, k_f32, v_f32, stream)
    st = (_lib or lib()).hs_kv8_read(
        cache, slots.data_ptr(), n_tokens, k_bf16 if k_bf16 is None else k_bf16.data_ptr(),
        v_bf16 if v_bf16 is None else v_bf16.data_ptr(), k_f32 if k_f32 is None else k_f32.data_ptr(),
        v_f32 if v_f32 is None else v_f32.data_ptr(),
        _current[1](_current[0]()) if stream is None and _current else _kv4_stream(stream))
    if st:
        raise HsError("hs_kv8_read", st)


def hs_kv8_attention_workspace_size(cache: hs_kv8_cache, n_seqs, n_q_heads) -> int:
    return lib().hs_kv8_attention_workspace_size(cache.ref, n_seqs, n_q_heads)


def hs_kv8_attention(cache: hs_kv8_cache, q, q_start, seq_len, table, n_seqs, max_new, scale, window, out,
                     workspace=None, workspace_bytes=None, stream=None):
    """As hs_kv4_attention."""
    (qt, qh, qc), (ot, oh, oc), shape, (rows, width) = q.stride(), out.stride(), q.shape, table.shape
    tokens, heads, dim = shape
    if (qc != 1 or oc != 1 or dim != cache.head_dim or out.shape != shape or rows < n_seqs or not table.is_contiguous()
            or q_start.numel() <= n_seqs or seq_len.numel() < n_seqs or q.dtype is not _b16 or out.dtype is not _b16
            or not (q_start.dtype is seq_len.dtype is table.dtype is _i32 and q_start.is_contiguous() and seq_len.is_contiguous())):
        if _kv4_refuse("hs_kv8_attention"):
            return hs_kv8_attention(cache, q, q_start, seq_len, table, n_seqs, max_new, scale, window, out, workspace, workspace_bytes,
                                    stream)
    if workspace is None:
        ws, nb = None, 0
    else:
        ws, nb = workspace.data_ptr(), workspace.nbytes if workspace_bytes is None else workspace_bytes
    st = (_lib or lib()).hs_kv8_attention(
        cache, q.data_ptr(), qt, qh, q_start.data_ptr(), seq_len.data_ptr(), table.data_ptr(), width,
        n_seqs, tokens, heads, max_new, scale, window, out.data_ptr(), ot, oh, ws, nb,
        _current[1](_current[0]()) if stream is None and _current else _kv4_stream(stream))
    if st:
        raise HsError("hs_kv8_attention", st)


# Pages shared, copied, given back and moved.  The pointers do not tell the
# library how long the tensors behind them are, nor their types, so each is
# looked at here, in one expression: a loop over them costs as much as the call.
class make_kv_pools:
    """The pools of a model's layers for hs_kv_copy_pages: device tensors, which
    are kept, all of one size."""

    def __init__(self, pools):
        pools = list(pools)
        if not pools or any(not p.is_contiguous() or p.nbytes != pools[0].nbytes for p in pools):
            raise HsError("make_kv_pools", HS_ERR_INVALID_ARG)
        self.tensors, self.nbytes, self.n = pools, pools[0].nbytes, len(pools)
        self.c = (C.c_void_p * len(pools))(*[p.data_ptr() for p in pools])


def hs_kv_pages_workspace_size(n_pages) -> int:
    return lib().hs_kv_pages_workspace_size(n_pages)


def hs_kv_fork(parent, child, length, n_forks, cached_len, n_seqs, page_tokens, n_pages, table_in, table_width, shared, ring,
               counters_in, table_out, len_out, copy_src, copy_dst, counters_out, short, stream=None):
    """Tensors of the header's types and sizes, each contiguous; table_out may be table_in."""
    cells = n_seqs * table_width
    if not (parent.dtype is child.dtype is length.dtype is cached_len.dtype is table_in.dtype is shared.dtype is ring.dtype
            is table_out.dtype is len_out.dtype is copy_src.dtype is copy_dst.dtype is short.dtype is _i32
            and counters_in.dtype is counters_out.dtype is _i64
            and parent.is_contiguous() and child.is_contiguous() and length.is_contiguous() and cached_len.is_contiguous()
            and table_in.is_contiguous() and shared.is_contiguous() and ring.is_contiguous() and counters_in.is_contiguous()
            and table_out.is_contiguous() and len_out.is_contiguous() and copy_src.is_contiguous() and copy_dst.is_contiguous()
            and counters_out.is_contiguous()
            and parent.numel() >= n_forks <= child.numel() and length.numel() >= n_forks <= copy_src.numel()
            and copy_dst.numel() >= n_forks and cached_len.numel() >= n_seqs <= len_out.numel() and table_in.numel() >= cells <= table_out.numel()
            and shared.numel() >= n_pages <= ring.numel() and counters_in.numel() >= 2 <= counters_out.numel() and short.numel()):
        if _kv4_refuse("hs_kv_fork"):
            return hs_kv_fork(parent, child, length, n_forks, cached_len, n_seqs, page_tokens, n_pages, table_in, table_width, shared,
                              ring, counters_in, table_out, len_out, copy_src, copy_dst, counters_out, short, stream)
    st = (_lib or lib()).hs_kv_fork(
        parent.data_ptr(), child.data_ptr(), length.data_ptr(), n_forks, cached_len.data_ptr(), n_seqs, page_tokens, n_pages,
        table_in.data_ptr(), table_width, shared.data_ptr(), ring.data_ptr(), counters_in.data_ptr(), table_out.data_ptr(),
        len_out.data_ptr(), copy_src.data_ptr(), copy_dst.data_ptr(), counters_out.data_ptr(), short.data_ptr(),
        _current[1](_current[0]()) if stream is None and _current else _kv4_stream(stream))
    if st:
        raise HsError("hs_kv_fork", st)


def hs_kv_copy_pages(pools, page_bytes, n_pages, src, dst, n_copies, stream=None):
    """pools: make_kv_pools of the layers' pools, or the tensors themselves."""
    if not isinstance(pools, make_kv_pools):
        pools = make_kv_pools(pools)
    if not (src.dtype is dst.dtype is _i32 and src.is_contiguous() and dst.is_contiguous() and src.numel() >= n_copies <= dst.numel()
            and pools.nbytes >= n_pages * page_bytes):
        if _kv4_refuse("hs_kv_copy_pages"):
            return hs_kv_copy_pages(pools, page_bytes, n_pages, src, dst, n_copies, stream)
    st = (_lib or lib()).hs_kv_copy_pages(pools.c, pools.n, page_bytes, n_pages, src.data_ptr(), dst.data_ptr(), n_copies,
                                          _current[1](_current[0]()) if stream is None and _current else _kv4_stream(stream))
    if st:
        raise HsError("hs_kv_copy_pages", st)


def hs_kv_release(cached_len, keep_len, n_seqs, page_tokens, n_pages, table_in, table_width, shared, ring, counters_in, table_out,
                  len_out, counters_out, workspace=None, workspace_bytes=None, stream=None):
    """Tensors of the header's types and sizes, each contiguous; table_out may be table_in."""
    cells = n_seqs * table_width
    if not (cached_len.dtype is keep_len.dtype is table_in.dtype is shared.dtype is ring.dtype is table_out.dtype is len_out.dtype is _i32
            and counters_in.dtype is counters_out.dtype is _i64
            and cached_len.is_contiguous() and keep_len.is_contiguous() and table_in.is_contiguous() and shared.is_contiguous()
            and ring.is_contiguous() and counters_in.is_contiguous() and table_out.is_contiguous() and len_out.is_contiguous()
            and counters_out.is_contiguous()
            and cached_len.numel() >= n_seqs <= keep_len.numel() and len_out.numel() >= n_seqs
            and table_in.numel() >= cells <= table_out.numel() and shared.numel() >= n_pages <= ring.numel()
            and counters_in.numel() >= 2 <= counters_out.numel()):
        if _kv4_refuse("hs_kv_release"):
            return hs_kv_release(cached_len, keep_len, n_seqs, page_tokens, n_pages, table_in, table_width, shared, ring, counters_in,
                                 table_out, len_out, counters_out, workspace, workspace_bytes, stream)
    if workspace is None:
        ws, nb = None, 0
    else:
        ws, nb = workspace.data_ptr(), workspace.nbytes if workspace_bytes is None else workspace_bytes
    st = (_lib or lib()).hs_kv_release(
        cached_len.data_ptr(), keep_len.data_ptr(), n_seqs, page_tokens, n_pages, table_in.data_ptr(), table_width, shared.data_ptr(),
        ring.data_ptr(), counters_in.data_ptr(), table_out.data_ptr(), len_out.data_ptr(), counters_out.data_ptr(), ws, nb,
        _current[1](_current[0]()) if stream is None and _current else _kv4_stream(stream))
    if st:
        raise HsError("hs_kv_release", st)


def hs_kv_compact(cached_len, n_seqs, page_tokens, n_pages, table_in, table_width, shared_in, ring, counters_in, max_copies, table_out,
                  shared_out, copy_src, copy_dst, counters_out, short, workspace=None, workspace_bytes=None, stream=None):
    """Tensors of the header's types and sizes, each contiguous; table_out and shared_out may be the inputs."""
    cells = n_seqs * table_width
    if not (cached_len.dtype is table_in.dtype is shared_in.dtype is ring.dtype is table_out.dtype is shared_out.dtype is copy_src.dtype
            is copy_dst.dtype is short.dtype is _i32 and counters_in.dtype is counters_out.dtype is _i64
            and cached_len.is_contiguous() and table_in.is_contiguous() and shared_in.is_contiguous() and ring.is_contiguous()
            and counters_in.is_contiguous() and table_out.is_contiguous() and shared_out.is_contiguous() and copy_src.is_contiguous()
            and copy_dst.is_contiguous() and counters_out.is_contiguous()
            and cached_len.numel() >= n_seqs and table_in.numel() >= cells <= table_out.numel()
            and shared_in.numel() >= n_pages <= shared_out.numel() and ring.numel() >= n_pages
            and copy_src.numel() >= max_copies <= copy_dst.numel() and counters_in.numel() >= 2 <= counters_out.numel() and short.numel()):
        if _kv4_refuse("hs_kv_compact"):
            return hs_kv_compact(cached_len, n_seqs, page_tokens, n_pages, table_in, table_width, shared_in, ring, counters_in, max_copies,
                                 table_out, shared_out, copy_src, copy_dst, counters_out, short, workspace, workspace_bytes, stream)
    if workspace is None:
        ws, nb = None, 0
    else:
        ws, nb = workspace.data_ptr(), workspace.nbytes if workspace_bytes is None else workspace_bytes
    st = (_lib or lib()).hs_kv_compact(
        cached_len.data_ptr(), n_seqs, page_tokens, n_pages, table_in.data_ptr(), table_width, shared_in.data_ptr(), ring.data_ptr(),
        counters_in.data_ptr(), max_copies, table_out.data_ptr(), shared_out.data_ptr(), copy_src.data_ptr(), copy_dst.data_ptr(),
        counters_out.data_ptr(), short.data_ptr(), ws, nb,
        _current[1](_current[0]()) if stream is None and _current else _kv4_stream(stream))
    if st:
        raise HsError("hs_kv_compact", st)
