"""Thin ctypes binding of libcacheblend.so: the C entry points under the same names,
taking torch tensors (device memory) and marshalling them to raw pointers.  No arithmetic
of the method happens here; every step runs in the library's CUDA kernels.  Raises
CBError on any non-zero status.  Fails loudly when the library has not been built."""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Sequence

from . import build as _build

CB_OK = 0
CB_F32, CB_BF16 = 0, 1
CB_DEV_KV, CB_DEV_K = 0, 1
CB_LAYER_PRECHECK, CB_LAYER_CHECK, CB_LAYER_STEADY, CB_LAYER_GRADUAL = 0, 1, 2, 3
STATUS_NAMES = {0: "CB_OK", 1: "CB_ERR_INVALID_ARG", 2: "CB_ERR_SHAPE", 3: "CB_ERR_DTYPE",
                4: "CB_ERR_WORKSPACE", 5: "CB_ERR_NONFINITE", 6: "CB_ERR_CUDA", 7: "CB_ERR_TIMEOUT",
                8: "CB_ERR_UNSUPPORTED", 9: "CB_ERR_DEVICE", 10: "CB_ERR_IO"}


class CBError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class cb_layer_opts(C.Structure):
    _fields_ = [("forced_mask", C.c_void_p), ("n_forced", C.c_int32), ("kv_ready", C.c_void_p),
                ("recompute_kv", C.c_int32), ("recompute_from", C.c_int32), ("x_rows", C.c_void_p),
                ("n_x_rows", C.c_int64), ("aux_stream", C.c_void_p), ("aux_fork", C.c_void_p),
                ("aux_join", C.c_void_p), ("x_out_ssq", C.c_void_p), ("x_out_ssq_parts_host", C.POINTER(C.c_int32)),
                ("x_in_ssq", C.c_void_p), ("x_in_ssq_parts", C.c_int32)]


class cb_dims(C.Structure):
    _fields_ = [("d_model", C.c_int32), ("n_heads", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("d_ff", C.c_int32), ("vocab", C.c_int32),
                ("rope_base", C.c_double), ("rms_eps", C.c_float), ("dtype", C.c_int32)]


class cb_layer_w(C.Structure):
    _fields_ = [("attn_norm", C.c_void_p), ("wqkv", C.c_void_p), ("wo", C.c_void_p),
                ("ffn_norm", C.c_void_p), ("w_gate_up", C.c_void_p), ("w_down", C.c_void_p)]


class cb_prof_record(C.Structure):
    _fields_ = [("kind", C.c_int32), ("aux", C.c_int32), ("m", C.c_int64), ("n", C.c_int64), ("k", C.c_int64),
                ("flops", C.c_double), ("bytes", C.c_double), ("ms", C.c_float), ("span_ms", C.c_float)]


class cb_kv8_cache(C.Structure):
    """A layer's 8-bit KV cache (see cacheblend.h); made by kv8_cache(), which also keeps the
    tensors alive and their head count and width for the checks."""
    _fields_ = [("k_codes", C.c_void_p), ("v_codes", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("capacity", C.c_int64), ("n_seq", C.c_int32), ("block", C.c_int32)]


class cb_logit_rules(C.Structure):
    """The rules of cb_logits_process (see cacheblend.h); made by logit_rules()."""
    _fields_ = [("history", C.c_void_p), ("history_len", C.c_void_p), ("prompt_len", C.c_void_p),
                ("repetition", C.c_void_p), ("presence", C.c_void_p), ("frequency", C.c_void_p),
                ("bias_id", C.c_void_p), ("bias", C.c_void_p), ("mask", C.c_void_p), ("history_ld", C.c_int64),
                ("mask_ld", C.c_int64), ("n_bias", C.c_int32)]


PROF_KINDS = {0: "rope_shift", 1: "copy_rows", 2: "rmsnorm", 3: "gemm", 4: "attention", 5: "deviation",
              6: "topk", 7: "index", 8: "lmhead_gemv", 9: "argmax", 10: "rope_table", 11: "kv_quantize", 12: "kv8_append",
              13: "kv8_read", 14: "kv8_attention", 15: "kv8_evict", 16: "logits"}

_P = C.c_void_p
_I32 = C.c_int32
_I64 = C.c_int64
_SZ = C.c_size_t
_PROTOS = {
    "cb_status_string": (C.c_char_p, [C.c_int]),
    "cb_last_error_message": (C.c_char_p, []),
    "cb_last_cuda_error": (C.c_char_p, []),
    "cb_sync": (C.c_int, [_P, C.c_double]),
    "cb_workspace_bytes": (C.c_int, [C.POINTER(cb_dims), _I64, _I64, C.POINTER(_SZ)]),
    "cb_hkvd_budget": (_I64, [_I64, C.c_double, _I64]),
    "cb_gradual_ratio": (C.c_double, [C.c_double, _I32, _I32, C.c_double]),
    "cb_load_controller_ratio": (C.c_double, [C.c_double, C.c_double, C.c_double]),
    "cb_rope_table": (C.c_int, [_P, _I32, _I32, C.c_double, _P]),
    "cb_shutdown": (None, []),
    "cb_rope_shift": (C.c_int, [_P, _P, _P, _P, _P, _I64, _P, _I64, C.POINTER(cb_dims), _P, _I32, _P]),
    "cb_kv_deviation_topk": (C.c_int, [_P, _P, _I64, _P, _P, _I64, _P, _P, _I32, _I32, _I32, C.POINTER(cb_dims),
                                       _P, _P, _P, _SZ, _P]),
    "cb_kv_deviation_topk_noalloc": (C.c_int, [_P, _P, _I64, _P, _P, _I64, _P, _P, _I32, _I32, _I32,
                                               C.POINTER(cb_dims), _P, _P, _P]),
    "cb_topk_from_scores": (C.c_int, [_P, _P, _I32, _I32, _P, _P, _SZ, _P]),
    "cb_gather_rows": (C.c_int, [_P, _P, _I64, _P, _I64, _I64, _P]),
    "cb_scatter_kv": (C.c_int, [_P, _P, _I64, _P, _P, _I64, _P, _P, _I64, C.POINTER(cb_dims), _P]),
    "cb_selective_qkv": (C.c_int, [_P, _I64, _P, _P, _I32, C.POINTER(cb_dims), C.POINTER(cb_layer_w), _P, _I32,
                                   _P, _P, _P, _P, _SZ, _P]),
    "cb_partial_attention": (C.c_int, [_P, _P, _I32, _P, _P, _I64, C.POINTER(cb_dims), _P, _P, _SZ, _P]),
    "cb_o_proj_ffn": (C.c_int, [_P, _P, _I32, C.POINTER(cb_dims), C.POINTER(cb_layer_w), _P, _P, _SZ, _P]),
    "cb_blend_layer": (C.c_int, [C.POINTER(cb_dims), C.POINTER(cb_layer_w), _I32, _P, _P, _I32, _I64, _I64,
                                 _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, C.POINTER(_I32), _P,
                                 C.POINTER(cb_layer_opts), _P, _SZ, _P]),
    "cb_blend_steady_batch": (C.c_int, [C.POINTER(cb_dims), C.POINTER(cb_layer_w), _I32, C.POINTER(_I32), _P, _P,
                                        _I64, _P, _P, _P, _I32, _P, _P, _SZ, _P]),
    "cb_full_prefill": (C.c_int, [C.POINTER(cb_dims), _I32, C.POINTER(cb_layer_w), _P, _P, _I32, _I32,
                                  C.POINTER(_P), C.POINTER(_P), _P, _P, _P, _I32, _P, _SZ, _P]),
    "cb_lmhead_argmax": (C.c_int, [_P, _P, _P, C.POINTER(cb_dims), _P, _P, _P, _SZ, _P]),
    "cb_linear": (C.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, _P]),
    "cb_kv_quantize": (C.c_int, [_P, _I64, _I32, _I32, _P, _P, _P, _P]),
    "cb_file_read": (C.c_int, [C.c_char_p, C.c_uint64, _P, _SZ, _I32]),
    "cb_selftest_wait": (C.c_int, [_I32, _I32, _P]),
    "cb_copy_async": (C.c_int, [_P, _P, _SZ, _P]),
    "cb_rmsnorm": (C.c_int, [_P, _P, _I64, _P, _I64, _I32, _P, C.c_float, _I32, _I32, _P]),
    "cb_io_error_message": (C.c_char_p, []),
    "cb_rope_shift_q8": (C.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _I32, _P, _I64,
                                   C.POINTER(cb_dims), _P, _I32, _P]),
    "cb_kv8_append": (C.c_int, [_P, _P, _I32, _P, _P, C.POINTER(cb_kv8_cache), C.POINTER(cb_dims), _P]),
    "cb_kv8_read": (C.c_int, [C.POINTER(cb_kv8_cache), _P, _P, _I32, C.POINTER(cb_dims), _P, _P, _P]),
    "cb_kv8_workspace_bytes": (C.c_int, [C.POINTER(cb_dims), _I32, _I64, _I32, _I32, C.POINTER(_SZ)]),
    "cb_kv8_attention": (C.c_int, [_P, _P, _I32, C.POINTER(cb_kv8_cache), C.POINTER(cb_dims), _P, _P, _P, _SZ, _P]),
    "cb_kv8_evict": (C.c_int, [C.POINTER(cb_kv8_cache), _P, _P, _I32, _I32, _I32, C.POINTER(cb_kv8_cache), _P, _P, _P,
                               C.POINTER(cb_dims), _P]),
    "cb_logits_process": (C.c_int, [_P, _I32, _I32, _I32, C.POINTER(cb_logit_rules), _P, _P, _P]),
    "cb_prefetch_layer": (C.c_int, [_P, _P, _SZ, _P, _P]),
    "cb_stream_wait": (C.c_int, [_P, _P]),
    "cb_kernel_launch_count": (_I64, []),
    "cb_profile_begin": (C.c_int, [_I32]),
    "cb_profile_begin_spans": (C.c_int, [_I32]),
    "cb_profile_end": (C.c_int, [C.POINTER(cb_prof_record), _I32, C.POINTER(_I32)]),
}

_LIB = None


def lib():
    """Load the in-tree library (never builds implicitly on the call path)."""
    global _LIB
    if _LIB is None:
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with non_prefix_kv_gb300.build.build()")
        L = C.CDLL(path)
        for name, (res, args) in _PROTOS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, st: int):
    if st != CB_OK:
        raise CBError(fn, st, lib().cb_last_error_message().decode(errors="replace"))


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def cb_last_cuda_error() -> str:
    """The last failing CUDA runtime call on this thread ("" if none)."""
    return lib().cb_last_cuda_error().decode(errors="replace")


# ---- host helpers -------------------------------------------------------------------------
def cb_hkvd_budget(n_cached: int, ratio: float, n_cand: int) -> int:
    return int(lib().cb_hkvd_budget(n_cached, ratio, n_cand))


def cb_gradual_ratio(r: float, layer: int, check_layer: int, r1_factor: float = 1.5) -> float:
    return float(lib().cb_gradual_ratio(r, layer, check_layer, r1_factor))


def cb_load_controller_ratio(r_min: float, t_load_s: float, t_prefill_s: float) -> float:
    return float(lib().cb_load_controller_ratio(r_min, t_load_s, t_prefill_s))


def cb_workspace_bytes(dims: cb_dims, n_tok: int, m_max: int) -> int:
    out = _SZ(0)
    _check("cb_workspace_bytes", lib().cb_workspace_bytes(C.byref(dims), n_tok, m_max, C.byref(out)))
    return int(out.value)


def cb_sync(stream=None, timeout_s: float = 60.0) -> None:
    _check("cb_sync", lib().cb_sync(_stream(stream), timeout_s))


def cb_shutdown() -> None:
    lib().cb_shutdown()


def _rows(t, n: Optional[int]) -> int:
    """Row count of a buffer for the index checks: given, or the tensor's first dimension."""
    if n is not None:
        return int(n)
    if t is None or isinstance(t, int):
        raise ValueError("the row count of a raw pointer must be given")
    return int(t.shape[0])


# ---- device entry points --------------------------------------------------------------------
def cb_rope_table(cos_sin, max_pos: int, head_dim: int, base: float, stream=None):
    _check("cb_rope_table", lib().cb_rope_table(_ptr(cos_sin), max_pos, head_dim, base, _stream(stream)))


def cb_rope_shift(k_dst, v_dst, k_src, v_src, src_row, delta, n_rows: int, dims: cb_dims, cos_sin,
                  max_pos: int, stream=None, n_src_rows: Optional[int] = None):
    """n_src_rows: rows of k_src/v_src (default: k_src's first dimension)."""
    _check("cb_rope_shift", lib().cb_rope_shift(_ptr(k_dst), _ptr(v_dst), _ptr(k_src), _ptr(v_src),
                                                _ptr(src_row), _rows(k_src, n_src_rows), _ptr(delta), n_rows,
                                                C.byref(dims), _ptr(cos_sin), max_pos, _stream(stream)))


def cb_kv_deviation_topk(k_new, v_new, k_ref, v_ref, new_row, ref_row, n_cand: int, k: int, dev_mode: int,
                         dims: cb_dims, scores, sel, ws, stream=None, n_new_rows: Optional[int] = None,
                         n_ref_rows: Optional[int] = None):
    """n_new_rows / n_ref_rows: rows of k_new and k_ref (default: their first dimension)."""
    _check("cb_kv_deviation_topk", lib().cb_kv_deviation_topk(
        _ptr(k_new), _ptr(v_new), _rows(k_new, n_new_rows), _ptr(k_ref), _ptr(v_ref), _rows(k_ref, n_ref_rows),
        _ptr(new_row), _ptr(ref_row), n_cand, k, dev_mode, C.byref(dims), _ptr(scores), _ptr(sel), _ptr(ws),
        _nbytes(ws), _stream(stream)))


def cb_kv_deviation_topk_noalloc(k_new, v_new, k_ref, v_ref, new_row, ref_row, n_cand: int, k: int,
                                 dev_mode: int, dims: cb_dims, scores, sel, stream=None,
                                 n_new_rows: Optional[int] = None, n_ref_rows: Optional[int] = None):
    """Same as cb_kv_deviation_topk, with the scratch in the library's fixed device array
    (for callers that cannot allocate; at most 65536 candidates; overlapping calls race)."""
    _check("cb_kv_deviation_topk_noalloc", lib().cb_kv_deviation_topk_noalloc(
        _ptr(k_new), _ptr(v_new), _rows(k_new, n_new_rows), _ptr(k_ref), _ptr(v_ref), _rows(k_ref, n_ref_rows),
        _ptr(new_row), _ptr(ref_row), n_cand, k, dev_mode, C.byref(dims), _ptr(scores), _ptr(sel),
        _stream(stream)))


def cb_topk_from_scores(scores, cand, n_cand: int, k: int, sel, ws, stream=None):
    _check("cb_topk_from_scores", lib().cb_topk_from_scores(_ptr(scores), _ptr(cand), n_cand, k, _ptr(sel),
                                                            _ptr(ws), _nbytes(ws), _stream(stream)))


def cb_gather_rows(dst, src, idx, n: int, row_bytes: int, stream=None, n_src_rows: Optional[int] = None):
    """n_src_rows: rows of src that idx may address (default: src's first dimension)."""
    _check("cb_gather_rows", lib().cb_gather_rows(_ptr(dst), _ptr(src), _rows(src, n_src_rows), _ptr(idx), n,
                                                  row_bytes, _stream(stream)))


def cb_scatter_kv(k_cache, v_cache, k_rows, v_rows, dst_idx, src_idx, n: int, dims: cb_dims, stream=None,
                  n_cache_rows: Optional[int] = None, n_src_rows: Optional[int] = None):
    _check("cb_scatter_kv", lib().cb_scatter_kv(_ptr(k_cache), _ptr(v_cache), _rows(k_cache, n_cache_rows),
                                                _ptr(k_rows), _ptr(v_rows), _rows(k_rows, n_src_rows),
                                                _ptr(dst_idx), _ptr(src_idx), n, C.byref(dims),
                                                _stream(stream)))


def cb_selective_qkv(x, rows, pos, M: int, dims: cb_dims, w: cb_layer_w, cos_sin, max_pos: int, q, k, v,
                     ws, stream=None, n_x_rows: Optional[int] = None):
    _check("cb_selective_qkv", lib().cb_selective_qkv(
        _ptr(x), _rows(x, n_x_rows), _ptr(rows), _ptr(pos), M, C.byref(dims), C.byref(w), _ptr(cos_sin), max_pos,
        _ptr(q), _ptr(k), _ptr(v), _ptr(ws), _nbytes(ws), _stream(stream)))


def cb_partial_attention(q, q_pos, M: int, k_cache, v_cache, n_kv: int, dims: cb_dims, out, ws=None,
                         stream=None):
    _check("cb_partial_attention", lib().cb_partial_attention(
        _ptr(q), _ptr(q_pos), M, _ptr(k_cache), _ptr(v_cache), n_kv, C.byref(dims), _ptr(out), _ptr(ws),
        _nbytes(ws), _stream(stream)))


def cb_o_proj_ffn(attn, x_res, M: int, dims: cb_dims, w: cb_layer_w, x_out, ws, stream=None):
    _check("cb_o_proj_ffn", lib().cb_o_proj_ffn(_ptr(attn), _ptr(x_res), M, C.byref(dims), C.byref(w),
                                                _ptr(x_out), _ptr(ws), _nbytes(ws), _stream(stream)))


def cb_blend_layer(dims: cb_dims, w: cb_layer_w, mode: int, x_in, s_in, m_in: int, n_tok: int, n_cached: int,
                   k_cache, v_cache, cos_sin, max_pos: int, k_budget: int, dev_mode: int, sel_override,
                   x_out, s_out, scores_out, ws, stream=None, kv_ready=None, forced_mask=None,
                   n_forced: int = 0, recompute_kv: bool = False, recompute_from: int = 0, x_rows=None,
                   n_x_rows: int = 0, aux=None, x_out_ssq=None, ssq_parts_out: Optional[list] = None, x_in_ssq=None,
                   x_in_ssq_parts: int = 0) -> int:
    """kv_ready: a torch.cuda.Event (or raw cudaEvent_t) the layer waits for just before it
    first touches the cached rows, or None.  forced_mask/n_forced: uncached rows anywhere
    (a uint8 device tensor over the tokens, marking the last row too), or None.
    recompute_from: PRECHECK only, recompute K/V from this row on (0: off).
    x_rows / n_x_rows: PRECHECK only, input row i is x_in[x_rows[i]] (e.g. x_in = the embedding
    table, x_rows = the token ids).
    aux: (stream, fork event, join event) for the CHECK/GRADUAL KV expansion beside the Q GEMM,
    or None.
    x_out_ssq: a float32 device buffer that receives the output rows' partial sums of squares;
    their count is stored in ssq_parts_out[0].  x_in_ssq / x_in_ssq_parts: the same from the
    call that produced x_in (lets the bf16 path with unit attention-norm gains skip the norm)."""
    m_out = _I32(0)
    opts = None
    parts = _I32(0)
    if (kv_ready is not None or forced_mask is not None or recompute_kv or recompute_from or x_rows is not None
            or aux is not None or x_out_ssq is not None or x_in_ssq is not None):
        ev = kv_ready if (kv_ready is None or isinstance(kv_ready, int)) else kv_ready.cuda_event
        ax = (None, None, None) if aux is None else (_stream(aux[0]), _event(aux[1]), _event(aux[2]))
        opts = C.byref(cb_layer_opts(_ptr(forced_mask), n_forced if forced_mask is not None else 0, ev,
                                     1 if recompute_kv else 0, int(recompute_from), _ptr(x_rows),
                                     int(n_x_rows) if x_rows is not None else 0, *ax, _ptr(x_out_ssq),
                                     C.pointer(parts) if x_out_ssq is not None else None, _ptr(x_in_ssq),
                                     int(x_in_ssq_parts) if x_in_ssq is not None else 0))
    _check("cb_blend_layer", lib().cb_blend_layer(
        C.byref(dims), C.byref(w), mode, _ptr(x_in), _ptr(s_in), m_in, n_tok, n_cached, _ptr(k_cache),
        _ptr(v_cache), _ptr(cos_sin), max_pos, k_budget, dev_mode, _ptr(sel_override), _ptr(x_out),
        _ptr(s_out), C.byref(m_out), _ptr(scores_out), opts, _ptr(ws), _nbytes(ws), _stream(stream)))
    if ssq_parts_out is not None:
        ssq_parts_out[:] = [int(parts.value)]
    return int(m_out.value)


def cb_blend_steady_batch(dims: cb_dims, w: cb_layer_w, row0: Sequence[int], x_in, s_in, n_tok: int, k_cache,
                          v_cache, cos_sin, max_pos: int, x_out, ws, stream=None):
    """One steady layer of len(row0) - 1 requests at once (request r: rows [row0[r], row0[r+1]))."""
    arr = (C.c_int32 * len(row0))(*[int(v) for v in row0])
    _check("cb_blend_steady_batch", lib().cb_blend_steady_batch(
        C.byref(dims), C.byref(w), len(row0) - 1, arr, _ptr(x_in), _ptr(s_in), n_tok, _ptr(k_cache), _ptr(v_cache),
        _ptr(cos_sin), max_pos, _ptr(x_out), _ptr(ws), _nbytes(ws), _stream(stream)))


def cb_full_prefill(dims: cb_dims, layers: Sequence[cb_layer_w], embed, tokens, n: int, pos0: int,
                    k_out: Sequence, v_out: Sequence, h_last, x_all, cos_sin, max_pos: int, ws, stream=None):
    L = len(layers)
    arr_w = (cb_layer_w * L)(*layers)
    arr_k = (C.c_void_p * L)(*[_ptr(t) for t in k_out])
    arr_v = (C.c_void_p * L)(*[_ptr(t) for t in v_out])
    _check("cb_full_prefill", lib().cb_full_prefill(
        C.byref(dims), L, arr_w, _ptr(embed), _ptr(tokens), n, pos0, arr_k, arr_v, _ptr(h_last), _ptr(x_all),
        _ptr(cos_sin), max_pos, _ptr(ws), _nbytes(ws), _stream(stream)))


def cb_lmhead_argmax(h, final_norm, w_lm, dims: cb_dims, logits, token, ws, stream=None):
    _check("cb_lmhead_argmax", lib().cb_lmhead_argmax(_ptr(h), _ptr(final_norm), _ptr(w_lm), C.byref(dims),
                                                      _ptr(logits), _ptr(token), _ptr(ws), _nbytes(ws),
                                                      _stream(stream)))


def cb_linear(x, w, y, M: int, N: int, K: int, dtype: int, stream=None):
    _check("cb_linear", lib().cb_linear(_ptr(x), _ptr(w), _ptr(y), M, N, K, dtype, _stream(stream)))


def cb_file_read(path: str, offset: int, dst, nbytes: int, n_threads: int = 8):
    """Read nbytes of the file at offset into dst (a pinned host tensor or raw pointer)."""
    st = lib().cb_file_read(path.encode(), offset, _ptr(dst), nbytes, n_threads)
    if st != CB_OK:
        raise CBError("cb_file_read", st, lib().cb_io_error_message().decode(errors="replace"))


def cb_rmsnorm(out, x, rows, n: int, d: int, gain, eps: float, dtype_in: int, dtype_out: int, stream=None,
               n_x_rows: Optional[int] = None):
    _check("cb_rmsnorm", lib().cb_rmsnorm(_ptr(out), _ptr(x), _rows(x, n_x_rows), _ptr(rows), n, d, _ptr(gain),
                                          eps, dtype_in, dtype_out, _stream(stream)))


def cb_copy_async(dst, src, nbytes: int, stream=None):
    _check("cb_copy_async", lib().cb_copy_async(_ptr(dst), _ptr(src), nbytes, _stream(stream)))


def cb_selftest_wait(max_polls: int, arrive: bool, stream=None):
    _check("cb_selftest_wait", lib().cb_selftest_wait(max_polls, 1 if arrive else 0, _stream(stream)))


def cb_kv_quantize(x, n_rows: int, W: int, dtype: int, codes, scale, zero, stream=None):
    _check("cb_kv_quantize", lib().cb_kv_quantize(_ptr(x), n_rows, W, dtype, _ptr(codes), _ptr(scale), _ptr(zero),
                                                  _stream(stream)))


def cb_rope_shift_q8(k_dst, v_dst, k_codes, v_codes, k_scale, k_zero, v_scale, v_zero, src_row, n_src_rows: int,
                     qrow, n_qrows: int, delta, n_rows: int, dims: cb_dims, cos_sin, max_pos: int, stream=None):
    _check("cb_rope_shift_q8", lib().cb_rope_shift_q8(
        _ptr(k_dst), _ptr(v_dst), _ptr(k_codes), _ptr(v_codes), _ptr(k_scale), _ptr(k_zero), _ptr(v_scale),
        _ptr(v_zero), _ptr(src_row), n_src_rows, _ptr(qrow), n_qrows, _ptr(delta), n_rows, C.byref(dims),
        _ptr(cos_sin), max_pos, _stream(stream)))


def cb_kernel_launch_count() -> int:
    return int(lib().cb_kernel_launch_count())


def cb_profile_begin(max_records: int = 4096):
    _check("cb_profile_begin", lib().cb_profile_begin(max_records))


def cb_profile_begin_spans(max_records: int = 4096):
    _check("cb_profile_begin_spans", lib().cb_profile_begin_spans(max_records))


def cb_profile_end(max_records: int = 4096):
    """Returns a list of dicts {kind, aux, m, n, k, flops, bytes, ms, span_ms}, one per launch."""
    arr = (cb_prof_record * max_records)()
    n = _I32(0)
    _check("cb_profile_end", lib().cb_profile_end(arr, max_records, C.byref(n)))
    return [{"kind": PROF_KINDS.get(r.kind, str(r.kind)), "aux": r.aux, "m": r.m, "n": r.n, "k": r.k,
             "flops": r.flops, "bytes": r.bytes, "ms": r.ms, "span_ms": r.span_ms} for r in arr[:n.value]]


def _event(ev) -> int:
    return ev if isinstance(ev, int) else ev.cuda_event


def cb_prefetch_layer(dev_dst, pinned_src, nbytes: int, side_stream, done_event):
    _check("cb_prefetch_layer", lib().cb_prefetch_layer(_ptr(dev_dst), _ptr(pinned_src), nbytes,
                                                        _stream(side_stream), _event(done_event)))


def cb_stream_wait(stream, event):
    _check("cb_stream_wait", lib().cb_stream_wait(_stream(stream), _event(event)))


# ---- 8-bit KV cache of an answer in progress, rules on the logits ---------------------------
# These calls come once per token and layer, so their marshalling is kept short: the current
# device and stream are looked up once per call, torch's types once per process.
class _Torch:
    """torch and the types of the row dtypes, loaded at the first use."""

    def __init__(self):
        import torch
        self.mod, self.i8, self.i32, self.f32 = torch, torch.int8, torch.int32, torch.float32
        self.row = {CB_F32: torch.float32, CB_BF16: torch.bfloat16}
        self.cb = {v: k for k, v in self.row.items()}
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.raw_device = getattr(torch._C, "_cuda_getDevice", None)

    def device(self) -> int:
        cuda = self.mod.cuda
        if cuda.is_initialized() and self.raw_device is not None:
            return self.raw_device()
        return cuda.current_device() if cuda.is_available() else -2

    def stream(self, stream, dev: int):
        if stream is None and self.raw_stream is not None and dev >= 0:
            return self.raw_stream(dev)
        return _stream(stream)


_TORCH = None


def _torch() -> _Torch:
    global _TORCH
    if _TORCH is None:
        _TORCH = _Torch()
    return _TORCH


def _buf(what: str, t, dtype, n: Optional[int], dev: int) -> Optional[int]:
    """The address of a buffer.  A tensor must be contiguous, on the current CUDA device, of
    the element type and hold n elements (None: any number); raw pointers pass unchecked."""
    if t is None or type(t) is int:
        return t
    if t.dtype is not dtype:
        raise ValueError(f"{what}: {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: not contiguous")
    if n is not None and t.numel() != n:
        raise ValueError(f"{what}: {tuple(t.shape)} holds {t.numel()} elements, expected {n}")
    if t.get_device() != dev:
        raise ValueError(f"{what}: on {t.device}, not on the current CUDA device")
    return t.data_ptr()


def _ws(t, dev: int):
    """Address and size of a workspace tensor."""
    if t is None:
        return None, 0
    return _buf("ws", t, t.dtype, None, dev), t.numel() * t.element_size()


def kv8_cache(k_codes, v_codes, k_scale, v_scale, block: int) -> cb_kv8_cache:
    """The handle of a cache in these tensors: codes [n_seq, Hkv, capacity, head_dim] int8,
    scales [n_seq, Hkv, capacity / block] float32."""
    T = _torch()
    dev = T.device()
    n_seq, hkv, cap, hd = k_codes.shape
    if block not in (16, 32, 64, 128):
        raise ValueError(f"block {block} is not 16, 32, 64 or 128")
    ptr = _buf("k_codes", k_codes, T.i8, None, dev)
    if cap % block:
        raise ValueError(f"capacity {cap} is not a multiple of block {block}")
    scales = (n_seq, hkv, cap // block)
    for what, t, shape in (("v_codes", v_codes, k_codes.shape), ("k_scale", k_scale, scales), ("v_scale", v_scale, scales)):
        if tuple(t.shape) != tuple(shape):       # (the right number of elements in another layout would give wrong values)
            raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    c = cb_kv8_cache(ptr, _buf("v_codes", v_codes, T.i8, None, dev), _buf("k_scale", k_scale, T.f32, None, dev),
                     _buf("v_scale", v_scale, T.f32, None, dev), cap, n_seq, block)
    c.hkv, c.hd, c.dev, c.tensors = hkv, hd, dev, (k_codes, v_codes, k_scale, v_scale)
    return c


def _kv8(cache: cb_kv8_cache, dims: cb_dims, dev: int):
    if cache.dev != dev:
        raise ValueError(f"cache: on cuda:{cache.dev}, not on the current CUDA device")
    if cache.hkv != dims.n_kv_heads or cache.hd != dims.head_dim:
        raise ValueError(f"cache of {cache.hkv} heads of {cache.hd}, dims of {dims.n_kv_heads} heads of {dims.head_dim}")
    return C.byref(cache)


def cb_kv8_append(k, v, n_rows: int, start, count, cache: cb_kv8_cache, dims: cb_dims, stream=None):
    T = _torch()
    dev, dt, ns = T.device(), T.row[dims.dtype], cache.n_seq
    n = ns * n_rows * cache.hkv * cache.hd
    _check("cb_kv8_append", lib().cb_kv8_append(
        _buf("k", k, dt, n, dev), _buf("v", v, dt, n, dev), n_rows, _buf("start", start, T.i32, ns, dev),
        _buf("count", count, T.i32, ns, dev), _kv8(cache, dims, dev), C.byref(dims), T.stream(stream, dev)))


def cb_kv8_read(cache: cb_kv8_cache, start, count, n_rows: int, dims: cb_dims, k_out, v_out, stream=None):
    T = _torch()
    dev, dt, ns = T.device(), T.row[dims.dtype], cache.n_seq
    n = ns * n_rows * cache.hkv * cache.hd
    _check("cb_kv8_read", lib().cb_kv8_read(
        _kv8(cache, dims, dev), _buf("start", start, T.i32, ns, dev), _buf("count", count, T.i32, ns, dev), n_rows,
        C.byref(dims), _buf("k_out", k_out, dt, n, dev), _buf("v_out", v_out, dt, n, dev), T.stream(stream, dev)))


def cb_kv8_workspace_bytes(dims: cb_dims, n_seq: int, capacity: int, n_q: int, with_weights: bool = False) -> int:
    """Bytes for one call of these sizes.  Fewer queries may need more: for calls of several n_q on
    one buffer take the largest of what each asks for."""
    out = _SZ(0)
    _check("cb_kv8_workspace_bytes", lib().cb_kv8_workspace_bytes(C.byref(dims), n_seq, capacity, n_q,
                                                                  1 if with_weights else 0, C.byref(out)))
    return int(out.value)


def cb_kv8_attention(q, last, n_q: int, cache: cb_kv8_cache, dims: cb_dims, out, weights=None, ws=None, stream=None):
    T = _torch()
    dev, dt, ns = T.device(), T.row[dims.dtype], cache.n_seq
    n = ns * n_q * dims.n_heads * dims.head_dim
    w, wn = _ws(ws, dev)
    _check("cb_kv8_attention", lib().cb_kv8_attention(
        _buf("q", q, dt, n, dev), _buf("last", last, T.i32, ns * n_q, dev), n_q, _kv8(cache, dims, dev), C.byref(dims),
        _buf("out", out, dt, n, dev), _buf("weights", weights, T.f32, ns * cache.hkv * cache.capacity, dev), w, wn,
        T.stream(stream, dev)))


def cb_kv8_evict(src: cb_kv8_cache, length, weights, n_keep: int, n_sink: int, n_recent: int, dst: cb_kv8_cache,
                 dst_len, dst_weights, kept, dims: cb_dims, stream=None):
    T = _torch()
    dev, ns, heads = T.device(), src.n_seq, src.n_seq * src.hkv
    _check("cb_kv8_evict", lib().cb_kv8_evict(
        _kv8(src, dims, dev), _buf("length", length, T.i32, ns, dev),
        _buf("weights", weights, T.f32, heads * src.capacity, dev), n_keep, n_sink, n_recent, _kv8(dst, dims, dev),
        _buf("dst_len", dst_len, T.i32, ns, dev),
        _buf("dst_weights", dst_weights, T.f32, heads * dst.capacity, dev),
        _buf("kept", kept, T.i32, heads * n_keep, dev), C.byref(dims), T.stream(stream, dev)))


def logit_rules(history=None, history_len=None, prompt_len=None, repetition=None, presence=None, frequency=None,
                bias_id=None, bias=None, mask=None) -> cb_logit_rules:
    """The rules of one batch: history [n_rows, ld] int32 with its lengths, penalties [n_rows]
    float32, bias_id / bias [n_rows, n_bias], mask [n_rows, words] (32 ids a word, int32).
    None switches a rule off."""
    rows = [t.shape[0] for t in (history, history_len, prompt_len, repetition, presence, frequency, bias_id, bias, mask)
            if t is not None]
    if rows and min(rows) != max(rows):
        raise ValueError("the rules' tensors differ in their row count")
    if bias is not None and (bias_id is None or bias.shape != bias_id.shape):
        raise ValueError("bias and bias_id must have one shape")
    if history is None and any(t is not None for t in (history_len, prompt_len, repetition, presence, frequency)):
        raise ValueError("lengths and penalties need a history")
    T = _torch()
    dev, n = T.device(), rows[0] if rows else None
    r = cb_logit_rules(
        _buf("history", history, T.i32, None, dev), _buf("history_len", history_len, T.i32, n, dev),
        _buf("prompt_len", prompt_len, T.i32, n, dev), _buf("repetition", repetition, T.f32, n, dev),
        _buf("presence", presence, T.f32, n, dev), _buf("frequency", frequency, T.f32, n, dev),
        _buf("bias_id", bias_id, T.i32, None, dev), _buf("bias", bias, T.f32, None, dev),
        _buf("mask", mask, T.i32, None, dev), 0 if history is None else history.shape[1],
        0 if mask is None else mask.shape[1], 0 if bias_id is None else bias_id.shape[1])
    r.n_rows = rows[0] if rows else None
    r.dev = dev if rows else None
    r.tensors = (history, history_len, prompt_len, repetition, presence, frequency, bias_id, bias, mask)
    return r


def cb_logits_process(logits, rules: cb_logit_rules, out=None, token=None, stream=None):
    """logits [n_rows, vocab] float32 or bfloat16; out (may be logits) and token as in the header."""
    T = _torch()
    dev = T.device()
    n, vocab = logits.shape
    if rules.n_rows is not None and rules.n_rows != n:
        raise ValueError(f"rules for {rules.n_rows} rows, logits of {n}")
    if rules.dev is not None and rules.dev != dev:
        raise ValueError(f"rules: on cuda:{rules.dev}, not on the current CUDA device")
    dt = T.cb.get(logits.dtype)
    if dt is None:
        raise ValueError(f"logits: {logits.dtype}, expected float32 or bfloat16")
    _check("cb_logits_process", lib().cb_logits_process(
        _buf("logits", logits, logits.dtype, None, dev), n, vocab, dt, C.byref(rules),
        _buf("out", out, logits.dtype, n * vocab, dev), _buf("token", token, T.i32, n, dev), T.stream(stream, dev)))
