"""ctypes mirror of include/dsv4.h and tensor-to-argument marshalling.

Each ``dsv4_*`` function takes torch tensors, checks dtype/device/contiguity/shape, fills
the C argument struct with their data pointers, and calls the library on the current (or
given) CUDA stream. A non-zero status raises :class:`Dsv4Error`.
"""
from __future__ import annotations

import ctypes
import math
import os

HERE = os.path.dirname(os.path.abspath(__file__))

DSV4_OK = 0
DSV4_ERR_INVALID_ARG = 1
DSV4_ERR_LAUNCH = 2
DSV4_ERR_BAD_INDEX = 3
DSV4_ERR_TIMEOUT = 4
DSV4_ERR_UNSUPPORTED = 5
DSV4_ERR_NO_PAGES = 6
DSV4_EWORD_BAD_INDEX = 0x1
DSV4_EWORD_TIMEOUT = 0x2
DSV4_EWORD_NO_PAGES = 0x4
DSV4_WAIT_FAULT_NONE = 0
DSV4_WAIT_FAULT_SCORER_STAGE = 1
DSV4_WAIT_FAULT_ATTN_QUERY = 2
DSV4_WAIT_FAULT_PAGED_ATTN = 4
DSV4_WAIT_FAULT_PAGED_WEIGHTS = 8
DSV4_WAIT_FAULT_PAGED_PREFIX = 32

EXPORTED_SYMBOLS = (
    "dsv4_compress", "dsv4_compress_step", "dsv4_quantize_rows_fp8", "dsv4_indexer_topk_workspace_size",
    "dsv4_indexer_topk",
    "dsv4_index_score_workspace_size", "dsv4_index_score",
    "dsv4_topk_workspace_size", "dsv4_topk", "dsv4_topk_noalloc", "dsv4_sparse_attn_workspace_size",
    "dsv4_sparse_attn_decode", "dsv4_csa_decode_workspace_size", "dsv4_csa_decode",
    "dsv4_status_string", "dsv4_read_error_word", "dsv4_last_launch_count", "dsv4_max_comp",
    "dsv4_test_wait_fault", "dsv4_copy_async",
    "dsv4_norm_rope_append", "dsv4_paged_attn_workspace_size", "dsv4_paged_attn",
    "dsv4_paged_attn_weights_workspace_size", "dsv4_paged_attn_weights",
    "dsv4_paged_evict_workspace_size", "dsv4_paged_evict",
    "dsv4_paged_plan_workspace_size", "dsv4_paged_plan", "dsv4_rope",
    "dsv4_paged_prefix_attn_workspace_size", "dsv4_paged_prefix_attn",
)

P = ctypes.c_void_p
I = ctypes.c_int
L = ctypes.c_longlong


class CompressArgs(ctypes.Structure):
    _fields_ = [("C", P), ("Z", P), ("bias", P), ("gamma", P), ("pos0", P), ("out", P),
                ("out_row0", P), ("batch", I), ("tokens", I), ("dim", I), ("ratio", I),
                ("rope_dim", I), ("out_rows", I), ("eps", ctypes.c_float),
                ("rope_theta", ctypes.c_double), ("overlap", I), ("prev_C", P), ("prev_Z", P),
                ("out_fp8", I), ("out_scale", P), ("out_rope", P)]


class StepArgs(ctypes.Structure):
    _fields_ = [("C", P), ("Z", P), ("bias", P), ("gamma", P), ("pos", P), ("stage", P),
                ("fill", P), ("n_comp", P), ("out", P), ("batch", I), ("dim", I), ("ratio", I),
                ("rope_dim", I), ("out_rows", I), ("overlap", I), ("eps", ctypes.c_float),
                ("rope_theta", ctypes.c_double), ("out_fp8", I), ("out_scale", P), ("out_rope", P)]


class IndexArgs(ctypes.Structure):
    _fields_ = [("q", P), ("w", P), ("keys", P), ("n_comp", P), ("q_pos", P), ("idx_out", P),
                ("scores_out", P), ("batch", I), ("n_q", I), ("heads", I), ("dim", I),
                ("max_comp", I), ("top_k", I), ("ratio", I), ("key_fp8", I), ("q_scale", P),
                ("key_scale", P)]


class TopkArgs(ctypes.Structure):
    _fields_ = [("scores", P), ("n_vis", P), ("idx_out", P), ("rows", I), ("max_comp", I),
                ("top_k", I)]


class AttnArgs(ctypes.Structure):
    _fields_ = [("q", P), ("sink", P), ("comp_kv", P), ("n_comp", P), ("idx", P), ("q_pos", P),
                ("win", P), ("win_len", P), ("gather", P), ("out", P), ("batch", I), ("n_q", I),
                ("heads", I), ("dim", I), ("max_comp", I), ("top_k", I), ("window", I),
                ("win_rows", I), ("ratio", I), ("scale", ctypes.c_float), ("out_rope_pos", P),
                ("out_rope_dim", I), ("out_rope_theta", ctypes.c_double), ("kv_fp8", I),
                ("kv_nope", P), ("kv_scale", P), ("kv_rope", P), ("kv_rope_dim", I)]


class NormRopeArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k", P), ("v", P), ("q_out", P), ("k_pages", P), ("v_pages", P),
                ("slots", P), ("pos", P), ("gamma_q", P), ("gamma_k", P),
                ("q_stride", L), ("k_stride", L), ("v_stride", L), ("q_out_stride", L),
                ("tokens", I), ("heads", I), ("kv_heads", I), ("dim", I), ("page_size", I),
                ("num_pages", I), ("rope_dim", I), ("eps", ctypes.c_float),
                ("rope_theta", ctypes.c_double)]


class PagedAttnArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k_pages", P), ("v_pages", P), ("block_table", P), ("cu_q", P),
                ("kv_len", P), ("sink", P), ("out", P), ("lse", P), ("out_rope_pos", P),
                ("q_stride", L), ("batch", I), ("total_q", I), ("heads", I), ("kv_heads", I),
                ("dim", I), ("page_size", I), ("num_pages", I), ("max_pages", I), ("max_q", I),
                ("window", I), ("scale", ctypes.c_float), ("out_rope_dim", I),
                ("out_rope_theta", ctypes.c_double)]


class PagedWeightsArgs(ctypes.Structure):
    _fields_ = [("q", P), ("lse", P), ("k_pages", P), ("block_table", P), ("cu_q", P),
                ("kv_len", P), ("acc_in", P), ("acc", P), ("q_stride", L), ("batch", I),
                ("total_q", I), ("heads", I), ("kv_heads", I), ("dim", I), ("page_size", I),
                ("num_pages", I), ("max_pages", I), ("max_q", I), ("window", I), ("acc_rows", I),
                ("scale", ctypes.c_float)]


class PagedEvictArgs(ctypes.Structure):
    _fields_ = [("k_pages", P), ("v_pages", P), ("block_table", P), ("out_table", P),
                ("kv_len", P), ("kv_len_out", P), ("acc", P), ("acc_out", P), ("keep", P),
                ("batch", I), ("kv_heads", I), ("dim", I), ("page_size", I), ("num_pages", I),
                ("max_pages", I), ("out_pages", I), ("acc_rows", I), ("budget", I), ("recent", I)]


class PagedPlanArgs(ctypes.Structure):
    _fields_ = [("new_len", P), ("kv_len", P), ("held", P), ("shared", P), ("next_pos", P),
                ("block_table", P), ("free_pages", P), ("free_count", P), ("cu_q", P),
                ("kv_len_out", P), ("held_out", P), ("next_pos_out", P), ("free_count_out", P),
                ("slots", P), ("pos", P), ("seq", P), ("batch", I), ("total_q", I),
                ("page_size", I), ("num_pages", I), ("max_pages", I), ("free_cap", I)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k", P), ("v", P), ("q_out", P), ("k_out", P), ("v_out", P),
                ("slots", P), ("pos", P), ("q_stride", L), ("k_stride", L), ("v_stride", L),
                ("q_out_stride", L), ("k_out_stride", L), ("tokens", I), ("heads", I),
                ("kv_heads", I), ("dim", I), ("page_size", I), ("num_pages", I), ("dtype", I),
                ("rope_dim", I), ("first", I), ("layout", I), ("inverse", I), ("scaling", I),
                ("rope_theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("magnitude", ctypes.c_double)]


class PagedPrefixArgs(ctypes.Structure):
    _fields_ = [("q", P), ("k_pages", P), ("v_pages", P), ("block_table", P), ("cu_q", P),
                ("kv_len", P), ("prefix_len", P), ("group_start", P), ("sink", P), ("out", P),
                ("lse", P), ("out_rope_pos", P), ("q_stride", L), ("batch", I), ("groups", I),
                ("total_q", I), ("heads", I), ("kv_heads", I), ("dim", I), ("page_size", I),
                ("num_pages", I), ("max_pages", I), ("scale", ctypes.c_float),
                ("out_rope_dim", I), ("out_rope_theta", ctypes.c_double)]


class CsaArgs(ctypes.Structure):
    _fields_ = [("compress_kv", ctypes.POINTER(CompressArgs)),
                ("compress_keys", ctypes.POINTER(CompressArgs)),
                ("index", ctypes.POINTER(IndexArgs)), ("attn", ctypes.POINTER(AttnArgs))]


class Dsv4Error(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {dsv4_status_string(status)} (status {status})")


_lib = None


def library_path() -> str:
    return os.path.join(HERE, "libdsv4.so")


def library():
    """The loaded CUDA library. Raises if it has not been built: there is no fallback."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"CSA CUDA library not built ({path}); run "
                               "`python -m compressed_sparse_attention_08_gb300._build`")
        lib = ctypes.CDLL(path)
        lib.dsv4_compress.argtypes = [ctypes.POINTER(CompressArgs), P]
        lib.dsv4_compress_step.argtypes = [ctypes.POINTER(StepArgs), P]
        lib.dsv4_quantize_rows_fp8.argtypes = [P, I, I, P, P, P]
        lib.dsv4_indexer_topk_workspace_size.argtypes = [ctypes.POINTER(IndexArgs)]
        lib.dsv4_indexer_topk_workspace_size.restype = ctypes.c_size_t
        lib.dsv4_indexer_topk.argtypes = [ctypes.POINTER(IndexArgs), P, ctypes.c_size_t, P]
        lib.dsv4_index_score_workspace_size.argtypes = [ctypes.POINTER(IndexArgs)]
        lib.dsv4_index_score_workspace_size.restype = ctypes.c_size_t
        lib.dsv4_index_score.argtypes = [ctypes.POINTER(IndexArgs), P, ctypes.c_size_t, P]
        lib.dsv4_topk_workspace_size.argtypes = [ctypes.POINTER(TopkArgs)]
        lib.dsv4_topk_workspace_size.restype = ctypes.c_size_t
        lib.dsv4_topk.argtypes = [ctypes.POINTER(TopkArgs), P, ctypes.c_size_t, P]
        lib.dsv4_topk_noalloc.argtypes = [ctypes.POINTER(TopkArgs), P]
        lib.dsv4_topk_noalloc.restype = I
        lib.dsv4_sparse_attn_workspace_size.argtypes = [ctypes.POINTER(AttnArgs)]
        lib.dsv4_sparse_attn_workspace_size.restype = ctypes.c_size_t
        lib.dsv4_sparse_attn_decode.argtypes = [ctypes.POINTER(AttnArgs), P, ctypes.c_size_t, P]
        lib.dsv4_csa_decode_workspace_size.argtypes = [ctypes.POINTER(CsaArgs)]
        lib.dsv4_csa_decode_workspace_size.restype = ctypes.c_size_t
        lib.dsv4_csa_decode.argtypes = [ctypes.POINTER(CsaArgs), P, ctypes.c_size_t, P]
        lib.dsv4_status_string.argtypes = [I]
        lib.dsv4_status_string.restype = ctypes.c_char_p
        lib.dsv4_read_error_word.argtypes = [P, P, ctypes.POINTER(ctypes.c_uint32)]
        lib.dsv4_last_launch_count.restype = I
        lib.dsv4_max_comp.argtypes = [ctypes.c_int64, I]
        lib.dsv4_max_comp.restype = ctypes.c_int64
        lib.dsv4_test_wait_fault.argtypes = [I, ctypes.c_uint32]
        lib.dsv4_test_wait_fault.restype = I
        lib.dsv4_copy_async.argtypes = [P, P, ctypes.c_size_t, P]
        lib.dsv4_copy_async.restype = I
        lib.dsv4_norm_rope_append.argtypes = [ctypes.POINTER(NormRopeArgs), P]
        lib.dsv4_norm_rope_append.restype = I
        lib.dsv4_rope.argtypes = [ctypes.POINTER(RopeArgs), P]
        lib.dsv4_rope.restype = I
        for name, st in (("dsv4_paged_attn", PagedAttnArgs), ("dsv4_paged_attn_weights", PagedWeightsArgs),
                         ("dsv4_paged_evict", PagedEvictArgs), ("dsv4_paged_plan", PagedPlanArgs),
                         ("dsv4_paged_prefix_attn", PagedPrefixArgs)):
            size = getattr(lib, name + "_workspace_size")
            size.argtypes = [ctypes.POINTER(st)]
            size.restype = ctypes.c_size_t
            getattr(lib, name).argtypes = [ctypes.POINTER(st), P, ctypes.c_size_t, P]
            getattr(lib, name).restype = I
        for f in ("dsv4_compress", "dsv4_indexer_topk", "dsv4_index_score", "dsv4_topk", "dsv4_sparse_attn_decode",
                  "dsv4_csa_decode", "dsv4_read_error_word"):
            getattr(lib, f).restype = I
        _lib = lib
    return _lib


# ------------------------------------------------------------------ marshalling helpers
def _ptr(t, dtype=None, name="tensor", optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(status, what):
    if status != DSV4_OK:
        raise Dsv4Error(status, what)


def _dt():
    import torch
    return torch.bfloat16, torch.float32, torch.int32, torch.int64


# ------------------------------------------------------------------ argument builders
def compress_args(C, Z, bias, gamma, pos0, out, *, ratio, rope_dim=64, eps=1e-6,
                  rope_theta=10000.0, out_row0=None, overlap=False, prev_C=None, prev_Z=None,
                  out_scale=None, out_rope=None):
    """overlap=True: the two-stream (CSA) form, C and Z [B, T, 2*dim], bias [ratio, 2*dim],
    optional prev_C / prev_Z [B, ratio, 2*dim] (the block before C's first block).
    out_scale given: FP8 entries, out uint8 [B, rows, dim] and out_scale fp32 [B, rows].
    out_scale and out_rope given: the mixed KV storage, out uint8 [B, rows, dim - rope_dim]
    codes, out_scale fp32 [B, rows], out_rope bf16 [B, rows, rope_dim]."""
    import torch
    bf16, f32, i32, i64 = _dt()
    B, T, w = C.shape
    d = w // 2 if overlap else w
    fp8 = out_scale is not None
    mode = 2 if (fp8 and out_rope is not None) else (1 if fp8 else 0)
    return CompressArgs(_ptr(C, bf16, "C"), _ptr(Z, bf16, "Z"), _ptr(bias, f32, "bias"),
                        _ptr(gamma, f32, "gamma"), _ptr(pos0, i64, "pos0"),
                        _ptr(out, torch.uint8 if fp8 else bf16, "out"),
                        _ptr(out_row0, i32, "out_row0", True), B, T, d, ratio, rope_dim,
                        out.shape[1], eps, rope_theta, 1 if overlap else 0,
                        _ptr(prev_C, bf16, "prev_C", True), _ptr(prev_Z, bf16, "prev_Z", True),
                        mode, _ptr(out_scale, f32, "out_scale", True),
                        _ptr(out_rope, bf16, "out_rope", True))


def index_args(q, w, keys, n_comp, idx_out, *, ratio, q_pos=None, scores_out=None, q_scale=None,
               key_scale=None):
    """q_scale / key_scale given: q and keys are FP8 E4M3 codes (uint8), as
    dsv4_quantize_rows_fp8 writes them."""
    bf16, f32, i32, i64 = _dt()
    import torch
    fp8 = q_scale is not None
    kt = torch.uint8 if fp8 else bf16
    B, n_q, H, Di = q.shape
    return IndexArgs(_ptr(q, kt, "q"), _ptr(w, f32, "w"), _ptr(keys, kt, "keys"),
                     _ptr(n_comp, i32, "n_comp"), _ptr(q_pos, i64, "q_pos", True),
                     _ptr(idx_out, i32, "idx_out"), _ptr(scores_out, f32, "scores_out", True),
                     B, n_q, H, Di, keys.shape[1], idx_out.shape[-1], ratio, 1 if fp8 else 0,
                     _ptr(q_scale, f32, "q_scale", True), _ptr(key_scale, f32, "key_scale", True))


def topk_args(scores, n_vis, idx_out):
    bf16, f32, i32, i64 = _dt()
    rows = n_vis.numel()
    return TopkArgs(_ptr(scores, f32, "scores"), _ptr(n_vis, i32, "n_vis"),
                    _ptr(idx_out, i32, "idx_out"), rows, scores.shape[-1], idx_out.shape[-1])


def attn_args(q, sink, comp_kv, n_comp, win, win_len, out, *, idx=None, top_k=None, window=128,
              ratio=4, q_pos=None, gather=None, scale=None, out_rope_pos=None, out_rope_dim=64,
              out_rope_theta=10000.0, kv_nope=None, kv_scale=None, kv_rope=None):
    """out_rope_pos (int64 [B, n_q]): rotate the output's last out_rope_dim channels back at
    these positions (inverse RoPE). comp_kv None and kv_nope / kv_scale / kv_rope given: the
    mixed FP8 / bf16 compressed KV (codes uint8 [B, max_comp, D - rd], scales fp32
    [B, max_comp], RoPE part bf16 [B, max_comp, rd])."""
    import torch
    bf16, f32, i32, i64 = _dt()
    B, n_q, H, D = q.shape
    kv_fp8 = comp_kv is None
    max_comp = kv_nope.shape[1] if kv_fp8 else comp_kv.shape[1]
    if top_k is None:
        top_k = idx.shape[-1] if idx is not None else max_comp
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    return AttnArgs(_ptr(q, bf16, "q"), _ptr(sink, f32, "sink"), _ptr(comp_kv, bf16, "comp_kv", kv_fp8),
                    _ptr(n_comp, i32, "n_comp"), _ptr(idx, i32, "idx", True),
                    _ptr(q_pos, i64, "q_pos", True), _ptr(win, bf16, "win"),
                    _ptr(win_len, i32, "win_len"), _ptr(gather, bf16, "gather", True),
                    _ptr(out, bf16, "out"), B, n_q, H, D, max_comp, top_k, window, win.shape[1],
                    ratio, scale, _ptr(out_rope_pos, i64, "out_rope_pos", True),
                    out_rope_dim if out_rope_pos is not None else 0, out_rope_theta,
                    1 if kv_fp8 else 0, _ptr(kv_nope, torch.uint8, "kv_nope", True),
                    _ptr(kv_scale, f32, "kv_scale", True), _ptr(kv_rope, bf16, "kv_rope", True),
                    kv_rope.shape[-1] if kv_fp8 else 0)


# ------------------------------------------------------------------ entry points
def dsv4_compress(C, Z, bias, gamma, pos0, out, *, ratio, rope_dim=64, eps=1e-6,
                  rope_theta=10000.0, out_row0=None, overlap=False, prev_C=None, prev_Z=None,
                  out_scale=None, out_rope=None, stream=None):
    a = compress_args(C, Z, bias, gamma, pos0, out, ratio=ratio, rope_dim=rope_dim, eps=eps,
                      rope_theta=rope_theta, out_row0=out_row0, overlap=overlap, prev_C=prev_C,
                      prev_Z=prev_Z, out_scale=out_scale, out_rope=out_rope)
    _check(library().dsv4_compress(ctypes.byref(a), _stream(stream)), "dsv4_compress")


def dsv4_quantize_rows_fp8(x, q, scale, *, stream=None):
    """FP8 E4M3 rows: x bf16 [..., dim] -> q uint8 [..., dim], scale fp32 [...]."""
    import torch
    bf16, f32, i32, i64 = _dt()
    dim = x.shape[-1]
    rows = x.numel() // dim
    _check(library().dsv4_quantize_rows_fp8(_ptr(x, bf16, "x"), rows, dim, _ptr(q, torch.uint8, "q"),
                                            _ptr(scale, f32, "scale"), _stream(stream)),
           "dsv4_quantize_rows_fp8")


def compress_step_state(batch, dim, ratio, *, overlap=False, device="cuda"):
    """Zeroed state for dsv4_compress_step: (stage, fill, n_comp)."""
    import torch
    w = 2 * dim if overlap else dim
    return (torch.zeros(batch, 2, 2, ratio, w, dtype=torch.bfloat16, device=device),
            torch.zeros(batch, dtype=torch.int32, device=device),
            torch.zeros(batch, dtype=torch.int32, device=device))


def dsv4_compress_step(C, Z, bias, gamma, pos, stage, fill, n_comp, out, *, ratio, rope_dim=64,
                       eps=1e-6, rope_theta=10000.0, overlap=False, out_scale=None, out_rope=None,
                       stream=None):
    """One decode token per sequence: C, Z [B, w] (w = dim, or 2*dim two-stream); pos int64 [B];
    state stage / fill / n_comp (see compress_step_state) updated on the device; a completed
    block goes to out[s, n_comp[s]]. out_scale (and out_rope): the FP8 (mixed) cache formats,
    as compress_args."""
    import torch
    bf16, f32, i32, i64 = _dt()
    B, w = C.shape
    fp8 = out_scale is not None
    mode = 2 if (fp8 and out_rope is not None) else (1 if fp8 else 0)
    d = out.shape[2] + (out_rope.shape[2] if mode == 2 else 0)
    a = StepArgs(_ptr(C, bf16, "C"), _ptr(Z, bf16, "Z"), _ptr(bias, f32, "bias"), _ptr(gamma, f32, "gamma"),
                 _ptr(pos, i64, "pos"), _ptr(stage, bf16, "stage"), _ptr(fill, i32, "fill"),
                 _ptr(n_comp, i32, "n_comp"), _ptr(out, torch.uint8 if fp8 else bf16, "out"), B, d, ratio,
                 rope_dim, out.shape[1], 1 if overlap else 0, eps, rope_theta, mode,
                 _ptr(out_scale, f32, "out_scale", True), _ptr(out_rope, bf16, "out_rope", True))
    _check(library().dsv4_compress_step(ctypes.byref(a), _stream(stream)), "dsv4_compress_step")


def dsv4_indexer_topk_workspace_size(q, w, keys, n_comp, idx_out, *, ratio, q_pos=None,
                                     scores_out=None, q_scale=None, key_scale=None):
    a = index_args(q, w, keys, n_comp, idx_out, ratio=ratio, q_pos=q_pos, scores_out=scores_out,
                   q_scale=q_scale, key_scale=key_scale)
    return int(library().dsv4_indexer_topk_workspace_size(ctypes.byref(a)))


def dsv4_indexer_topk(q, w, keys, n_comp, idx_out, ws, *, ratio, q_pos=None, scores_out=None,
                      q_scale=None, key_scale=None, stream=None):
    """q_scale / key_scale given: FP8 E4M3 queries and keys (see index_args)."""
    a = index_args(q, w, keys, n_comp, idx_out, ratio=ratio, q_pos=q_pos, scores_out=scores_out,
                   q_scale=q_scale, key_scale=key_scale)
    _check(library().dsv4_indexer_topk(ctypes.byref(a), _ptr(ws, None, "ws"), ws.numel() * ws.element_size(),
                                       _stream(stream)), "dsv4_indexer_topk")


def dsv4_index_score_workspace_size(q, w, keys, n_comp, scores_out, *, ratio, q_pos=None,
                                    q_scale=None, key_scale=None):
    import torch
    idx = torch.empty(1, dtype=torch.int32, device=q.device)
    a = index_args(q, w, keys, n_comp, idx, ratio=ratio, q_pos=q_pos, scores_out=scores_out,
                   q_scale=q_scale, key_scale=key_scale)
    a.top_k = 1
    return int(library().dsv4_index_score_workspace_size(ctypes.byref(a)))


def dsv4_index_score(q, w, keys, n_comp, scores_out, ws, *, ratio, q_pos=None, q_scale=None,
                     key_scale=None, stream=None):
    """Scores only (no top-k): scores_out [B, n_q, max_comp] fp32 gets the visible scores."""
    import torch
    idx = torch.empty(1, dtype=torch.int32, device=q.device)
    a = index_args(q, w, keys, n_comp, idx, ratio=ratio, q_pos=q_pos, scores_out=scores_out,
                   q_scale=q_scale, key_scale=key_scale)
    a.top_k = 1
    _check(library().dsv4_index_score(ctypes.byref(a), _ptr(ws, None, "ws"), ws.numel() * ws.element_size(),
                                      _stream(stream)), "dsv4_index_score")


def dsv4_topk_workspace_size(scores, n_vis, idx_out):
    a = topk_args(scores, n_vis, idx_out)
    return int(library().dsv4_topk_workspace_size(ctypes.byref(a)))


def dsv4_topk(scores, n_vis, idx_out, ws, *, stream=None):
    a = topk_args(scores, n_vis, idx_out)
    _check(library().dsv4_topk(ctypes.byref(a), _ptr(ws, None, "ws"), ws.numel() * ws.element_size(),
                               _stream(stream)), "dsv4_topk")


def dsv4_topk_noalloc(scores, n_vis, idx_out, *, stream=None):
    """dsv4_topk without a workspace, for callers that cannot allocate device memory: the
    library's fixed 16 MiB per-GPU scratch array is used instead. Calls must not overlap on
    the GPU; sizes needing more scratch than the array holds raise Dsv4Error
    (DSV4_ERR_INVALID_ARG)."""
    a = topk_args(scores, n_vis, idx_out)
    _check(library().dsv4_topk_noalloc(ctypes.byref(a), _stream(stream)), "dsv4_topk_noalloc")


def dsv4_sparse_attn_workspace_size(q, sink, comp_kv, n_comp, win, win_len, out, **kw):
    a = attn_args(q, sink, comp_kv, n_comp, win, win_len, out, **kw)
    return int(library().dsv4_sparse_attn_workspace_size(ctypes.byref(a)))


def dsv4_sparse_attn_decode(q, sink, comp_kv, n_comp, win, win_len, out, ws, *, stream=None, **kw):
    a = attn_args(q, sink, comp_kv, n_comp, win, win_len, out, **kw)
    _check(library().dsv4_sparse_attn_decode(ctypes.byref(a), _ptr(ws, None, "ws"),
                                             ws.numel() * ws.element_size(), _stream(stream)),
           "dsv4_sparse_attn_decode")


def _csa(compress_kv, compress_keys, index, attn):
    keep = (compress_kv, compress_keys, index, attn)
    c = CsaArgs(ctypes.pointer(compress_kv) if compress_kv is not None else None,
                ctypes.pointer(compress_keys) if compress_keys is not None else None,
                ctypes.pointer(index) if index is not None else None, ctypes.pointer(attn))
    return c, keep


def dsv4_csa_decode_workspace_size(*, attn, index=None, compress_kv=None, compress_keys=None):
    c, _keep = _csa(compress_kv, compress_keys, index, attn)
    return int(library().dsv4_csa_decode_workspace_size(ctypes.byref(c)))


def dsv4_csa_decode(ws, *, attn, index=None, compress_kv=None, compress_keys=None, stream=None):
    """One decode step from prepared argument structs (see compress_args / index_args /
    attn_args); the structs keep raw pointers, so the tensors must outlive the call."""
    c, _keep = _csa(compress_kv, compress_keys, index, attn)
    _check(library().dsv4_csa_decode(ctypes.byref(c), _ptr(ws, None, "ws"),
                                     ws.numel() * ws.element_size(), _stream(stream)),
           "dsv4_csa_decode")


def dsv4_read_error_word(ws, stream=None):
    v = ctypes.c_uint32(0)
    st = library().dsv4_read_error_word(_ptr(ws, None, "ws"), _stream(stream), ctypes.byref(v))
    return st, int(v.value)


def dsv4_status_string(status):
    try:
        return library().dsv4_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def dsv4_last_launch_count():
    return int(library().dsv4_last_launch_count())


def dsv4_max_comp(max_context, ratio):
    return int(library().dsv4_max_comp(int(max_context), int(ratio)))


def dsv4_copy_async(dst, src, stream=None):
    """Copies tensor src into dst (same byte size, contiguous; each on the GPU or in pinned host
    memory) with the library's copy kernel, after the kernel before it on the stream."""
    import torch
    for t, name in ((dst, "dst"), (src, "src")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.device.type != "cuda" and not t.is_pinned():
            raise ValueError(f"{name} must be on the GPU or in pinned host memory")
    nbytes = dst.numel() * dst.element_size()
    if src.numel() * src.element_size() != nbytes:
        raise ValueError("dst and src differ in size")
    _check(library().dsv4_copy_async(ctypes.c_void_p(dst.data_ptr()), ctypes.c_void_p(src.data_ptr()), nbytes,
                                     _stream(stream)), "dsv4_copy_async")


def dsv4_test_wait_fault(which, wait_limit_us=0):
    """Test support: from now on every launch of kernel `which` (DSV4_WAIT_FAULT_*) leaves one
    copy unissued so its bounded wait runs out after wait_limit_us microseconds (0: the
    default 2 s); DSV4_WAIT_FAULT_NONE restores normal launches."""
    _check(library().dsv4_test_wait_fault(int(which), int(wait_limit_us)), "dsv4_test_wait_fault")


# ------------------------------------------------------------------ the paged cache
# Prepared argument structs, as for dsv4_csa_decode: a serving loop builds them once over its
# buffers and issues the same call every step. A struct holds its tensors, and the call runs on
# the device they are on.
def _heads_ptr(t, name, optional=False, dtype=None):
    """[tokens, heads, dim] in bf16 (or dtype) whose tokens may be further apart than their heads (a
    part of a fused projection): (pointer, token stride in elements)."""
    if t is None:
        if optional:
            return None, 0
        raise ValueError(f"{name} is required")
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != (dtype or torch.bfloat16):
        raise TypeError(f"{name} must be {dtype or torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim]")
    n, h, d = t.shape
    if t.numel() and ((d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d)):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return ctypes.c_void_p(t.data_ptr()), t.stride(0) if n > 1 else h * d


def _shape(t, shape, name):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _struct(cls, *values):
    """cls(*values), whose counts must fit their 32 bits (ctypes would keep the low ones)."""
    if len(values) != len(cls._fields_):
        raise ValueError(f"{cls.__name__} has {len(cls._fields_)} fields, got {len(values)}")
    for (name, kind), v in zip(cls._fields_, values):
        if kind is I and not -(1 << 31) <= v < 1 << 31:
            raise ValueError(f"{name} is out of range: {v}")
    return cls(*values)


def _held(args, *tensors):
    """Keeps the tensors with the struct; all must be on one device. (Nothing here may refer back to the struct, a stored
    byref included: the tensors would then live until the cyclic collector runs.)"""
    kept = [t for t in tensors if t is not None]
    if any(t.device != kept[0].device for t in kept):
        raise ValueError("all tensors must be on one device")
    args.tensors = kept
    args.device = kept[0].device.index
    return args


def _call(fn, args, stream, what, ws=None):
    """fn on the struct (and a workspace), with the struct's device current, on its current stream
    unless one is given."""
    import torch
    dev = args.device
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _call(fn, args, stream, what, ws)
    # (the raw handle: torch.cuda.current_stream() takes 3 us to wrap it)
    st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    if ws is None:
        status = fn(args, st)
    else:
        if ws.device.index != dev or not ws.is_contiguous():
            raise ValueError("ws must be contiguous, on the tensors' device")
        status = fn(args, ws.data_ptr(), ws.numel() * ws.element_size(), st)
    if status:
        _check(status, what)


def norm_rope_args(q, q_out, pos, *, k=None, k_pages=None, v=None, v_pages=None, slots=None,
                   gamma_q=None, gamma_k=None, rope_dim=64, eps=1e-6, rope_theta=10000.0):
    """q bf16 [T, H, D] -> q_out (may be q); k bf16 [T, KV, D] -> row slots[t] (int64 [T], page *
    page_size + slot, negative: not stored) of k_pages bf16 [pages, page_size, KV, D]; v likewise,
    unchanged. pos int64 [T]. q or k may be None."""
    bf16, f32, i32, i64 = _dt()
    some = q if q is not None else k
    if some is None:
        raise ValueError("q or k is required")
    T, _, D = some.shape
    H = 0 if q is None else q.shape[1]
    KV = 0 if k is None else k.shape[1]
    _shape(q, (T, H, D), "q")
    _shape(q_out, (T, H, D), "q_out")
    _shape(k, (T, KV, D), "k")
    _shape(v, (T, KV, D), "v")
    _shape(pos, (T,), "pos")
    _shape(slots, (T,), "slots")
    _shape(gamma_q, (D,), "gamma_q")
    _shape(gamma_k, (D,), "gamma_k")
    if k is not None:
        if k_pages is None or slots is None:
            raise ValueError("k needs k_pages and slots")
        _shape(k_pages, (*k_pages.shape[:2], KV, D), "k_pages")
        _shape(v_pages, k_pages.shape, "v_pages")
    elif v is not None:
        raise ValueError("v needs k")
    qp, qs = _heads_ptr(q, "q", True)
    op, os_ = _heads_ptr(q_out, "q_out", q is None)
    kp, ks = _heads_ptr(k, "k", True)
    vp, vs = _heads_ptr(v, "v", True)
    a = _struct(NormRopeArgs, qp, kp, vp, op, _ptr(k_pages, bf16, "k_pages", True), _ptr(v_pages, bf16, "v_pages", True),
                _ptr(slots, i64, "slots", True), _ptr(pos, i64, "pos"), _ptr(gamma_q, f32, "gamma_q", True),
                _ptr(gamma_k, f32, "gamma_k", True), qs, ks, vs, os_, T, H, KV, D,
                0 if k_pages is None else k_pages.shape[1], 0 if k_pages is None else k_pages.shape[0],
                rope_dim, eps, rope_theta)
    return _held(a, q, q_out, pos, k, k_pages, v, v_pages, slots, gamma_q, gamma_k)


def dsv4_norm_rope_append(args, *, stream=None):
    """RMSNorm per head, RoPE and the append to the pages, from a norm_rope_args struct."""
    _call(library().dsv4_norm_rope_append, args, stream, "dsv4_norm_rope_append")


def _paged(q, k_pages, block_table, cu_q, kv_len):
    bf16, f32, i32, i64 = _dt()
    qp, qs = _heads_ptr(q, "q")
    T, H, D = q.shape
    if k_pages.dim() != 4 or k_pages.shape[3] != D:
        raise ValueError("k_pages must be [num_pages, page_size, kv_heads, dim]")
    B = kv_len.shape[0]
    _shape(block_table, (B, block_table.shape[-1]), "block_table")
    _shape(cu_q, (B + 1,), "cu_q")
    _shape(kv_len, (B,), "kv_len")
    return qp, qs, T, H, D, B, k_pages.shape[0], k_pages.shape[1], k_pages.shape[2], block_table.shape[1]


def paged_attn_args(q, out, k_pages, block_table, cu_q, kv_len, *, v_pages=None, max_q=None,
                    sink=None, lse=None, window=0, scale=None, out_rope_pos=None, out_rope_dim=64,
                    out_rope_theta=10000.0):
    """q bf16 [T, H, D], out bf16 [T, H, D], k_pages (v_pages) bf16 [pages, page_size, KV, D],
    block_table int32 [B, max_pages], cu_q int32 [B + 1], kv_len int32 [B], sink fp32 [H], lse
    fp32 [T, H], out_rope_pos int64 [T]. max_q: the most tokens of one sequence (default T)."""
    bf16, f32, i32, i64 = _dt()
    qp, qs, T, H, D, B, n, ps, KV, mp = _paged(q, k_pages, block_table, cu_q, kv_len)
    _shape(out, (T, H, D), "out")
    _shape(v_pages, k_pages.shape, "v_pages")
    _shape(sink, (H,), "sink")
    _shape(lse, (T, H), "lse")
    _shape(out_rope_pos, (T,), "out_rope_pos")
    a = _struct(PagedAttnArgs, qp, _ptr(k_pages, bf16, "k_pages"), _ptr(v_pages, bf16, "v_pages", True),
                _ptr(block_table, i32, "block_table"), _ptr(cu_q, i32, "cu_q"), _ptr(kv_len, i32, "kv_len"),
                _ptr(sink, f32, "sink", True), _ptr(out, bf16, "out"), _ptr(lse, f32, "lse", True),
                _ptr(out_rope_pos, i64, "out_rope_pos", True), qs, B, T, H, KV, D, ps, n, mp,
                max(1, T if max_q is None else max_q), window, 1.0 / math.sqrt(D) if scale is None else scale,
                out_rope_dim if out_rope_pos is not None else 0, out_rope_theta)
    return _held(a, q, out, k_pages, v_pages, block_table, cu_q, kv_len, sink, lse, out_rope_pos)


def dsv4_paged_attn_workspace_size(args):
    return int(library().dsv4_paged_attn_workspace_size(ctypes.byref(args)))


def dsv4_paged_attn(args, ws, *, stream=None):
    """Attention of the new tokens over their sequences' pages, from a paged_attn_args struct."""
    _call(library().dsv4_paged_attn, args, stream, "dsv4_paged_attn", ws)


def paged_weights_args(q, lse, k_pages, block_table, cu_q, kv_len, acc, *, acc_in=None, max_q=None,
                       window=0, scale=None):
    """q, pages, tables and lengths as paged_attn_args, lse fp32 [T, H] as that call wrote it; acc
    fp32 [B, rows] = acc_in (or 0) + the weights."""
    bf16, f32, i32, i64 = _dt()
    qp, qs, T, H, D, B, n, ps, KV, mp = _paged(q, k_pages, block_table, cu_q, kv_len)
    _shape(lse, (T, H), "lse")
    _shape(acc, (B, acc.shape[-1]), "acc")
    _shape(acc_in, acc.shape, "acc_in")
    a = _struct(PagedWeightsArgs, qp, _ptr(lse, f32, "lse"), _ptr(k_pages, bf16, "k_pages"), _ptr(block_table, i32, "block_table"),
                _ptr(cu_q, i32, "cu_q"), _ptr(kv_len, i32, "kv_len"), _ptr(acc_in, f32, "acc_in", True),
                _ptr(acc, f32, "acc"), qs, B, T, H, KV, D, ps, n, mp, max(1, T if max_q is None else max_q),
                window, acc.shape[1], 1.0 / math.sqrt(D) if scale is None else scale)
    return _held(a, q, lse, k_pages, block_table, cu_q, kv_len, acc, acc_in)


def dsv4_paged_attn_weights_workspace_size(args):
    return int(library().dsv4_paged_attn_weights_workspace_size(ctypes.byref(args)))


def dsv4_paged_attn_weights(args, ws, *, stream=None):
    """The weight each cached row received, from a paged_weights_args struct."""
    _call(library().dsv4_paged_attn_weights, args, stream, "dsv4_paged_attn_weights", ws)


def paged_evict_args(k_pages, block_table, kv_len, acc, keep, *, budget, recent, v_pages=None,
                     out_table=None, kv_len_out=None, acc_out=None):
    """Cut the caches to `budget` rows: acc fp32 [B, rows], keep int32 [B, budget]. out_table,
    kv_len_out and acc_out default to block_table, kv_len and acc (in place)."""
    bf16, f32, i32, i64 = _dt()
    B = kv_len.shape[0]
    out_table = block_table if out_table is None else out_table
    kv_len_out = kv_len if kv_len_out is None else kv_len_out
    acc_out = acc if acc_out is None else acc_out
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be [num_pages, page_size, kv_heads, dim]")
    _shape(v_pages, k_pages.shape, "v_pages")
    _shape(block_table, (B, block_table.shape[-1]), "block_table")
    _shape(out_table, (B, out_table.shape[-1]), "out_table")
    _shape(kv_len, (B,), "kv_len")
    _shape(kv_len_out, (B,), "kv_len_out")
    _shape(acc, (B, acc.shape[-1]), "acc")
    _shape(acc_out, acc.shape, "acc_out")
    _shape(keep, (B, budget), "keep")
    n, ps, KV, D = k_pages.shape
    a = _struct(PagedEvictArgs, _ptr(k_pages, bf16, "k_pages"), _ptr(v_pages, bf16, "v_pages", True),
                _ptr(block_table, i32, "block_table"), _ptr(out_table, i32, "out_table"),
                _ptr(kv_len, i32, "kv_len"), _ptr(kv_len_out, i32, "kv_len_out"), _ptr(acc, f32, "acc"),
                _ptr(acc_out, f32, "acc_out"), _ptr(keep, i32, "keep"), B, KV, D, ps, n, block_table.shape[1],
                out_table.shape[1], acc.shape[1], budget, recent)
    return _held(a, k_pages, v_pages, block_table, out_table, kv_len, kv_len_out, acc, acc_out, keep)


def dsv4_paged_evict_workspace_size(args):
    return int(library().dsv4_paged_evict_workspace_size(ctypes.byref(args)))


def dsv4_paged_evict(args, ws, *, stream=None):
    """Eviction by accumulated weight, from a paged_evict_args struct."""
    _call(library().dsv4_paged_evict, args, stream, "dsv4_paged_evict", ws)


def paged_plan_args(new_len, kv_len, held, block_table, free_pages, free_count, cu_q, slots, *, page_size,
                    num_pages, shared=None, pos=None, seq=None, next_pos=None, kv_len_out=None, held_out=None,
                    free_count_out=None, next_pos_out=None):
    """A step's offsets, slots and pages from its lengths: new_len (or None: pages are only given back), kv_len, held
    (and shared) int32 [B], block_table int32 [B, max_pages], free_pages int32 [capacity] with free_count int32 [1] of
    them in use -> cu_q int32 [B + 1], slots int64 [T], and, where given, pos int64 [T] (from next_pos int64 [B], else
    kv_len) and seq int32 [T]. kv_len_out, held_out, free_count_out and next_pos_out default to the arrays they follow
    (in place)."""
    bf16, f32, i32, i64 = _dt()
    B = kv_len.shape[0]
    kv_len_out = kv_len if kv_len_out is None else kv_len_out
    held_out = held if held_out is None else held_out
    free_count_out = free_count if free_count_out is None else free_count_out
    if next_pos is None and next_pos_out is not None:
        raise ValueError("next_pos_out needs next_pos")
    next_pos_out = next_pos if next_pos_out is None else next_pos_out
    for t, name in ((new_len, "new_len"), (kv_len, "kv_len"), (held, "held"), (shared, "shared"), (next_pos, "next_pos"),
                    (kv_len_out, "kv_len_out"), (held_out, "held_out"), (next_pos_out, "next_pos_out")):
        _shape(t, (B,), name)
    _shape(block_table, (B, block_table.shape[-1]), "block_table")
    _shape(free_pages, (free_pages.shape[0],), "free_pages")
    _shape(free_count, (1,), "free_count")
    _shape(free_count_out, (1,), "free_count_out")
    _shape(cu_q, (B + 1,), "cu_q")
    T = slots.shape[0]
    _shape(slots, (T,), "slots")
    _shape(pos, (T,), "pos")
    _shape(seq, (T,), "seq")
    a = _struct(PagedPlanArgs, _ptr(new_len, i32, "new_len", True), _ptr(kv_len, i32, "kv_len"), _ptr(held, i32, "held"),
                _ptr(shared, i32, "shared", True), _ptr(next_pos, i64, "next_pos", True), _ptr(block_table, i32, "block_table"),
                _ptr(free_pages, i32, "free_pages"), _ptr(free_count, i32, "free_count"), _ptr(cu_q, i32, "cu_q"),
                _ptr(kv_len_out, i32, "kv_len_out"), _ptr(held_out, i32, "held_out"),
                _ptr(next_pos_out, i64, "next_pos_out", True), _ptr(free_count_out, i32, "free_count_out"),
                _ptr(slots, i64, "slots"), _ptr(pos, i64, "pos", True), _ptr(seq, i32, "seq", True), B, T, page_size,
                num_pages, block_table.shape[1], free_pages.shape[0])
    return _held(a, new_len, kv_len, held, shared, next_pos, block_table, free_pages, free_count, cu_q, kv_len_out, held_out,
                 next_pos_out, free_count_out, slots, pos, seq)


def dsv4_paged_plan_workspace_size(args):
    return int(library().dsv4_paged_plan_workspace_size(ctypes.byref(args)))


def dsv4_paged_plan(args, ws, *, stream=None):
    """The bookkeeping of a step, from a paged_plan_args struct."""
    _call(library().dsv4_paged_plan, args, stream, "dsv4_paged_plan", ws)


ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "turns": 2, "index": 3}


def rope_args(q, q_out, pos, *, k=None, k_out=None, v=None, v_out=None, slots=None, rope_dim, first=None,
              layout="interleaved", inverse=False, rope_theta=10000.0, scaling="none", factor=1.0, original_len=0,
              beta_fast=32.0, beta_slow=1.0, magnitude=1.0):
    """Rotate q [T, H, D] -> q_out and k [T, KV, D] -> k_out [T, KV, D], all bf16, fp16 or fp32, or, with slots int64 [T],
    to rows of a pool k_out [pages, page_size, KV, D] (v beside it, unchanged). pos int64 [T]. The channels first ..
    first + rope_dim (default: the last) turn; layout: "interleaved" (2j, 2j + 1) or "half" (j, j + rope_dim / 2);
    scaling: "none", "linear", "turns" or "index". inverse=True turns back (and is the backward pass). q or k may be
    None; in place: q_out is q, k_out is k."""
    import torch
    bf16, f32, i32, i64 = _dt()
    some = q if q is not None else k
    if some is None:
        raise ValueError("q or k is required")
    types = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    if some.dtype not in types:
        raise TypeError(f"q and k must be bf16, fp16 or fp32, got {some.dtype}")
    if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
        raise ValueError(f"layout is one of {list(ROPE_LAYOUTS)}, scaling one of {list(ROPE_SCALINGS)}")
    dt = some.dtype
    T, _, D = some.shape
    H = 0 if q is None else q.shape[1]
    KV = 0 if k is None else k.shape[1]
    _shape(q, (T, H, D), "q")
    _shape(q_out, (T, H, D), "q_out")
    _shape(k, (T, KV, D), "k")
    _shape(v, (T, KV, D), "v")
    _shape(pos, (T,), "pos")
    _shape(slots, (T,), "slots")
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or (v is None) != (v_out is None):
        raise ValueError("q, k and v need their outputs")
    if v is not None and slots is None:
        raise ValueError("v is only stored by slots")
    pages = page_size = 0
    if slots is not None:
        if k is None or k_out.dim() != 4:
            raise ValueError("slots need k and a pool k_out [num_pages, page_size, kv_heads, dim]")
        pages, page_size = k_out.shape[:2]
        _shape(k_out, (pages, page_size, KV, D), "k_out")
        _shape(v_out, k_out.shape, "v_out")
        kop, kos = _ptr(k_out, dt, "k_out"), 0
    else:
        _shape(k_out, (T, KV, D), "k_out")
        kop, kos = _heads_ptr(k_out, "k_out", True, dt)
    qp, qs = _heads_ptr(q, "q", True, dt)
    op, os_ = _heads_ptr(q_out, "q_out", True, dt)
    kp, ks = _heads_ptr(k, "k", True, dt)
    vp, vs = _heads_ptr(v, "v", True, dt)
    a = _struct(RopeArgs, qp, kp, vp, op, kop, _ptr(v_out, dt, "v_out", True), _ptr(slots, i64, "slots", True),
                _ptr(pos, i64, "pos"), qs, ks, vs, os_, kos, T, H, KV, D, page_size, pages, types[dt], rope_dim,
                D - rope_dim if first is None else first, ROPE_LAYOUTS[layout], int(bool(inverse)), ROPE_SCALINGS[scaling],
                rope_theta, factor, original_len, beta_fast, beta_slow, magnitude)
    return _held(a, q, q_out, pos, k, k_out, v, v_out, slots)


def dsv4_rope(args, *, stream=None):
    """Rotary positions (and the append to the pages), from a rope_args struct."""
    _call(library().dsv4_rope, args, stream, "dsv4_rope")


def paged_prefix_args(q, out, k_pages, block_table, cu_q, kv_len, prefix_len, *, group_start=None, v_pages=None,
                      sink=None, lse=None, scale=None, out_rope_pos=None, out_rope_dim=64, out_rope_theta=10000.0):
    """q, out, pages, table, lengths and options as paged_attn_args; prefix_len int32 [groups]: the rows that the
    sequences group_start[g] .. group_start[g + 1] - 1 (int32 [groups + 1]; None: one group of all) share."""
    bf16, f32, i32, i64 = _dt()
    qp, qs, T, H, D, B, n, ps, KV, mp = _paged(q, k_pages, block_table, cu_q, kv_len)
    _shape(out, (T, H, D), "out")
    _shape(v_pages, k_pages.shape, "v_pages")
    _shape(sink, (H,), "sink")
    _shape(lse, (T, H), "lse")
    _shape(out_rope_pos, (T,), "out_rope_pos")
    G = prefix_len.shape[0]
    _shape(prefix_len, (G,), "prefix_len")
    _shape(group_start, (G + 1,), "group_start")
    if group_start is None and G != 1:
        raise ValueError("several groups need group_start")
    a = _struct(PagedPrefixArgs, qp, _ptr(k_pages, bf16, "k_pages"), _ptr(v_pages, bf16, "v_pages", True),
                _ptr(block_table, i32, "block_table"), _ptr(cu_q, i32, "cu_q"), _ptr(kv_len, i32, "kv_len"),
                _ptr(prefix_len, i32, "prefix_len"), _ptr(group_start, i32, "group_start", True), _ptr(sink, f32, "sink", True),
                _ptr(out, bf16, "out"), _ptr(lse, f32, "lse", True), _ptr(out_rope_pos, i64, "out_rope_pos", True), qs, B, G, T,
                H, KV, D, ps, n, mp, 1.0 / math.sqrt(D) if scale is None else scale,
                out_rope_dim if out_rope_pos is not None else 0, out_rope_theta)
    return _held(a, q, out, k_pages, v_pages, block_table, cu_q, kv_len, prefix_len, group_start, sink, lse, out_rope_pos)


def dsv4_paged_prefix_attn_workspace_size(args):
    return int(library().dsv4_paged_prefix_attn_workspace_size(ctypes.byref(args)))


def dsv4_paged_prefix_attn(args, ws, *, stream=None):
    """Attention of the new tokens where groups of sequences share their first rows, from a paged_prefix_args struct."""
    _call(library().dsv4_paged_prefix_attn, args, stream, "dsv4_paged_prefix_attn", ws)
