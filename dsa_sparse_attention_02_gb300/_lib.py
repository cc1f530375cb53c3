"""ctypes binding of libdsa.so (include/dsa.h): argument marshalling only.

Every function here forwards torch tensors' device pointers, the host sizes and
the current CUDA stream to the C ABI and raises DsaError on a non-OK status. No
step of the DSA computation runs in Python; if libdsa.so is missing the first
call raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdsa.so")

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_CUDA = 0, 1, 2, 3
DSA_ERR_TIMEOUT, DSA_ERR_WORKSPACE, DSA_ERR_BAD_INDEX = 4, 5, 6
DSA_BF16, DSA_E4M3, DSA_I8 = 0, 1, 2

EXPORTED = (
    "dsa_indexer_scores", "dsa_indexer_scores_workspace_size",
    "dsa_topk", "dsa_topk_workspace_size",
    "dsa_sparse_mla_attend", "dsa_sparse_mla_attend_workspace_size", "dsa_sparse_mla_attend_static",
    "dsa_decode_step", "dsa_decode_step_workspace_size",
    "dsa_decode_step_bounded", "dsa_decode_step_bounded_workspace_size", "dsa_decode_step_wait_q",
    "dsa_decode_step_hist", "dsa_decode_step_hist_workspace_size",
    "dsa_cache_append", "dsa_cache_append_workspace_size",
    "dsa_indexer_prepare", "dsa_indexer_prepare_workspace_size", "dsa_stage_copy",
    "dsa_gqa_append", "dsa_gqa_append_workspace_size", "dsa_gqa_attend", "dsa_gqa_attend_workspace_size",
    "dsa_block_select", "dsa_block_select_workspace_size",
    "dsa_gqa_attend_blocks", "dsa_gqa_attend_blocks_workspace_size",
    "dsa_get_error", "dsa_clear_error", "dsa_wait_probe", "dsa_status_string", "dsa_last_error", "dsa_abi_version",
)


class DsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = ""
        if status in (DSA_ERR_CUDA, DSA_ERR_WORKSPACE):
            try:
                detail = " [" + load().dsa_last_error().decode() + "]"
            except ImportError:
                pass
        super().__init__(f"{where}: {status_string(status)} (status {status}){detail}")


class dsa_geom_t(C.Structure):
    _fields_ = [("B", C.c_int32), ("T", C.c_int32), ("max_seq_len", C.c_int32),
                ("num_pages", C.c_int32), ("page_size", C.c_int32), ("bt_stride", C.c_int32),
                ("seq_lens", C.c_void_p), ("cu_q", C.c_void_p), ("block_table", C.c_void_p)]


class dsa_step_args_t(C.Structure):
    _fields_ = [("geom", dsa_geom_t), ("topk", C.c_int32),
                ("qk_dtype", C.c_int), ("Hi", C.c_int32),
                ("q_idx", C.c_void_p), ("q_scale", C.c_void_p), ("w", C.c_void_p),
                ("idx_k_cache", C.c_void_p), ("idx_k_scale", C.c_void_p),
                ("reuse_idx", C.c_void_p), ("idx_out", C.c_void_p),
                ("kv_dtype", C.c_int), ("H", C.c_int32),
                ("q", C.c_void_p), ("kv_cache", C.c_void_p), ("sm_scale", C.c_float),
                ("out", C.c_void_p), ("lse", C.c_void_p)]


class dsa_gqa_cache_t(C.Structure):
    _fields_ = [("dtype", C.c_int), ("Hkv", C.c_int32), ("D", C.c_int32),
                ("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("k_mean", C.c_void_p), ("k_mean_scale", C.c_void_p)]


_lib = None


def load(path: str = LIB_PATH):
    """Loads libdsa.so once and declares every entry point's signature."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m dsa_sparse_attention_02_gb300.build`")
    lib = C.CDLL(path)
    P, I32, I64, SZ, F = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t, C.c_float
    G = C.POINTER(dsa_geom_t)
    S = C.POINTER(dsa_step_args_t)
    K = C.POINTER(dsa_gqa_cache_t)
    sig = {
        "dsa_indexer_scores": (C.c_int, [G, C.c_int, I32, P, P, P, P, P, P, I64, P, SZ, P]),
        "dsa_indexer_scores_workspace_size": (SZ, [G]),
        "dsa_topk": (C.c_int, [G, P, I64, I32, P, P, SZ, P]),
        "dsa_topk_workspace_size": (SZ, [G, I32]),
        "dsa_sparse_mla_attend": (C.c_int, [G, C.c_int, I32, P, P, P, I32, F, P, P, P, SZ, P]),
        "dsa_sparse_mla_attend_workspace_size": (SZ, [G, I32, I32]),
        "dsa_sparse_mla_attend_static": (C.c_int, [G, C.c_int, I32, P, P, P, I32, F, P, P, P, P]),
        "dsa_decode_step": (C.c_int, [S, P, SZ, P]),
        "dsa_decode_step_workspace_size": (SZ, [S]),
        "dsa_decode_step_bounded": (C.c_int, [S, SZ, P, SZ, P]),
        "dsa_decode_step_wait_q": (C.c_int, [S, P, P, SZ, P]),
        "dsa_decode_step_hist": (C.c_int, [S, P, SZ, P]),
        "dsa_decode_step_hist_workspace_size": (SZ, [S]),
        "dsa_decode_step_bounded_workspace_size": (SZ, [S, SZ]),
        "dsa_cache_append": (C.c_int, [G, C.c_int, P, P, C.c_int, P, P, P, P, SZ, P]),
        "dsa_cache_append_workspace_size": (SZ, [G]),
        "dsa_indexer_prepare": (C.c_int, [G, I32, I32, P, P, P, P, P, P, F, P, P, P, P, P, SZ, P]),
        "dsa_indexer_prepare_workspace_size": (SZ, [G]),
        "dsa_stage_copy": (C.c_int, [P, P, SZ, P]),
        "dsa_gqa_append": (C.c_int, [G, K, P, I64, P, I64, I32, P, I64, P, I32, P, P, P, SZ, P]),
        "dsa_gqa_append_workspace_size": (SZ, [G, K]),
        "dsa_gqa_attend": (C.c_int, [G, K, I32, P, I64, F, P, P, P, SZ, P]),
        "dsa_gqa_attend_workspace_size": (SZ, [G, K, I32]),
        "dsa_block_select": (C.c_int, [G, K, I32, P, I64, I32, I32, I32, P, P, SZ, P]),
        "dsa_block_select_workspace_size": (SZ, [G, K, I32]),
        "dsa_gqa_attend_blocks": (C.c_int, [G, K, I32, P, I64, P, I32, F, P, P, P, SZ, P]),
        "dsa_gqa_attend_blocks_workspace_size": (SZ, [G, K, I32, I32]),
        "dsa_get_error": (C.c_int, [P, P]),
        "dsa_clear_error": (C.c_int, [P, P]),
        "dsa_wait_probe": (C.c_int, [P, SZ, C.c_uint32, P]),
        "dsa_status_string": (C.c_char_p, [C.c_int]),
        "dsa_last_error": (C.c_char_p, []),
        "dsa_abi_version": (I32, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load().dsa_status_string(int(status)).decode()
    except ImportError:
        return f"status {status}"


def _ptr(t):
    """Address of a tensor of any device (None -> NULL): only for dsa_stage_copy, whose
    C side resolves and checks both ends itself."""
    return None if t is None else t.data_ptr()


def _dptr(t):
    """Address of a CUDA tensor (None -> NULL). Anything else is refused here, so that a
    host address never reaches a kernel."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"expected a CUDA tensor, got {type(t).__name__}"
                        + (f" on {t.device}" if isinstance(t, torch.Tensor) else ""))
    return t.data_ptr()


def _optr(t):
    """Address of an attention output (None -> NULL): a CUDA tensor, or a page-locked
    host tensor, which the C side resolves to its device mapping (and refuses if it has
    none). Anything else is refused here."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and not t.is_cuda and t.is_pinned():
        return t.data_ptr()
    return _dptr(t)


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _check(status: int, where: str):
    if status != DSA_OK:
        raise DsaError(status, where)


class Geometry:
    """Request geometry: device tensors plus the host sizes the C ABI needs."""

    def __init__(self, seq_lens: torch.Tensor, cu_q: torch.Tensor, block_table: torch.Tensor,
                 num_pages: int, max_seq_len: int, T: int):
        for name, t in (("seq_lens", seq_lens), ("cu_q", cu_q), ("block_table", block_table)):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous int32 tensor")
        self.seq_lens, self.cu_q, self.block_table = seq_lens, cu_q, block_table
        self.B = int(seq_lens.shape[0])
        self.T = int(T)
        self.num_pages = int(num_pages)
        self.max_seq_len = int(max_seq_len)
        self.c = dsa_geom_t(self.B, self.T, self.max_seq_len, self.num_pages, 64,
                            int(block_table.shape[1]) if block_table.dim() == 2 else 0,
                            _dptr(seq_lens), _dptr(cu_q), _dptr(block_table))

    @property
    def ref(self):
        return C.byref(self.c)


def workspace(nbytes: int, device) -> torch.Tensor:
    """A zeroed device workspace of at least `nbytes` (256-byte aligned by the allocator)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def dsa_indexer_scores_workspace_size(geom: Geometry) -> int:
    return int(load().dsa_indexer_scores_workspace_size(geom.ref))


def dsa_indexer_scores(geom: Geometry, qk_dtype: int, q_idx, q_scale, w, idx_k_cache, idx_k_scale,
                       scores: torch.Tensor, ws: torch.Tensor, stream=None):
    Hi = int(w.shape[1])
    st = load().dsa_indexer_scores(geom.ref, qk_dtype, Hi, _dptr(q_idx), _dptr(q_scale), _dptr(w),
                                   _dptr(idx_k_cache), _dptr(idx_k_scale), _dptr(scores),
                                   int(scores.stride(0)), _dptr(ws), ws.numel(), _stream(stream))
    _check(st, "dsa_indexer_scores")


def dsa_topk_workspace_size(geom: Geometry, k: int) -> int:
    return int(load().dsa_topk_workspace_size(geom.ref, int(k)))


def dsa_topk(geom: Geometry, scores: torch.Tensor, k: int, idx: torch.Tensor, ws: torch.Tensor,
             stream=None):
    st = load().dsa_topk(geom.ref, _dptr(scores), int(scores.stride(0)), int(k), _dptr(idx),
                         _dptr(ws), ws.numel(), _stream(stream))
    _check(st, "dsa_topk")


def dsa_sparse_mla_attend_workspace_size(geom: Geometry, H: int, k: int) -> int:
    return int(load().dsa_sparse_mla_attend_workspace_size(geom.ref, int(H), int(k)))


def dsa_sparse_mla_attend(geom: Geometry, kv_dtype: int, q, kv_cache, idx, k: int, sm_scale: float,
                          out, lse, ws, stream=None):
    H = int(q.shape[1])
    st = load().dsa_sparse_mla_attend(geom.ref, kv_dtype, H, _dptr(q), _dptr(kv_cache), _dptr(idx),
                                      int(k), float(sm_scale), _optr(out), _optr(lse),
                                      _dptr(ws), ws.numel(), _stream(stream))
    _check(st, "dsa_sparse_mla_attend")


def dsa_sparse_mla_attend_static(geom: Geometry, kv_dtype: int, q, kv_cache, idx, k: int,
                                 sm_scale: float, out, lse, err_word, stream=None):
    """dsa_sparse_mla_attend without a workspace, for callers that cannot allocate device
    memory at call time; its partials use the library's static per-GPU buffer. err_word
    is a device int32 (zeroed by the caller) that receives device-side errors."""
    H = int(q.shape[1])
    st = load().dsa_sparse_mla_attend_static(geom.ref, kv_dtype, H, _dptr(q), _dptr(kv_cache), _dptr(idx),
                                             int(k), float(sm_scale), _optr(out), _optr(lse),
                                             _dptr(err_word), _stream(stream))
    _check(st, "dsa_sparse_mla_attend_static")


def dsa_cache_append_workspace_size(geom: Geometry) -> int:
    return int(load().dsa_cache_append_workspace_size(geom.ref))


def dsa_cache_append(geom: Geometry, kv_dtype: int, kv_new, kv_cache, qk_dtype: int = DSA_E4M3, k_new=None,
                     idx_k_cache=None, idx_k_scale=None, ws=None, stream=None):
    """Writes the geom.T new tokens (flattened like queries) into the paged caches."""
    st = load().dsa_cache_append(geom.ref, kv_dtype, _dptr(kv_new), _dptr(kv_cache), qk_dtype, _dptr(k_new),
                                 _dptr(idx_k_cache), _dptr(idx_k_scale), _dptr(ws), ws.numel() if ws is not None else 0,
                                 _stream(stream))
    _check(st, "dsa_cache_append")


def dsa_indexer_prepare_workspace_size(geom: Geometry) -> int:
    return int(load().dsa_indexer_prepare_workspace_size(geom.ref))


def dsa_indexer_prepare(geom: Geometry, Hi: int, rope_dim: int, q_in, k_in, rope_cos, rope_sin, ln_gamma,
                        ln_beta, ln_eps: float, q_out, q_scale, idx_k_cache=None, idx_k_scale=None, ws=None,
                        stream=None):
    """RoPE + e4m3 of the indexer queries into q_out / q_scale; LayerNorm + RoPE + e4m3
    of the new tokens' keys (k_in, or None) into the paged index cache."""
    st = load().dsa_indexer_prepare(geom.ref, int(Hi), int(rope_dim), _dptr(q_in), _dptr(k_in), _dptr(rope_cos),
                                    _dptr(rope_sin), _dptr(ln_gamma), _dptr(ln_beta), float(ln_eps), _dptr(q_out),
                                    _dptr(q_scale), _dptr(idx_k_cache), _dptr(idx_k_scale), _dptr(ws),
                                    ws.numel() if ws is not None else 0, _stream(stream))
    _check(st, "dsa_indexer_prepare")


def make_step_args(geom: Geometry, topk: int, *, qk_dtype=DSA_E4M3, q_idx=None, q_scale=None,
                   w=None, idx_k_cache=None, idx_k_scale=None, reuse_idx=None, idx_out=None,
                   kv_dtype=DSA_BF16, q=None, kv_cache=None, sm_scale=1.0, out=None,
                   lse=None) -> dsa_step_args_t:
    Hi = int(w.shape[1]) if w is not None else 0
    H = int(q.shape[1]) if q is not None else 0
    return dsa_step_args_t(geom.c, int(topk), int(qk_dtype), Hi, _dptr(q_idx), _dptr(q_scale),
                           _dptr(w), _dptr(idx_k_cache), _dptr(idx_k_scale), _dptr(reuse_idx),
                           _dptr(idx_out), int(kv_dtype), H, _dptr(q), _dptr(kv_cache),
                           float(sm_scale), _optr(out), _optr(lse))


def dsa_decode_step_workspace_size(args: dsa_step_args_t) -> int:
    return int(load().dsa_decode_step_workspace_size(C.byref(args)))


def dsa_decode_step(args: dsa_step_args_t, ws: torch.Tensor, stream=None):
    st = load().dsa_decode_step(C.byref(args), _dptr(ws), ws.numel(), _stream(stream))
    _check(st, "dsa_decode_step")


def dsa_decode_step_hist_workspace_size(args: dsa_step_args_t) -> int:
    return int(load().dsa_decode_step_hist_workspace_size(C.byref(args)))


def dsa_decode_step_hist(args: dsa_step_args_t, ws: torch.Tensor, stream=None):
    """dsa_decode_step with the top-k's first radix digit counted by the indexer."""
    st = load().dsa_decode_step_hist(C.byref(args), _dptr(ws), ws.numel(), _stream(stream))
    _check(st, "dsa_decode_step_hist")


class GqaCache:
    """Handle of a grouped-query cache: codes k, v [P, Hkv, 64, D] (torch.float8_e4m3fn or
    torch.int8), their scales [P, Hkv] fp32 and, for dsa_block_select, the blocks' key
    means [P, Hkv, D] int8 with scales [P, Hkv] fp32."""

    def __init__(self, k, v, k_scale, v_scale, k_mean=None, k_mean_scale=None):
        kinds = {torch.float8_e4m3fn: DSA_E4M3, torch.int8: DSA_I8}
        if k.dtype not in kinds or k.dim() != 4 or k.shape[2] != 64:
            raise TypeError("k must be a [P, Hkv, 64, D] tensor of float8_e4m3fn or int8 codes")
        P, Hkv, _, D = k.shape
        like = {"k": (k, k.dtype, (P, Hkv, 64, D)), "v": (v, k.dtype, (P, Hkv, 64, D)),
                "k_scale": (k_scale, torch.float32, (P, Hkv)), "v_scale": (v_scale, torch.float32, (P, Hkv)),
                "k_mean": (k_mean, torch.int8, (P, Hkv, D)), "k_mean_scale": (k_mean_scale, torch.float32, (P, Hkv))}
        if (k_mean is None) != (k_mean_scale is None):
            raise TypeError("k_mean and k_mean_scale go together")
        for name, (t, dtype, shape) in like.items():
            if t is None and name in ("k_mean", "k_mean_scale"):
                continue
            if not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
            if t.device != k.device:
                raise TypeError(f"{name} is on {t.device}, k on {k.device}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.k_mean, self.k_mean_scale = k_mean, k_mean_scale
        self.Hkv, self.D, self.num_pages = int(Hkv), int(D), int(P)
        self.device, self.index = k.device, k.get_device()
        self.c = dsa_gqa_cache_t(kinds[k.dtype], self.Hkv, self.D, _dptr(k), _dptr(v), _dptr(k_scale), _dptr(v_scale),
                                 _dptr(k_mean), _dptr(k_mean_scale))
        self.ref = C.byref(self.c)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _gqa_call(geom: Geometry, cache: GqaCache, ws, stream):
    """Checks common to the grouped-query calls; the raw stream to enqueue on. (These calls
    take microseconds: on the way of a call that fits, nothing is formatted or looked up twice.)"""
    dev = cache.index
    if ws is None or not ws.is_contiguous():      # (its size goes by its elements)
        raise TypeError("ws must be a contiguous tensor, as workspace() makes it")
    if cache.num_pages < geom.num_pages:
        raise ValueError(f"the cache has {cache.num_pages} pages, the geometry {geom.num_pages}")
    if ws.get_device() != dev or geom.seq_lens.get_device() != dev or torch.cuda.current_device() != dev:
        raise ValueError(f"cache on {cache.device}, geometry on {geom.seq_lens.device}, workspace on {ws.device}: "
                         f"all must be on the current device, cuda:{torch.cuda.current_device()}")
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _heads(name, t, geom, cache, heads=None, strided=True):
    """Address and token stride of a bf16 [T, heads, D] tensor (heads of a token side by side)."""
    if t is None:
        raise TypeError(f"{name} is missing")
    sh, st, D = t.shape, t.stride(), cache.D
    if (t.dtype is _BF16 and len(sh) == 3 and sh[0] == geom.T and sh[2] == D and (heads is None or sh[1] == heads)
            and t.get_device() == cache.index):
        row = sh[1] * D
        if st[2] == 1 and (st[1] == D or sh[1] == 1) and (st[0] == row or strided or sh[0] <= 1):
            return t.data_ptr(), (st[0] if sh[0] > 1 else row)
        raise TypeError(f"{name}: " + ("each token's heads must lie side by side" if strided else "must be contiguous"))
    if t.device != cache.device:
        raise ValueError(f"{name} is on {t.device}, the cache on {cache.device}")
    raise TypeError(f"{name} must be a {_BF16} tensor of shape [{geom.T}, {heads or 'H'}, {D}]")


def _plain(name, t, dtype, shape, cache):
    if t is None:
        raise TypeError(f"{name} is missing")
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == cache.index:
        return t.data_ptr()
    if t.device != cache.device:
        raise ValueError(f"{name} is on {t.device}, the cache on {cache.device}")
    raise TypeError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")


def dsa_gqa_append_workspace_size(geom: Geometry, cache: GqaCache) -> int:
    return int(load().dsa_gqa_append_workspace_size(geom.ref, cache.ref))


def dsa_gqa_append(geom: Geometry, cache: GqaCache, k_new, v_new, q_in=None, q_out=None, rope_dim: int = 0,
                   rope_cos=None, rope_sin=None, ws=None, stream=None):
    """Rotates the new tokens' keys (and queries into q_out), quantises keys and values
    into the cache's blocks and refreshes the blocks' means."""
    if (q_in is None) != (q_out is None):
        raise TypeError("q_in and q_out go together")
    st = _gqa_call(geom, cache, ws, stream)
    k, ks = _heads("k_new", k_new, geom, cache, cache.Hkv)
    v, vs = _heads("v_new", v_new, geom, cache, cache.Hkv)
    H, q, qs, qo = 0, None, 0, None
    if q_in is not None:
        H = q_in.shape[1]
        q, qs = _heads("q_in", q_in, geom, cache)
        qo, _ = _heads("q_out", q_out, geom, cache, H, False)
    cos = sin = None
    if rope_dim:
        table = (geom.max_seq_len, rope_dim // 2)
        cos = _plain("rope_cos", rope_cos, _F32, table, cache)
        sin = _plain("rope_sin", rope_sin, _F32, table, cache)
    s = load().dsa_gqa_append(geom.ref, cache.ref, k, ks, v, vs, H, q, qs, qo, rope_dim, cos, sin, ws.data_ptr(),
                              ws.numel(), st)
    if s:
        raise DsaError(s, "dsa_gqa_append")


def dsa_gqa_attend_workspace_size(geom: Geometry, cache: GqaCache, H: int) -> int:
    return int(load().dsa_gqa_attend_workspace_size(geom.ref, cache.ref, int(H)))


def dsa_gqa_attend(geom: Geometry, cache: GqaCache, q, sm_scale: float, out, lse, ws, stream=None):
    """Causal grouped-query attention of q [T, H, D] over the whole context into out
    [T, H, D] bf16 and lse [T, H] fp32 (or None)."""
    st = _gqa_call(geom, cache, ws, stream)
    H = q.shape[1]
    qp, qs = _heads("q", q, geom, cache)
    o, _ = _heads("out", out, geom, cache, H, False)
    le = None if lse is None else _plain("lse", lse, _F32, (geom.T, H), cache)
    s = load().dsa_gqa_attend(geom.ref, cache.ref, H, qp, qs, sm_scale, o, le, ws.data_ptr(), ws.numel(), st)
    if s:
        raise DsaError(s, "dsa_gqa_attend")


def dsa_block_select_workspace_size(geom: Geometry, cache: GqaCache, n_sel: int) -> int:
    return int(load().dsa_block_select_workspace_size(geom.ref, cache.ref, int(n_sel)))


def dsa_block_select(geom: Geometry, cache: GqaCache, q, n_sel: int, n_first: int, n_last: int, blocks, ws, stream=None):
    """The n_sel blocks of each (token, key head) that score best by their means, the first
    n_first and last n_last visible ones always among them, into blocks [T, Hkv, n_sel]."""
    st = _gqa_call(geom, cache, ws, stream)
    qp, qs = _heads("q", q, geom, cache)
    bp = _plain("blocks", blocks, _I32, (geom.T, cache.Hkv, n_sel), cache)
    s = load().dsa_block_select(geom.ref, cache.ref, q.shape[1], qp, qs, n_sel, n_first, n_last, bp, ws.data_ptr(),
                                ws.numel(), st)
    if s:
        raise DsaError(s, "dsa_block_select")


def dsa_gqa_attend_blocks_workspace_size(geom: Geometry, cache: GqaCache, H: int, n_sel: int) -> int:
    return int(load().dsa_gqa_attend_blocks_workspace_size(geom.ref, cache.ref, int(H), int(n_sel)))


def dsa_gqa_attend_blocks(geom: Geometry, cache: GqaCache, q, blocks, sm_scale: float, out, lse, ws, stream=None):
    """dsa_gqa_attend over the listed blocks [T, Hkv, n_sel] of each (token, key head)."""
    st = _gqa_call(geom, cache, ws, stream)
    H, n = q.shape[1], blocks.shape[-1]
    qp, qs = _heads("q", q, geom, cache)
    bp = _plain("blocks", blocks, _I32, (geom.T, cache.Hkv, n), cache)
    o, _ = _heads("out", out, geom, cache, H, False)
    le = None if lse is None else _plain("lse", lse, _F32, (geom.T, H), cache)
    s = load().dsa_gqa_attend_blocks(geom.ref, cache.ref, H, qp, qs, bp, n, sm_scale, o, le, ws.data_ptr(), ws.numel(), st)
    if s:
        raise DsaError(s, "dsa_gqa_attend_blocks")


def dsa_stage_copy(dst, src, nbytes: int, stream=None):
    """Copies nbytes from src to dst (device tensors or pinned host tensors) with the SMs."""
    st = load().dsa_stage_copy(_ptr(dst), _ptr(src), int(nbytes), _stream(stream))
    _check(st, "dsa_stage_copy")


def dsa_decode_step_wait_q(args: dsa_step_args_t, q_ready: torch.cuda.Event, ws: torch.Tensor, stream=None):
    """dsa_decode_step whose attention waits on q_ready (the MLA query's copy)."""
    ev = None if q_ready is None else C.c_void_p(q_ready.cuda_event)
    st = load().dsa_decode_step_wait_q(C.byref(args), ev, _dptr(ws), ws.numel(), _stream(stream))
    _check(st, "dsa_decode_step_wait_q")


def dsa_decode_step_bounded_workspace_size(args: dsa_step_args_t, score_budget_bytes: int) -> int:
    return int(load().dsa_decode_step_bounded_workspace_size(C.byref(args), int(score_budget_bytes)))


def dsa_decode_step_bounded(args: dsa_step_args_t, score_budget_bytes: int, ws: torch.Tensor, stream=None):
    """dsa_decode_step holding the scores of at most score_budget_bytes // (stride * 4)
    queries at a time; bitwise the same results."""
    st = load().dsa_decode_step_bounded(C.byref(args), int(score_budget_bytes), _dptr(ws), ws.numel(), _stream(stream))
    _check(st, "dsa_decode_step_bounded")


def dsa_get_error(ws: torch.Tensor, stream=None) -> int:
    return int(load().dsa_get_error(_dptr(ws), _stream(stream)))


def dsa_clear_error(ws: torch.Tensor, stream=None):
    _check(load().dsa_clear_error(_dptr(ws), _stream(stream)), "dsa_clear_error")


def dsa_wait_probe(ws: torch.Tensor, limit_us: int, stream=None):
    """Enqueues a wait that nothing completes, bounded by limit_us; the kernel records
    DSA_ERR_TIMEOUT in ws's error word (read it with dsa_get_error)."""
    _check(load().dsa_wait_probe(_dptr(ws), ws.numel(), int(limit_us), _stream(stream)), "dsa_wait_probe")


def dsa_abi_version() -> int:
    return int(load().dsa_abi_version())
