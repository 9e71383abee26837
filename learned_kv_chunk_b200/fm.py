"""Thin Python binding of libfm (ctypes).  Argument marshalling only: every
step of the retriever path runs in the library's CUDA kernels.  torch is used
for device memory and the current stream.

The functions carry the C ABI's names (include/fm.h); `Retriever` bundles a
context with its weights for convenience.  If libfm.so is missing, importing
this module raises: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("FM_LIBRARY_PATH") or os.path.join(_PKG, "lib", "libfm.so")

FM_OK, FM_ERR_INVALID_ARG, FM_ERR_ALIGNMENT, FM_ERR_UNSUPPORTED = 0, 1, 2, 3
FM_ERR_CUDA, FM_ERR_OOM, FM_ERR_DEVICE = 4, 5, 6
FM_ENSEMBLE_MAX, FM_ENSEMBLE_MEAN = 0, 1
MODES = {"max": FM_ENSEMBLE_MAX, "mean": FM_ENSEMBLE_MEAN}
FM_TOPK_SHARD_BINS = 2048
FM_KV4_TOKEN_BYTES = 68  # a record of the 4-bit cache: 64 code bytes and 4 scale bytes
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class fm_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("q_lora_rank", ctypes.c_int),
                ("n_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("n_layers", ctypes.c_int), ("rope_dim", ctypes.c_int),
                ("rope_base", ctypes.c_double), ("rope_factor", ctypes.c_double),
                ("rope_orig_max_pos", ctypes.c_double), ("rope_beta_fast", ctypes.c_double),
                ("rope_beta_slow", ctypes.c_double), ("rms_eps", ctypes.c_float),
                ("max_batch", ctypes.c_int), ("q_pieces", ctypes.c_int), ("cta_pairs", ctypes.c_int)]


class fm_layer_weights(ctypes.Structure):
    _fields_ = [("wq_a", ctypes.c_void_p), ("q_norm", ctypes.c_void_p),
                ("wq_b", ctypes.c_void_p), ("weights_proj", ctypes.c_void_p)]


class fm_level2_desc(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("resident_keys", ctypes.c_void_p * 4), ("resident_ids", ctypes.c_void_p),
                ("resident_count", ctypes.c_void_p), ("B", ctypes.c_int), ("R", ctypes.c_int),
                ("k", ctypes.c_int), ("mode", ctypes.c_int), ("out_ids", ctypes.c_void_p),
                ("out_count", ctypes.c_void_p)]


class fm_host_batch(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("hidden", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("comp_k", ctypes.c_void_p * 4),
                ("row_stride_bytes", ctypes.c_int64), ("n_valid", ctypes.c_void_p), ("mode", ctypes.c_int),
                ("top_k", ctypes.c_int), ("thr", ctypes.c_float), ("keep_topk", ctypes.c_void_p),
                ("keep_thr", ctypes.c_void_p)]


class fm_device_staging(ctypes.Structure):
    _fields_ = [("comp_k", ctypes.c_void_p * 4), ("hidden", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("n_valid", ctypes.c_void_p), ("q", ctypes.c_void_p), ("fused_w", ctypes.c_void_p),
                ("ens", ctypes.c_void_p), ("keep_topk", ctypes.c_void_p), ("keep_thr", ctypes.c_void_p),
                ("topk_ws", ctypes.c_void_p), ("topk_ws_bytes", ctypes.c_size_t)]


class fm_kv4_cache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("page_stride_bytes", ctypes.c_int64),
                ("head_stride_bytes", ctypes.c_int64), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("B", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("page_table_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p)]


class fm_kv4_append_desc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("T", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("q", ctypes.c_void_p), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
                ("seq", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p), ("rope_dim", ctypes.c_int), ("q_out", ctypes.c_void_p),
                ("k_hat", ctypes.c_void_p), ("v_hat", ctypes.c_void_p)]


class fm_kv4_attn_desc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("Tq", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("q", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("out", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("kv_start", ctypes.c_void_p), ("max_len", ctypes.c_int), ("idx", ctypes.c_void_p),
                ("count", ctypes.c_void_p), ("max_sel", ctypes.c_int), ("scale", ctypes.c_float),
                ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("window", ctypes.c_int)]


class FMError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.fm_strerror(status).decode() if _lib is not None else str(status)
        extra = ""
        if status == FM_ERR_CUDA:
            extra = f" (cudaError {_lib.fm_last_cuda_error()})"
        super().__init__(f"{where}: {msg}{extra}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libfm.so not built at {LIB_PATH}; run `python -m learned_kv_chunk_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    sig = {
        "fm_config_default": (None, [ctypes.POINTER(fm_config)]),
        "fm_create": (I, [ctypes.POINTER(fm_config), ctypes.POINTER(fm_layer_weights), I,
                          ctypes.POINTER(P)]),
        "fm_destroy": (I, [P]),
        "fm_query_prep": (I, [P, P, P, I, P, P, P]),
        "fm_score": (I, [P, P, I64, P, I, I, P, P, P, P]),
        "fm_ensemble": (I, [P, I, I, I, I, P, P]),
        "fm_score_fused": (I, [P, P, I64, P, I, I, P, P, I, F, P, P, P, P]),
        "fm_topk_workspace_bytes": (S, [I, I]),
        "fm_topk_workspace_bytes_fast": (S, [I, I]),
        "fm_select_topk": (I, [P, P, I, I, I, P, P, S, P]),
        "fm_select_threshold": (I, [P, P, I, I, F, P, P]),
        "fm_retrieve_host": (I, [P, ctypes.POINTER(fm_host_batch), ctypes.POINTER(fm_device_staging), P]),
        "fm_select_topk_static": (I, [P, P, I, I, I, P, P]),
        "fm_compact_workspace_bytes": (S, [I, I]),
        "fm_compact_mask": (I, [P, I, I, I, P, P, P, S, P]),
        "fm_gather_records": (I, [P, I64, I, I64, P, P, I, I, P, I64, P]),
        "fm_level2_create": (I, [P, ctypes.POINTER(fm_level2_desc), P, ctypes.POINTER(P)]),
        "fm_level2_launch": (I, [P, P]),
        "fm_level2_copy_scores": (I, [P, P, P]),
        "fm_level2_destroy": (I, [P]),
        "fm_decode_attention_workspace_bytes": (S, [I, I]),
        "fm_decode_attention": (I, [P, P, I64, I, P, P, I, I, P, P, S, P]),
        "fm_toy_decoder_update": (I, [P, P, I, I, F, P, P]),
        "fm_topk_shard_begin": (I, [P, I, I, I, P, P, S, P]),
        "fm_topk_shard_hist": (I, [P, I, I, I, P, P, S, P]),
        "fm_topk_shard_pick": (I, [I, I, I, P, P, S, P]),
        "fm_topk_shard_ties": (I, [P, I, I, P, P, S, P]),
        "fm_topk_shard_mask": (I, [P, I, I, P, I, P, P, S, P]),
        "fm_rope_frequencies": (I, [ctypes.POINTER(fm_config), P]),
        "fm_kv4_append": (I, [P, P, P]),
        "fm_kv4_attention_workspace_bytes": (S, [P, P]),
        "fm_kv4_attention": (I, [P, P, P, S, P]),
        "fm_index_append": (I, [P, I, I64, I, I, P, P, P, P, I, I, P, I64, I, I, P]),
        "fm_add_rmsnorm_fp8": (I, [P, I64, P, I64, P, I, I, I, F, I, P, P, P, P]),
        "fm_sync_status": (I, [P, P]),
        "fm_strerror": (ctypes.c_char_p, [I]),
        "fm_last_cuda_error": (I, []),
        "fm_launch_count": (ctypes.c_uint64, []),
        "fm_debug_fail_alloc": (None, [I]),
        "fm_debug_live_allocations": (I64, []),
        "fm_debug_stall_next_score": (I, [P, ctypes.c_uint64]),
        "fm_debug_tile_dots": (I, [P, P, I64, I, I, P, P, I, I, I, P, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def lib():
    return _lib


def _check(status: int, where: str):
    if status != FM_OK:
        raise FMError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fm_config_default() -> fm_config:
    c = fm_config()
    _lib.fm_config_default(ctypes.byref(c))
    return c


def fm_launch_count() -> int:
    return int(_lib.fm_launch_count())


def fm_topk_workspace_bytes(B: int, N: int) -> int:
    return int(_lib.fm_topk_workspace_bytes(B, N))


def fm_topk_workspace_bytes_fast(B: int, N: int) -> int:
    return int(_lib.fm_topk_workspace_bytes_fast(B, N))


def _comp_k_array(comp_k: Sequence[torch.Tensor]):
    for i, t in enumerate(comp_k):
        _need(t, torch.uint8, f"comp_k[{i}]")
    return (ctypes.c_void_p * len(comp_k))(*[t.data_ptr() for t in comp_k])


def _keys_shape(comp_k: Sequence[torch.Tensor], N: Optional[int]):
    B, N_pad, rec = comp_k[0].shape
    if rec != 132:
        raise ValueError("compressed keys must be [B, N, 132] uint8")
    for t in comp_k:
        if tuple(t.shape) != (B, N_pad, rec):
            raise ValueError("every layer's keys must have the same shape")
    N = N_pad if N is None else N
    return B, N, N_pad * 132


def fm_ensemble(scores: torch.Tensor, mode: str = "max", out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    _need(scores, torch.float32, "scores")
    L, B, N = scores.shape
    ens = out if out is not None else torch.empty(B, N, device=scores.device, dtype=torch.float32)
    _check(_lib.fm_ensemble(_ptr(scores), L, B, N, MODES[mode], _ptr(ens), _stream(stream)),
           "fm_ensemble")
    return ens


def fm_select_topk(ens: torch.Tensor, k: int, n_valid: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    _need(ens, torch.float32, "ens")
    B, N = ens.shape
    if n_valid is not None:
        _need(n_valid, torch.int32, "n_valid")
    keep = out if out is not None else torch.empty(B, N, device=ens.device, dtype=torch.bool)
    nbytes = fm_topk_workspace_bytes_fast(B, N)
    ws = workspace if workspace is not None else torch.empty(nbytes, device=ens.device, dtype=torch.uint8)
    _check(_lib.fm_select_topk(_ptr(ens), _ptr(n_valid), B, N, int(k), _ptr(keep), _ptr(ws),
                               ws.numel(), _stream(stream)), "fm_select_topk")
    return keep


def fm_select_topk_static(ens: torch.Tensor, k: int, n_valid: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fm_select_topk without a workspace: the library's fixed scratch array
    is used, so the C call allocates nothing (for callers that cannot
    allocate device memory).  Pass `out` to allocate nothing here either."""
    _need(ens, torch.float32, "ens")
    B, N = ens.shape
    if n_valid is not None:
        _need(n_valid, torch.int32, "n_valid")
    keep = out if out is not None else torch.empty(B, N, device=ens.device, dtype=torch.bool)
    _check(_lib.fm_select_topk_static(_ptr(ens), _ptr(n_valid), B, N, int(k), _ptr(keep),
                                      _stream(stream)), "fm_select_topk_static")
    return keep


def fm_select_threshold(ens: torch.Tensor, thr: float, n_valid: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _need(ens, torch.float32, "ens")
    B, N = ens.shape
    if n_valid is not None:
        _need(n_valid, torch.int32, "n_valid")
    keep = out if out is not None else torch.empty(B, N, device=ens.device, dtype=torch.bool)
    _check(_lib.fm_select_threshold(_ptr(ens), _ptr(n_valid), B, N, float(thr), _ptr(keep),
                                    _stream(stream)), "fm_select_threshold")
    return keep


def fm_compact_mask(keep: torch.Tensor, max_sel: int, idx: Optional[torch.Tensor] = None,
                    count: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None):
    """Keep mask [B, N] (bool or uint8, device) -> (idx [B, max_sel] int32, kept
    chunk indices in increasing order then -1; count [B] int32)."""
    if keep.dtype not in (torch.bool, torch.uint8):
        raise ValueError("keep must be bool or uint8")
    if not keep.is_cuda or not keep.is_contiguous():
        raise ValueError("keep must be a contiguous CUDA tensor")
    B, N = keep.shape
    dev = keep.device
    idx = idx if idx is not None else torch.empty(B, max_sel, device=dev, dtype=torch.int32)
    count = count if count is not None else torch.empty(B, device=dev, dtype=torch.int32)
    _need(idx, torch.int32, "idx")
    _need(count, torch.int32, "count")
    nbytes = int(_lib.fm_compact_workspace_bytes(B, N))
    ws = workspace if workspace is not None else torch.empty(nbytes, device=dev, dtype=torch.uint8)
    _check(_lib.fm_compact_mask(_ptr(keep), B, N, int(max_sel), _ptr(idx), _ptr(count), _ptr(ws), ws.numel(),
                                _stream(stream)), "fm_compact_mask")
    return idx, count


def fm_gather_records(src: torch.Tensor, idx: torch.Tensor, count: torch.Tensor,
                      dst: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Resident buffer [B, max_sel, rec] (uint8, device): slot j of row b holds
    record idx[b, j] of src[b] for j < min(count[b], max_sel); other slots are
    left as they were (zeros in a new buffer).  src [B, n_src, rec] uint8 on
    the device or in pinned host memory."""
    if src.dtype != torch.uint8 or src.dim() != 3 or not src.is_contiguous():
        raise ValueError("src must be a contiguous uint8 tensor [B, n_src, rec]")
    if not src.is_cuda and not src.is_pinned():
        raise ValueError("src must be on the device or in pinned host memory")
    _need(idx, torch.int32, "idx")
    _need(count, torch.int32, "count")
    B, n_src, rec = src.shape
    max_sel = idx.shape[1]
    if dst is None:
        dst = torch.zeros(B, max_sel, rec, device=idx.device, dtype=torch.uint8)
    _need(dst, torch.uint8, "dst")
    _check(_lib.fm_gather_records(_ptr(src), n_src * rec, n_src, rec, _ptr(idx), _ptr(count), B, max_sel,
                                  _ptr(dst), dst.stride(0), _stream(stream)), "fm_gather_records")
    return dst


class Level2Step:
    """The per-step selection over a resident set, as one CUDA graph
    (fm_level2_*): query prep for the step's hidden states, scoring of the
    resident records of every layer with the ensemble, top-k, and the kept
    slots mapped to chunk ids.  The graph reads `hidden` and `positions` at
    every launch: write the next step's values into them in place
    (Level2Step.hidden.copy_(...)) and call launch().

    resident_keys: per layer [B, R, 132] uint8 (fm_gather_records' output);
    resident_ids [B, R] int32 and resident_count [B] int32 (fm_compact_mask's
    output for the resident set)."""

    def __init__(self, retriever: "Retriever", resident_keys: Sequence[torch.Tensor],
                 resident_ids: torch.Tensor, resident_count: torch.Tensor, k: int = 512, mode: str = "max",
                 stream=None):
        for i, t in enumerate(resident_keys):
            _need(t, torch.uint8, f"resident_keys[{i}]")
        _need(resident_ids, torch.int32, "resident_ids")
        _need(resident_count, torch.int32, "resident_count")
        B, R = resident_ids.shape
        dev = resident_ids.device
        cfg = retriever.cfg
        self.hidden = torch.zeros(B, cfg.hidden, device=dev, dtype=torch.float32)
        self.positions = torch.zeros(B, device=dev, dtype=torch.int64)
        self.out_ids = torch.empty(B, k, device=dev, dtype=torch.int32)
        self.out_count = torch.empty(B, device=dev, dtype=torch.int32)
        self._keep_alive = (retriever, list(resident_keys), resident_ids, resident_count)
        self.B, self.R, self.k = B, R, int(k)
        d = fm_level2_desc()
        d.hidden, d.positions = self.hidden.data_ptr(), self.positions.data_ptr()
        for l, t in enumerate(resident_keys):
            d.resident_keys[l] = t.data_ptr()
        d.resident_ids, d.resident_count = resident_ids.data_ptr(), resident_count.data_ptr()
        d.B, d.R, d.k, d.mode = B, R, int(k), MODES[mode]
        d.out_ids, d.out_count = self.out_ids.data_ptr(), self.out_count.data_ptr()
        h = ctypes.c_void_p()
        _check(_lib.fm_level2_create(retriever.handle, ctypes.byref(d), _stream(stream), ctypes.byref(h)),
               "fm_level2_create")
        self._h = h

    def launch(self, stream=None):
        _check(_lib.fm_level2_launch(self._h, _stream(stream)), "fm_level2_launch")

    def scores(self, stream=None) -> torch.Tensor:
        """The ensembled scores [B, R] of the last step (a copy)."""
        out = torch.empty(self.B, self.R, device=self.out_ids.device, dtype=torch.float32)
        _check(_lib.fm_level2_copy_scores(self._h, _ptr(out), _stream(stream)), "fm_level2_copy_scores")
        return out

    def close(self):
        if getattr(self, "_h", None):
            _lib.fm_level2_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fm_decode_attention(q: torch.Tensor, mem: torch.Tensor, idx: Optional[torch.Tensor], count: torch.Tensor,
                        out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """The toy decoder's sparse attention over the kept chunks: q [B, 32, 128]
    fp32 (the hidden state [B, 4096] viewed as 32 heads), mem [B, N, 132]
    uint8 chunk records, idx/count from fm_compact_mask; with idx None, mem
    is the resident buffer [B, max_sel, 132] of the kept records in order
    (fm_gather_records).  Returns o [B, 32, 128]."""
    _need(q, torch.float32, "q")
    _need(mem, torch.uint8, "mem")
    if idx is not None:
        _need(idx, torch.int32, "idx")
    _need(count, torch.int32, "count")
    B, n_mem, rec = mem.shape
    if rec != 132:
        raise ValueError("mem must be [B, N, 132] uint8")
    max_sel = idx.shape[1] if idx is not None else n_mem
    out = out if out is not None else torch.empty(B, 32, 128, device=q.device, dtype=torch.float32)
    nbytes = int(_lib.fm_decode_attention_workspace_bytes(B, max_sel))
    ws = workspace if workspace is not None else torch.empty(nbytes, device=q.device, dtype=torch.uint8)
    _check(_lib.fm_decode_attention(_ptr(q), _ptr(mem), n_mem * 132, n_mem, _ptr(idx), _ptr(count), B, max_sel,
                                    _ptr(out), _ptr(ws), ws.numel(), _stream(stream)), "fm_decode_attention")
    return out


def fm_toy_decoder_update(hidden: torch.Tensor, attn_out: torch.Tensor, eps: float = 1e-6,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """hidden' = RMSNorm(hidden + attn_out) (no gain); out may be hidden itself."""
    _need(hidden, torch.float32, "hidden")
    _need(attn_out, torch.float32, "attn_out")
    B, H = hidden.shape
    out = out if out is not None else torch.empty_like(hidden)
    _check(_lib.fm_toy_decoder_update(_ptr(hidden), _ptr(attn_out), B, H, float(eps), _ptr(out),
                                      _stream(stream)), "fm_toy_decoder_update")
    return out


class ToySparseDecoder:
    """The README's toy decode loop ("Toy inference reference") on synthetic
    inputs: every `interval` (64) steps the retriever scores all chunks of the
    three layers for the current hidden state and the keep mask (top-K, or
    sigmoid > threshold) is compacted into index lists; every step the toy
    decoder attends over the kept chunks of the memory layer and updates its
    hidden state (fm_decode_attention, fm_toy_decoder_update).  Positions
    advance by one token per step from `positions`."""

    def __init__(self, retriever: "Retriever", comp_k: Sequence[torch.Tensor], n_valid: torch.Tensor,
                 hidden: torch.Tensor, positions: torch.Tensor, top_k: Optional[int] = 512,
                 threshold: Optional[float] = None, mode: str = "max", interval: int = 64,
                 memory_layer: int = 0):
        if (top_k is None) == (threshold is None):
            raise ValueError("give exactly one of top_k and threshold")
        self.r, self.comp_k, self.n_valid = retriever, list(comp_k), n_valid
        self.B, self.N = comp_k[0].shape[0], comp_k[0].shape[1]
        dev = hidden.device
        self.hidden = hidden.clone()
        self.positions0 = positions.detach().to("cpu", torch.int64)
        self.top_k, self.threshold, self.mode, self.interval = top_k, threshold, mode, int(interval)
        self.mem = self.comp_k[memory_layer]
        self.max_sel = int(top_k) if top_k is not None else self.N
        self.idx = torch.empty(self.B, self.max_sel, device=dev, dtype=torch.int32)
        self.count = torch.empty(self.B, device=dev, dtype=torch.int32)
        # top-K: the kept records are gathered once per retrieval into a
        # resident buffer that every step's attention reads in order
        self.resident = (torch.empty(self.B, self.max_sel, 132, device=dev, dtype=torch.uint8)
                         if top_k is not None else None)
        self.attn = torch.empty(self.B, 32, 128, device=dev, dtype=torch.float32)
        self._cws = torch.empty(int(_lib.fm_compact_workspace_bytes(self.B, self.N)), device=dev,
                                dtype=torch.uint8)
        self._aws = torch.empty(int(_lib.fm_decode_attention_workspace_bytes(self.B, self.max_sel)), device=dev,
                                dtype=torch.uint8)
        self.t = 0
        self.keep = None
        self.ens = None

    def retrieve(self):
        pos = (self.positions0 + self.t).to(self.hidden.device)
        ens, keep_topk, keep_thr = self.r.retrieve(self.hidden, self.comp_k, pos, self.n_valid, self.mode,
                                                   self.top_k, self.threshold, self.N)
        self.ens = ens
        self.keep = keep_topk if self.top_k is not None else keep_thr
        fm_compact_mask(self.keep, self.max_sel, idx=self.idx, count=self.count, workspace=self._cws)
        if self.resident is not None:
            fm_gather_records(self.mem, self.idx, self.count, self.resident)

    def attend(self):
        """The sparse attention of the current hidden state over the kept chunks."""
        if self.resident is not None:
            return fm_decode_attention(self.hidden.view(self.B, 32, 128), self.resident, None, self.count,
                                       out=self.attn, workspace=self._aws)
        return fm_decode_attention(self.hidden.view(self.B, 32, 128), self.mem, self.idx, self.count,
                                   out=self.attn, workspace=self._aws)

    def step(self):
        """One decode step; returns the new hidden state [B, 4096]."""
        if self.t % self.interval == 0:
            self.retrieve()
        self.attend()
        fm_toy_decoder_update(self.hidden, self.attn.view(self.B, -1), out=self.hidden)
        self.t += 1
        return self.hidden


class TopKShard:
    """One shard's side of the sharded top-K (fm_topk_shard_*): this shard's
    slice `ens_local` [B, N] of rows whose chunks are split over the shards in
    shard order, with its buffers (workspace, the histogram the shards sum, the
    tie count they gather, the keep mask).  The phases are called in the order
    fm_select_topk_sharded uses; the exchanges between them are the caller's."""

    def __init__(self, ens_local: torch.Tensor, k: int, n_valid_local: Optional[torch.Tensor] = None,
                 stream=None):
        _need(ens_local, torch.float32, "ens_local")
        if n_valid_local is not None:
            _need(n_valid_local, torch.int32, "n_valid_local")
        self.ens, self.k, self.n_valid, self.stream = ens_local, int(k), n_valid_local, stream
        self.B, self.N = ens_local.shape
        dev = ens_local.device
        self.ws = torch.empty(fm_topk_workspace_bytes(self.B, self.N), device=dev, dtype=torch.uint8)
        self.hist = torch.empty(self.B, FM_TOPK_SHARD_BINS, device=dev, dtype=torch.int32)
        self.eq_local = torch.empty(self.B, device=dev, dtype=torch.int32)
        self.keep = torch.empty(self.B, self.N, device=dev, dtype=torch.bool)

    def _tail(self):
        return _ptr(self.ws), self.ws.numel(), _stream(self.stream)

    def begin(self):
        _check(_lib.fm_topk_shard_begin(_ptr(self.n_valid), self.B, self.N, self.k, _ptr(self.hist),
                                        *self._tail()), "fm_topk_shard_begin")

    def hist_pass(self, p: int) -> torch.Tensor:
        """This slice's histogram of pass p, to be summed over the shards in place."""
        _check(_lib.fm_topk_shard_hist(_ptr(self.ens), self.B, self.N, p, _ptr(self.hist), *self._tail()),
               "fm_topk_shard_hist")
        return self.hist

    def pick(self, p: int):
        _check(_lib.fm_topk_shard_pick(self.B, self.N, p, _ptr(self.hist), *self._tail()),
               "fm_topk_shard_pick")

    def ties(self) -> torch.Tensor:
        """This slice's count of keys equal to the K-th, per row, to be gathered."""
        _check(_lib.fm_topk_shard_ties(_ptr(self.ens), self.B, self.N, _ptr(self.eq_local), *self._tail()),
               "fm_topk_shard_ties")
        return self.eq_local

    def mask(self, eq_all: torch.Tensor, shard: int) -> torch.Tensor:
        _need(eq_all, torch.int32, "eq_all")
        _check(_lib.fm_topk_shard_mask(_ptr(self.ens), self.B, self.N, _ptr(eq_all), int(shard),
                                       _ptr(self.keep), *self._tail()), "fm_topk_shard_mask")
        return self.keep


class TorchDistExchange:
    """The two exchanges of the sharded top-K over a torch.distributed group
    (NCCL between GPUs): a sum of the histograms and a gather of the tie counts.
    The shard index is the rank in the group."""

    def __init__(self, group=None):
        import torch.distributed as dist
        self.dist, self.group = dist, group
        self.rank = dist.get_rank(group)
        self.world = dist.get_world_size(group)

    def all_reduce_sum_(self, t: torch.Tensor):
        self.dist.all_reduce(t, op=self.dist.ReduceOp.SUM, group=self.group)

    def all_gather(self, t: torch.Tensor) -> torch.Tensor:
        t = t.contiguous()
        out = torch.empty(self.world * t.numel(), device=t.device, dtype=t.dtype)
        self.dist.all_gather_into_tensor(out, t.reshape(-1), group=self.group)
        return out.view((self.world,) + tuple(t.shape))


def fm_select_topk_sharded(ens_local: torch.Tensor, k: int, n_valid_local: Optional[torch.Tensor] = None,
                           exchange=None, shard=None) -> torch.Tensor:
    """Top-K keep mask of rows split over the ranks of a group: rank g holds the
    g-th consecutive slice of every row (`ens_local` [B, N_g]).  Returns this
    rank's slice of the mask that fm_select_topk gives on the whole rows.  Per
    pass one all-reduce of B*2048 int32, then one all-gather of B int32;
    scores never leave their GPU.  `exchange` defaults to the default
    torch.distributed group; `shard` (an object with TopKShard's phases)
    defaults to this library's kernels."""
    ex = exchange if exchange is not None else TorchDistExchange()
    sh = shard if shard is not None else TopKShard(ens_local, k, n_valid_local)
    sh.begin()
    for p in range(3):
        ex.all_reduce_sum_(sh.hist_pass(p))
        sh.pick(p)
    eq_all = ex.all_gather(sh.ties())
    return sh.mask(eq_all, ex.rank)


# ------------------------------------------------- the 4-bit paged cache


def _where(stream, first, *others):
    """Where a call runs: the index of the device that all its tensors are on,
    the raw stream (the device's current one unless the caller names another)
    and, if that is another, the stream itself: the call's tensors are then
    recorded on it, so that none is handed out again while its kernels use it."""
    index = first.get_device()
    if index < 0:
        raise ValueError("the tensors must be CUDA tensors")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"the tensors must be on one device, got {first.device} and {t.device}")
    raw = torch._C._cuda_getCurrentRawStream(index)
    if stream is None or stream.cuda_stream == raw and stream.device_index == index:
        return index, raw, None
    if stream.device_index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {first.device}")
    for t in (first, *others):
        if t is not None:
            t.record_stream(stream)
    return index, stream.cuda_stream, stream


def _new(like, shape, dtype, side, zero=False):
    """A tensor on like's device, empty or of zeros; from the side
    stream's own pool where the call runs on one (its memory may then be used
    there at once) and recorded on the current stream, where the caller goes on."""
    make = like.new_zeros if zero else like.new_empty
    if side is None:
        return make(shape, dtype=dtype)
    with torch.cuda.stream(side):
        t = make(shape, dtype=dtype)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _run(index, name, fn, *args):
    """The C call with its tensors' device as the current one."""
    back = torch._C._cuda_exchangeDevice(index)
    try:
        status = fn(*args)
    finally:
        if back != index:
            torch._C._cuda_exchangeDevice(back)
    if status:
        raise FMError(status, name)


def _i32(value, name: str) -> int:
    value = int(value)
    if not -1 << 31 <= value < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits, got {value}")
    return value


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _like(t: torch.Tensor, shape, dtype, name: str):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _heads(t: torch.Tensor, T: int, name: str, dtype=None) -> int:
    """[T, heads, 128] with packed heads -> the stride between tokens, in elements."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != 128 or t.dtype not in DTYPES:
        raise ValueError(f"{name} must be [{T}, heads, 128] fp32, bf16 or fp16, got {t.dtype} {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    st = t.stride()
    if st[2] != 1 or (st[1] != 128 and shape[1] > 1):
        raise ValueError(f"the heads of a token of {name} must be packed")
    return st[0] if T > 1 else shape[1] * 128


def _kv4_cache(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor) -> fm_kv4_cache:
    shape, st = k_pages.shape, k_pages.stride()
    if k_pages.dtype != torch.uint8 or v_pages.dtype != torch.uint8 or len(shape) != 3:
        raise ValueError("the pages must be uint8 [n_pages, n_kv_heads, page_size * 68]")
    n_pages, n_heads, block = shape
    if v_pages.shape != shape or v_pages.stride() != st:
        raise ValueError("k_pages and v_pages must have the same shape and strides")
    if block % FM_KV4_TOKEN_BYTES or st[2] != 1:
        raise ValueError("a page's block must be page_size * 68 contiguous bytes")
    rows = page_table.stride()
    if page_table.dtype != torch.int32 or len(rows) != 2 or (rows[1] != 1 and page_table.shape[1] > 1):
        raise ValueError("page_table must be int32 [B, max_pages] with contiguous rows")
    B, max_pages = page_table.shape
    head = st[1] if n_heads > 1 else block
    page = st[0] if n_pages > 1 else max(n_heads * head, block)
    return fm_kv4_cache(k_pages.data_ptr(), v_pages.data_ptr(), page, head, n_pages, block // FM_KV4_TOKEN_BYTES,
                        n_heads, B, max_pages, rows[0] if B > 1 else max_pages, page_table.data_ptr())


def _check_freq(inv_freq: Optional[torch.Tensor]) -> int:
    if inv_freq is None:
        return 0
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 vector (fm_rope_frequencies)")
    return 2 * inv_freq.numel()


def fm_rope_frequencies(device=None, rope_dim: int = 64, **overrides) -> torch.Tensor:
    """Query prep's rotary frequencies (YaRN; the shipped constants unless
    overridden: rope_base, rope_factor, rope_orig_max_pos, rope_beta_fast,
    rope_beta_slow) for the append calls: float64 [rope_dim / 2] on `device`
    (the host without one)."""
    cfg = fm_config_default()
    cfg.rope_dim = int(rope_dim)
    for k, v in overrides.items():
        if not k.startswith("rope_") or not hasattr(cfg, k):
            raise ValueError(f"unknown rotary constant {k}")
        setattr(cfg, k, v)
    f = torch.empty(max(0, int(rope_dim)) // 2, dtype=torch.float64)
    _check(_lib.fm_rope_frequencies(ctypes.byref(cfg), _ptr(f)), "fm_rope_frequencies")
    return f if device is None else f.to(device)


def fm_kv4_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                  page_table: torch.Tensor, seq: torch.Tensor, pos: torch.Tensor,
                  inv_freq: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                  q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                  k_hat: Optional[torch.Tensor] = None, v_hat: Optional[torch.Tensor] = None,
                  values: bool = False, stream=None):
    """Appends T tokens to the 4-bit paged cache: k, v [T, n_kv_heads, 128]
    (fp32, bf16 or fp16; views of one projection's output are fine), token t
    to position pos[t] (int64) of row seq[t] (int32; -1: padding).  Keys are
    rotated by pos (or `positions`) with inv_freq (fm_rope_frequencies: 32 or
    64 of them; None: no rotation).  q [T, n_q_heads, 128] is rotated into
    q_out (which may be q).  With `values` (or k_hat, v_hat) the values that
    the new records stand for come back in bf16, exactly.  Padding leaves its
    rows of every output as they were (zeros in a new one).
    k_pages, v_pages: uint8 [n_pages, n_kv_heads, page_size * 68]; page_table:
    int32 [B, max_pages].  Returns (q_out, k_hat, v_hat)."""
    cache = _kv4_cache(k_pages, v_pages, page_table)
    T = k.shape[0]
    ks, vs = _heads(k, T, "k"), _heads(v, T, "v", k.dtype)
    if k.shape[1] != k_pages.shape[1] or v.shape[1] != k_pages.shape[1]:
        raise ValueError("k and v must have the cache's heads")
    _like(seq, (T,), torch.int32, "seq")
    _like(pos, (T,), torch.int64, "pos")
    if positions is not None:
        _like(positions, (T,), torch.int64, "positions")
    rope_dim = _check_freq(inv_freq)
    index, raw, side = _where(stream, k, v, k_pages, v_pages, page_table, seq, pos, inv_freq, positions, q, q_out, k_hat,
                              v_hat)
    n_q = qs = qos = 0
    if q is not None:
        n_q, qs = q.shape[1], _heads(q, T, "q", k.dtype)
        if q_out is None:
            q_out = _new(k, (T, n_q, 128), k.dtype, side, zero=True)
        qos = _heads(q_out, T, "q_out", k.dtype)
        if q_out.shape[1] != n_q:
            raise ValueError("q_out must have q's shape")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if values and k_hat is None:
        k_hat = _new(k, k.shape, torch.bfloat16, side, zero=True)
    if values and v_hat is None:
        v_hat = _new(k, k.shape, torch.bfloat16, side, zero=True)
    if k_hat is not None:
        _like(k_hat, k.shape, torch.bfloat16, "k_hat")
    if v_hat is not None:
        _like(v_hat, k.shape, torch.bfloat16, "v_hat")
    if T == 0:
        return q_out, k_hat, v_hat
    d = fm_kv4_append_desc(DTYPES[k.dtype], T, n_q, k.data_ptr(), v.data_ptr(), _addr(q), ks, vs, qs, qos,
                           seq.data_ptr(), pos.data_ptr(), _addr(positions), _addr(inv_freq), rope_dim, _addr(q_out),
                           _addr(k_hat), _addr(v_hat))
    _run(index, "fm_kv4_append", _lib.fm_kv4_append, ctypes.byref(cache), ctypes.byref(d), raw)
    return q_out, k_hat, v_hat


def fm_kv4_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                     kv_len: torch.Tensor, scale: Optional[float] = None, softcap: float = 0.0,
                     slopes: Optional[torch.Tensor] = None, window: int = 0,
                     kv_start: Optional[torch.Tensor] = None, idx: Optional[torch.Tensor] = None,
                     count: Optional[torch.Tensor] = None, max_len: Optional[int] = None,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Attention of each row's newest tokens over its 4-bit paged cache:
    q [B, n_q_heads, 128] (one token a row) or [B, Tq, n_q_heads, 128] (the
    last Tq of the kv_len [B] int32 tokens, causal among themselves), fp32,
    bf16 or fp16.  scale (128^-1/2), softcap (scores capped by a tanh), slopes
    [n_q_heads] fp32 (a bias slope * (key position - query position)), window
    (positions a query sees back, itself included), kv_start [B] int32 (first
    visible position), idx / count (a list of cache positions: only those are
    read; fm_compact_mask's list of kept chunks where each token is a chunk).  max_len bounds kv_len where the caller knows it.
    Returns the output in q's type and shape; 0 for a query that sees nothing."""
    window, max_len = _i32(window, "window"), None if max_len is None else _i32(max_len, "max_len")
    shape, st = q.shape, q.stride()
    if len(shape) not in (3, 4) or shape[-1] != 128 or q.dtype not in DTYPES:
        raise ValueError("q must be [B, heads, 128] or [B, Tq, heads, 128] fp32, bf16 or fp16")
    B, Tq, n_q = shape[0], 1 if len(shape) == 3 else shape[1], shape[-2]
    if st[-1] != 1 or (n_q > 1 and st[-2] != 128):
        raise ValueError("the heads of a token of q must be packed")
    if Tq > 1:
        qs = st[1]
        if B > 1 and st[0] != Tq * qs:
            raise ValueError("the tokens of q must be evenly spaced")
    else:
        qs = st[0] if B > 1 else n_q * 128
    cache = _kv4_cache(k_pages, v_pages, page_table)
    if page_table.shape[0] != B:
        raise ValueError("page_table must have a row for each of q's")
    _like(kv_len, (B,), torch.int32, "kv_len")
    if kv_start is not None:
        _like(kv_start, (B,), torch.int32, "kv_start")
    if slopes is not None:
        _like(slopes, (n_q,), torch.float32, "slopes")
    max_sel = 0
    if idx is not None:
        if idx.dim() != 2 or count is None:
            raise ValueError("idx must be int32 [B, max_sel], with count")
        max_sel = _i32(idx.shape[1], "the entries of idx")
        _like(idx, (B, max_sel), torch.int32, "idx")
        _like(count, (B,), torch.int32, "count")
    elif count is not None:
        raise ValueError("count without idx")
    index, raw, side = _where(stream, q, k_pages, v_pages, page_table, kv_len, slopes, kv_start, idx, count, out,
                              workspace)
    if out is None:
        out = _new(q, q.shape, q.dtype, side)
    else:
        _like(out, q.shape, q.dtype, "out")
    if out.numel() == 0:
        return out
    if idx is not None and max_sel == 0:
        raise ValueError("idx has no entries")
    bound = cache.max_pages * cache.page_size if max_len is None else max_len
    d = fm_kv4_attn_desc(DTYPES[q.dtype], Tq, n_q, q.data_ptr(), qs, out.data_ptr(), kv_len.data_ptr(),
                         _addr(kv_start), bound, _addr(idx), _addr(count), max_sel,
                         128 ** -0.5 if scale is None else float(scale), float(softcap), _addr(slopes), window)
    rc, rd = ctypes.byref(cache), ctypes.byref(d)
    if workspace is None:
        workspace = _new(q, max(16, _lib.fm_kv4_attention_workspace_bytes(rc, rd)), torch.uint8, side)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    _run(index, "fm_kv4_attention", _lib.fm_kv4_attention, rc, rd, workspace.data_ptr(), workspace.numel(), raw)
    return out


def fm_index_append(k: torch.Tensor, comp_k: Sequence[torch.Tensor], row: torch.Tensor, chunk: torch.Tensor,
                    inv_freq: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                    hadamard: bool = True, N: Optional[int] = None, stream=None) -> None:
    """Appends indexer keys as the records that fm_score reads: k [T, L, 128]
    (fp32, bf16 or fp16), rotated by `positions` (int64 [T]) with inv_freq and
    Hadamard-transformed, into record chunk[t] of row row[t] (both int32; -1:
    padding) of each layer's comp_k [B, N_pad, 132] uint8."""
    T, L = k.shape[0], len(comp_k)
    ks = _heads(k, T, "k")
    if L < 1 or k.shape[1] != L:
        raise ValueError("k must hold a key for each layer of comp_k")
    B, N_pad, rec = comp_k[0].shape
    for i, t in enumerate(comp_k):
        if rec != 132:
            raise ValueError("compressed keys must be [B, N, 132] uint8")
        _like(t, (B, N_pad, rec), torch.uint8, f"comp_k[{i}]")
    _like(row, (T,), torch.int32, "row")
    _like(chunk, (T,), torch.int32, "chunk")
    rope_dim = _check_freq(inv_freq)
    if (inv_freq is None) != (positions is None):
        raise ValueError("positions and inv_freq belong together")
    if positions is not None:
        _like(positions, (T,), torch.int64, "positions")
    N = N_pad if N is None else _i32(N, "N")
    if N > N_pad:
        raise ValueError("N exceeds the rows of comp_k")
    index, raw, _ = _where(stream, k, *comp_k, row, chunk, inv_freq, positions)
    if T == 0 or N == 0 or B == 0:
        return
    arr = (ctypes.c_void_p * L)(*[t.data_ptr() for t in comp_k])
    _run(index, "fm_index_append", _lib.fm_index_append, k.data_ptr(), DTYPES[k.dtype], ks, T, L, row.data_ptr(),
         chunk.data_ptr(), _addr(positions), _addr(inv_freq), rope_dim, 1 if hadamard else 0, arr, N_pad * 132, B, N, raw)


def fm_add_rmsnorm_fp8(x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                       gain: Optional[torch.Tensor] = None, eps: float = 1e-6, group: int = 128,
                       sum_out: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
                       scales: Optional[torch.Tensor] = None, stream=None):
    """z = x + residual; RMSNorm(z) * gain in e4m3 with an fp32 scale for each
    `group` (128, or H: one a row) elements.  x, residual [T, H] fp32, bf16 or
    fp16 (rows may be strided).  Returns (z in x's type, codes [T, H]
    float8_e4m3fn, scales [T, H / group]); sum_out may be x or residual."""
    if x.dim() != 2 or x.dtype not in DTYPES or x.stride(1) != 1:
        raise ValueError("x must be [T, H] fp32, bf16 or fp16 with contiguous rows")
    T, H = x.shape
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype or residual.stride(1) != 1):
        raise ValueError("residual must have x's shape and type")
    if gain is not None:
        _like(gain, (H,), x.dtype, "gain")
    group = int(group)
    if group < 1 or H % group:
        raise ValueError("group must be 128 or H")
    index, raw, side = _where(stream, x, residual, gain, sum_out, codes, scales)
    if sum_out is None:
        sum_out = _new(x, (T, H), x.dtype, side)
    else:
        _like(sum_out, (T, H), x.dtype, "sum_out")
    if codes is None:
        codes = _new(x, (T, H), torch.float8_e4m3fn, side)
    else:
        _like(codes, (T, H), codes.dtype if codes.dtype == torch.uint8 else torch.float8_e4m3fn, "codes")
    if scales is None:
        scales = _new(x, (T, H // group), torch.float32, side)
    else:
        _like(scales, (T, H // group), torch.float32, "scales")
    if T == 0:
        return sum_out, codes, scales
    rs = 0 if residual is None else residual.stride(0) if T > 1 else H
    _run(index, "fm_add_rmsnorm_fp8", _lib.fm_add_rmsnorm_fp8, x.data_ptr(), x.stride(0) if T > 1 else H,
         _addr(residual), rs, _addr(gain), DTYPES[x.dtype], T, H, float(eps), group, sum_out.data_ptr(),
         codes.data_ptr(), scales.data_ptr(), raw)
    return sum_out, codes, scales


class Retriever:
    """A libfm context: the three CSA layers' weights on one device.

    weights: list (one per layer) of dicts with fp32 tensors wq_a [R, HID],
    q_norm [R], wq_b [H*D, R], weights_proj [H, HID] (CPU or CUDA)."""

    def __init__(self, weights: List[dict], device: int = 0, max_batch: int = 64,
                 q_pieces: int = 2, **overrides):
        cfg = fm_config_default()
        cfg.n_layers = len(weights)
        cfg.max_batch = max_batch
        cfg.q_pieces = q_pieces
        for k, v in overrides.items():
            setattr(cfg, k, v)
        self.cfg = cfg
        self.device = device
        keep = []
        arr = (fm_layer_weights * len(weights))()
        for i, w in enumerate(weights):
            ts = {k: w[k].detach().to(torch.float32).contiguous() for k in
                  ("wq_a", "q_norm", "wq_b", "weights_proj")}
            keep.append(ts)
            arr[i] = fm_layer_weights(*[ts[k].data_ptr() for k in ("wq_a", "q_norm", "wq_b", "weights_proj")])
        h = ctypes.c_void_p()
        _check(_lib.fm_create(ctypes.byref(cfg), arr, device, ctypes.byref(h)), "fm_create")
        self._h = h
        self.L = cfg.n_layers

    def close(self):
        if getattr(self, "_h", None):
            _lib.fm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def fm_query_prep(self, hidden: torch.Tensor, positions: torch.Tensor, q=None, fused_w=None,
                      stream=None):
        _need(hidden, torch.float32, "hidden")
        _need(positions, torch.int64, "positions")
        B = hidden.shape[0]
        dev = hidden.device
        q = q if q is not None else torch.empty(B, self.L, 64, 128, device=dev, dtype=torch.float32)
        fused_w = fused_w if fused_w is not None else torch.empty(B, self.L, 64, device=dev, dtype=torch.float32)
        _check(_lib.fm_query_prep(self._h, _ptr(hidden), _ptr(positions), B, _ptr(q), _ptr(fused_w),
                                  _stream(stream)), "fm_query_prep")
        return q, fused_w

    def fm_score(self, comp_k: Sequence[torch.Tensor], q: torch.Tensor, fused_w: torch.Tensor,
                 n_valid: Optional[torch.Tensor] = None, N: Optional[int] = None, out=None,
                 stream=None) -> torch.Tensor:
        B, N, stride = _keys_shape(comp_k, N)
        arr = _comp_k_array(comp_k)
        _need(q, torch.float32, "q")
        _need(fused_w, torch.float32, "fused_w")
        if n_valid is not None:
            _need(n_valid, torch.int32, "n_valid")
        scores = out if out is not None else torch.empty(self.L, B, N, device=q.device, dtype=torch.float32)
        _check(_lib.fm_score(self._h, arr, stride, _ptr(n_valid), B, N, _ptr(q), _ptr(fused_w),
                             _ptr(scores), _stream(stream)), "fm_score")
        return scores

    def fm_score_fused(self, comp_k: Sequence[torch.Tensor], q: torch.Tensor, fused_w: torch.Tensor,
                       mode: str = "max", threshold: Optional[float] = None,
                       n_valid: Optional[torch.Tensor] = None, N: Optional[int] = None,
                       want_layers: bool = False, ens=None, keep_thr=None, scores=None, stream=None):
        B, N, stride = _keys_shape(comp_k, N)
        arr = _comp_k_array(comp_k)
        _need(q, torch.float32, "q")
        _need(fused_w, torch.float32, "fused_w")
        if n_valid is not None:
            _need(n_valid, torch.int32, "n_valid")
        dev = q.device
        ens = ens if ens is not None else torch.empty(B, N, device=dev, dtype=torch.float32)
        if threshold is not None and keep_thr is None:
            keep_thr = torch.empty(B, N, device=dev, dtype=torch.bool)
        if want_layers and scores is None:
            scores = torch.empty(self.L, B, N, device=dev, dtype=torch.float32)
        thr = 0.0 if threshold is None else float(threshold)
        _check(_lib.fm_score_fused(self._h, arr, stride, _ptr(n_valid), B, N, _ptr(q), _ptr(fused_w),
                                   MODES[mode], thr, _ptr(scores), _ptr(ens),
                                   _ptr(keep_thr if threshold is not None else None),
                                   _stream(stream)), "fm_score_fused")
        return ens, keep_thr, scores

    def fm_sync_status(self, stream=None):
        _check(_lib.fm_sync_status(self._h, _stream(stream)), "fm_sync_status")

    def fm_debug_tile_dots(self, comp_k, q, fused_w, layer: int, b: int, t: int, N=None):
        B, N, stride = _keys_shape(comp_k, N)
        arr = _comp_k_array(comp_k)
        out = torch.zeros((128, 192), device=q.device, dtype=torch.float32)
        e = torch.zeros(64, device=q.device, dtype=torch.int32)
        _check(_lib.fm_debug_tile_dots(self._h, arr, stride, B, N, _ptr(q), _ptr(fused_w), layer, b, t,
                                       _ptr(out), _ptr(e), _stream()), "fm_debug_tile_dots")
        return out, e

    def retrieve_from_host(self, hidden, positions, comp_k, n_valid=None, mode="max", top_k=None,
                           threshold=None, N=None, device_buffers: Optional[dict] = None, sync=True):
        """The whole path for inputs in (pinned) host memory through the C call
        fm_retrieve_host: host inputs copied to device staging buffers, query
        prep, scoring, top-K, masks copied back.  Returns (keep_topk, keep_thr)
        as host uint8 tensors (either may be None).  `device_buffers` (a dict)
        keeps the staging buffers and the host masks between calls."""
        dev = torch.device("cuda", self.device)
        buf = device_buffers if device_buffers is not None else {}
        B, N_pad, rec = comp_k[0].shape
        N = N_pad if N is None else N
        for t in list(comp_k) + [hidden, positions] + ([n_valid] if n_valid is not None else []):
            if t.is_cuda or not t.is_contiguous():
                raise ValueError("fm_retrieve_host takes contiguous host tensors")

        def dbuf(name, shape, dtype):
            d = buf.get(name)
            if d is None or tuple(d.shape) != tuple(shape) or d.dtype != dtype:
                d = buf[name] = torch.empty(shape, dtype=dtype, device=dev)
            return d

        def hbuf(name, shape):
            h = buf.get(name)
            if h is None or tuple(h.shape) != tuple(shape):
                h = buf[name] = torch.empty(shape, dtype=torch.uint8, pin_memory=True)
            return h

        st = fm_device_staging()
        for l, t in enumerate(comp_k):
            st.comp_k[l] = dbuf(f"keys{l}", t.shape, torch.uint8).data_ptr()
        st.hidden = dbuf("hidden", hidden.shape, torch.float32).data_ptr()
        st.positions = dbuf("positions", positions.shape, torch.int64).data_ptr()
        st.n_valid = dbuf("n_valid", (B,), torch.int32).data_ptr()
        st.q = dbuf("q", (B, self.L, 64, 128), torch.float32).data_ptr()
        st.fused_w = dbuf("fused_w", (B, self.L, 64), torch.float32).data_ptr()
        st.ens = dbuf("ens", (B, N), torch.float32).data_ptr()
        st.keep_topk = dbuf("keep_topk", (B, N), torch.uint8).data_ptr()
        st.keep_thr = dbuf("keep_thr", (B, N), torch.uint8).data_ptr()
        ws = dbuf("topk_ws", (fm_topk_workspace_bytes_fast(B, N),), torch.uint8)
        st.topk_ws, st.topk_ws_bytes = ws.data_ptr(), ws.numel()
        hb = fm_host_batch()
        hb.B, hb.N = B, N
        hb.hidden, hb.positions = hidden.data_ptr(), positions.data_ptr()
        for l, t in enumerate(comp_k):
            hb.comp_k[l] = t.data_ptr()
        hb.row_stride_bytes = N_pad * rec
        hb.n_valid = n_valid.data_ptr() if n_valid is not None else None
        hb.mode = MODES[mode]
        hb.top_k = int(top_k) if top_k is not None else 0
        hb.thr = 0.0 if threshold is None else float(threshold)
        out_topk = hbuf("out_topk", (B, N)) if top_k is not None else None
        out_thr = hbuf("out_thr", (B, N)) if threshold is not None else None
        hb.keep_topk = out_topk.data_ptr() if out_topk is not None else None
        hb.keep_thr = out_thr.data_ptr() if out_thr is not None else None
        _check(_lib.fm_retrieve_host(self._h, ctypes.byref(hb), ctypes.byref(st), _stream()), "fm_retrieve_host")
        if sync:
            self.fm_sync_status()
        return out_topk, out_thr

    # the pages' calls, composed (README "Usage")
    def retrieve(self, hidden, comp_k, positions, n_valid=None, mode="max", top_k=None,
                 threshold=None, N=None):
        q, w = self.fm_query_prep(hidden, positions)
        ens, keep_thr, _ = self.fm_score_fused(comp_k, q, w, mode=mode, threshold=threshold,
                                               n_valid=n_valid, N=N)
        keep_topk = fm_select_topk(ens, top_k, n_valid) if top_k is not None else None
        return ens, keep_topk, keep_thr
