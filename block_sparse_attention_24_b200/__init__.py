"""Python binding of libveda.so, the B200 (sm_100a) hot path of Veda's
distilled tile-skipping sparse attention ("Technical Summary: Veda - Scalable
Video Diffusion via Distilled Sparse Attention", sections 2.1-2.3).

Argument marshalling only: every function here passes device pointers and
sizes to the C ABI declared in include/veda.h, on the current torch CUDA
stream. There is no CPU or PyTorch fallback; if the library is missing the
import fails.
"""
from __future__ import annotations

import ctypes
import os
from array import array
from typing import Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libveda.so")

VEDA_OK = 0
VEDA_ERR_INVALID_ARG = -1
VEDA_ERR_UNSUPPORTED = -2
VEDA_ERR_CUDA = -3
VEDA_ERR_TIMEOUT = -4
VEDA_ERR_BAD_INDEX = -5

EXPORTED = ("veda_layout", "veda_permute", "veda_trippool", "veda_permute_trippool", "veda_tile_scores", "veda_tile_scores_ws_bytes",
            "veda_tile_scores_noalloc",
            "veda_topk_mask", "veda_tile_scores_topk", "veda_tile_scores_heads", "veda_topk_mask_heads", "veda_score_cache_step", "veda_score_cache_ws_bytes", "veda_sparse_attn", "veda_sparse_attn_unpermute", "veda_sparse_attn_tokens", "veda_full_attn_tilemax", "veda_full_attn_tilemax_ws_bytes", "veda_tilemap_kl", "veda_tilemap_recall",
            "veda_check_status",
            "veda_estimator_grad", "veda_estimator_grad_ws_bytes", "veda_output_sq_error", "veda_selftest_wait_timeout", "veda_last_error",
            "veda_kv_append", "veda_kv_append_pending", "veda_kv_advance", "veda_kv_attn", "veda_kv_attn_fill", "veda_kv_attn_ws_bytes", "veda_kv_evict", "veda_kv_check_status")


class VedaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"veda error {code}: {msg}")
        self.code = code


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with `python block_sparse_attention_24_b200/build.py`")
    return ctypes.CDLL(_LIB_PATH)


_lib = _load()


class _Tiling(ctypes.Structure):
    _fields_ = [("pt", ctypes.c_int32), ("ph", ctypes.c_int32), ("pw", ctypes.c_int32)]


class _Layer(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("heads", ctypes.c_int32), ("d", ctypes.c_int32), ("T", ctypes.c_int32),
                ("H", ctypes.c_int32), ("W", ctypes.c_int32), ("tile", ctypes.c_int32),
                ("tilings", ctypes.POINTER(_Tiling)), ("dev_status", ctypes.c_void_p)]


class _KvCache(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "heads_kv", "d", "tile", "n_slots", "nb_cap")] +
                [(n, ctypes.c_void_p) for n in ("k8", "v8", "table", "pos", "k_scale", "v_scale", "weight", "len",
                                                "next_pos", "arrive", "dev_status")])


class _KvTail(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("codes", "key", "scale")]


_P = ctypes.c_void_p
_I = ctypes.c_int32
_F = ctypes.c_float
_LP = ctypes.POINTER(_Layer)
_lib.veda_layout.argtypes = [_LP, _P, _P, _P, _P]
_lib.veda_permute.argtypes = [_LP, _P, _P, _P, ctypes.c_int, _P]
_lib.veda_trippool.argtypes = [_LP, _P, _P, _P]
_lib.veda_permute_trippool.argtypes = [_LP, _P, _P, _P, _P, _P]
_lib.veda_tile_scores.argtypes = [_LP] + [_P] * 10 + [_I, _I, _F, _P, _P, _P]
_lib.veda_tile_scores_noalloc.argtypes = [_LP] + [_P] * 10 + [_I, _I, _F, _P, _P]
_lib.veda_tile_scores_ws_bytes.argtypes = [_LP, _I]
_lib.veda_tile_scores_ws_bytes.restype = ctypes.c_size_t
_lib.veda_topk_mask.argtypes = [_LP, _P, _P, _I, _P, _P, _P]
_lib.veda_tile_scores_heads.argtypes = [_LP] + [_P] * 10 + [_I, _I, _F, _P, _P, _P, _P]
_lib.veda_topk_mask_heads.argtypes = [_LP, _P, _P, _I, _P, _P, _P, _P]
_lib.veda_score_cache_step.argtypes = [_LP, _P, _P, _P, _P, _F, _I, _P, _P, _P, _P]
_lib.veda_score_cache_ws_bytes.argtypes = [_LP]
_lib.veda_score_cache_ws_bytes.restype = ctypes.c_size_t
_lib.veda_tile_scores_topk.argtypes = [_LP] + [_P] * 10 + [_I, _I, _F, _P, _I, _P, _P, _P, _P, _P]
_lib.veda_sparse_attn.argtypes = [_LP, _P, _P, _P, _P, _P, _I, _F, _P, _P, _P]
_lib.veda_sparse_attn_unpermute.argtypes = [_LP, _P, _P, _P, _P, _P, _I, _F, _P, _P, _P]
_lib.veda_sparse_attn_tokens.argtypes = [_LP, _P, _P, _P, _P, _P, _I, _F, _P, _P, _P]
_lib.veda_full_attn_tilemax.argtypes = [_LP, _P, _P, _P, _I, _P, _I, _F, _P, _P, _P, _P, _P, _P, _P]
_lib.veda_full_attn_tilemax_ws_bytes.argtypes = [_LP, _I, _I]
_lib.veda_tilemap_kl.argtypes = [_LP, _P, _I, _P, _I, _P, _P, _P, _P, _P]
_lib.veda_full_attn_tilemax_ws_bytes.restype = ctypes.c_size_t
_lib.veda_tilemap_recall.argtypes = [_LP, _P, _I, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P]
_lib.veda_estimator_grad.argtypes = [_LP] + [_P] * 10 + [_I, _I, _F, _P, _I, _P, _I, _P] + [_P] * 8 + [_P, _P, _P]
_lib.veda_estimator_grad_ws_bytes.argtypes = [_LP, _I, _I, _I, _I]
_lib.veda_estimator_grad_ws_bytes.restype = ctypes.c_size_t
_lib.veda_output_sq_error.argtypes = [_LP, _P, _P, _P, _P]
_lib.veda_check_status.argtypes = [_LP, _P]
_lib.veda_selftest_wait_timeout.argtypes = [_LP, ctypes.c_uint32, _P]
_CP = ctypes.POINTER(_KvCache)
_lib.veda_kv_append.argtypes = [_CP, _P, _P, _P, _P, _I, _P, _P]
_lib.veda_kv_append_pending.argtypes = [_CP, ctypes.POINTER(_KvTail), _P, _P, _P, _P, _I, _P, _P]
_lib.veda_kv_advance.argtypes = [_CP, _I, _P, _P]
_lib.veda_kv_attn.argtypes = [_CP, _P, _P, _I, _I, _P, _I, _I, _I, _I, _F, _P, _P, _P, _P, _F, _P, _P]
_lib.veda_kv_attn_fill.argtypes = _lib.veda_kv_attn.argtypes
_lib.veda_kv_attn_ws_bytes.argtypes = [_CP, _I, _I, _I]
_lib.veda_kv_attn_ws_bytes.restype = ctypes.c_size_t
_lib.veda_kv_evict.argtypes = [_CP, _P, _I, _I, _CP, _P]
_lib.veda_kv_check_status.argtypes = [_CP, _P]
_lib.veda_last_error.restype = ctypes.c_char_p
for _name in EXPORTED:
    getattr(_lib, _name)
    if _name not in ("veda_last_error", "veda_tile_scores_ws_bytes", "veda_estimator_grad_ws_bytes",
                     "veda_full_attn_tilemax_ws_bytes", "veda_score_cache_ws_bytes",
                     "veda_kv_attn_ws_bytes"):
        getattr(_lib, _name).restype = ctypes.c_int


def veda_last_error() -> str:
    return _lib.veda_last_error().decode()


def _check(rc: int):
    if rc != VEDA_OK:
        raise VedaError(rc, veda_last_error())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libveda must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


class Layer:
    """Geometry of one attention layer (veda_layer) plus its device status
    word. `tilings` is one (p_t, p_h, p_w) per head."""

    def __init__(self, B: int, heads: int, d: int, T: int, H: int, W: int, tile: int,
                 tilings: Sequence[Tuple[int, int, int]], device=None):
        self.B, self.heads, self.d, self.T, self.H, self.W, self.tile = B, heads, d, T, H, W, tile
        self.tilings = [tuple(int(v) for v in t) for t in tilings]
        self._til = (_Tiling * max(1, heads))(*[_Tiling(*t) for t in self.tilings])
        self.status = None
        if device is not None:
            self.status = torch.zeros(4, dtype=torch.int32, device=device)
        self._c = _Layer(B, heads, d, T, H, W, tile, ctypes.cast(self._til, ctypes.POINTER(_Tiling)),
                         ctypes.c_void_p(self.status.data_ptr()) if self.status is not None else None)
        nt = (ctypes.c_int32 * max(1, heads))()
        npad = (ctypes.c_int32 * max(1, heads))()
        ncap, ntcap = ctypes.c_int32(), ctypes.c_int32()
        _check(_lib.veda_layout(ctypes.byref(self._c), nt, npad, ctypes.byref(ncap), ctypes.byref(ntcap)))
        self.nt = list(nt)[:heads]
        self.n_pad = list(npad)[:heads]
        self.n_cap = ncap.value
        self.nt_cap = ntcap.value

    @property
    def N(self) -> int:
        return self.T * self.H * self.W

    @property
    def ref(self):
        return ctypes.byref(self._c)


def veda_layout(layer: Layer):
    """(nt per head, n_pad per head, n_cap, nt_cap)."""
    return layer.nt, layer.n_pad, layer.n_cap, layer.nt_cap


def veda_permute(layer: Layer, x: torch.Tensor, xp: torch.Tensor, perm: Optional[torch.Tensor] = None,
                 inverse: bool = False, stream=None):
    _check(_lib.veda_permute(layer.ref, _ptr(x), _ptr(xp), _ptr(perm), int(inverse), _stream(stream)))


def veda_trippool(layer: Layer, xp: torch.Tensor, desc: torch.Tensor, stream=None):
    _check(_lib.veda_trippool(layer.ref, _ptr(xp), _ptr(desc), _stream(stream)))


def veda_permute_trippool(layer: Layer, x: torch.Tensor, xp: torch.Tensor, desc: torch.Tensor,
                          perm: Optional[torch.Tensor] = None, stream=None):
    _check(_lib.veda_permute_trippool(layer.ref, _ptr(x), _ptr(xp), _ptr(perm), _ptr(desc), _stream(stream)))


def veda_tile_scores_ws_bytes(layer: Layer, out_dim: int) -> int:
    return int(_lib.veda_tile_scores_ws_bytes(layer.ref, out_dim))


def veda_tile_scores(layer: Layer, dq, dk, w1q, b1q, w2q, b2q, w1k, b1k, w2k, b2k, hidden: int, out_dim: int,
                     scale: float, scores: torch.Tensor, emb_ws: torch.Tensor, stream=None):
    _check(_lib.veda_tile_scores(layer.ref, *[_ptr(t) for t in (dq, dk, w1q, b1q, w2q, b2q, w1k, b1k, w2k, b2k)],
                                 hidden, out_dim, float(scale), _ptr(scores), _ptr(emb_ws), _stream(stream)))


def veda_tile_scores_noalloc(layer: Layer, dq, dk, w1q, b1q, w2q, b2q, w1k, b1k, w2k, b2k, hidden: int,
                             out_dim: int, scale: float, scores: torch.Tensor, stream=None):
    """veda_tile_scores for callers that cannot allocate device memory: the
    embeddings go to a 16 MiB array built into the library (shared by all
    calls; overlapping calls race)."""
    _check(_lib.veda_tile_scores_noalloc(layer.ref, *[_ptr(t) for t in (dq, dk, w1q, b1q, w2q, b2q, w1k, b1k, w2k,
                                                                         b2k)],
                                         hidden, out_dim, float(scale), _ptr(scores), _stream(stream)))


def _host_i32(vals):
    arr = (ctypes.c_int32 * max(1, len(vals)))(*[int(v) for v in vals])
    return arr


def veda_topk_mask(layer: Layer, scores: torch.Tensor, k: Sequence[int], k_cap: int, idx: torch.Tensor,
                   mask: Optional[torch.Tensor] = None, stream=None):
    _check(_lib.veda_topk_mask(layer.ref, _ptr(scores), _host_i32(k), int(k_cap), _ptr(idx), _ptr(mask),
                               _stream(stream)))


def veda_tile_scores_heads(layer: Layer, dq, dk, w1q, b1q, w2q, b2q, w1k, b1k, w2k, b2k, hidden: int,
                           out_dim: int, scale: float, scores: torch.Tensor, emb_ws: torch.Tensor,
                           head_on: Optional[torch.Tensor], stream=None):
    """veda_tile_scores for the (batch element, head) pairs with head_on != 0."""
    _check(_lib.veda_tile_scores_heads(layer.ref, *[_ptr(t) for t in (dq, dk, w1q, b1q, w2q, b2q, w1k, b1k, w2k,
                                                                        b2k)],
                                       hidden, out_dim, float(scale), _ptr(scores), _ptr(emb_ws), _ptr(head_on),
                                       _stream(stream)))


def veda_topk_mask_heads(layer: Layer, scores: torch.Tensor, k: Sequence[int], k_cap: int, idx: torch.Tensor,
                         mask: Optional[torch.Tensor], head_on: Optional[torch.Tensor], stream=None):
    """veda_topk_mask for the (batch element, head) pairs with head_on != 0."""
    _check(_lib.veda_topk_mask_heads(layer.ref, _ptr(scores), _host_i32(k), int(k_cap), _ptr(idx), _ptr(mask),
                                     _ptr(head_on), _stream(stream)))


def veda_score_cache_ws_bytes(layer: Layer) -> int:
    return int(_lib.veda_score_cache_ws_bytes(layer.ref))


def veda_score_cache_step(layer: Layer, dq, dk, dq_ref, dk_ref, tau: float, max_age: int, age: torch.Tensor,
                          refresh: torch.Tensor, ws: torch.Tensor, stream=None):
    """Temporal caching of tile scores: per (batch element, head), decide on
    the device whether its cached mask is reused (refresh 0) or rebuilt."""
    _check(_lib.veda_score_cache_step(layer.ref, _ptr(dq), _ptr(dk), _ptr(dq_ref), _ptr(dk_ref), float(tau),
                                      int(max_age), _ptr(age), _ptr(refresh), _ptr(ws), _stream(stream)))


def veda_tile_scores_topk(layer: Layer, dq, dk, w1q, b1q, w2q, b2q, w1k, b1k, w2k, b2k, hidden: int, out_dim: int,
                          scale: float, k: Sequence[int], k_cap: int, idx: torch.Tensor, emb_ws: torch.Tensor,
                          mask: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None, stream=None):
    _check(_lib.veda_tile_scores_topk(layer.ref, *[_ptr(t) for t in (dq, dk, w1q, b1q, w2q, b2q, w1k, b1k, w2k, b2k)],
                                      hidden, out_dim, float(scale), _host_i32(k), int(k_cap), _ptr(idx), _ptr(mask),
                                      _ptr(scores), _ptr(emb_ws), _stream(stream)))


def veda_sparse_attn(layer: Layer, qp, kp, vp, idx: Optional[torch.Tensor], k: Optional[Sequence[int]], k_cap: int,
                     scale: float, op: torch.Tensor, lse: Optional[torch.Tensor] = None, stream=None):
    karr = _host_i32(k) if k is not None else None
    _check(_lib.veda_sparse_attn(layer.ref, _ptr(qp), _ptr(kp), _ptr(vp), _ptr(idx), karr, int(k_cap),
                                 float(scale), _ptr(op), _ptr(lse), _stream(stream)))


def veda_sparse_attn_unpermute(layer: Layer, qp, kp, vp, idx: Optional[torch.Tensor], k: Optional[Sequence[int]],
                               k_cap: int, scale: float, o: torch.Tensor, lse: Optional[torch.Tensor] = None,
                               stream=None):
    """veda_sparse_attn with the output written in token order [B, N, heads, d]."""
    karr = _host_i32(k) if k is not None else None
    _check(_lib.veda_sparse_attn_unpermute(layer.ref, _ptr(qp), _ptr(kp), _ptr(vp), _ptr(idx), karr, int(k_cap),
                                           float(scale), _ptr(o), _ptr(lse), _stream(stream)))


def veda_sparse_attn_tokens(layer: Layer, q, k, v, idx: Optional[torch.Tensor], kk: Optional[Sequence[int]],
                            k_cap: int, scale: float, o: torch.Tensor, lse: Optional[torch.Tensor] = None,
                            stream=None):
    """Sparse attention with q, k, v and o in token order [B, N, heads, d]."""
    karr = _host_i32(kk) if kk is not None else None
    _check(_lib.veda_sparse_attn_tokens(layer.ref, _ptr(q), _ptr(k), _ptr(v), _ptr(idx), karr, int(k_cap),
                                        float(scale), _ptr(o), _ptr(lse), _stream(stream)))


def veda_full_attn_tilemax(layer: Layer, qp, kp, heads_sel: Sequence[int], qtile_rows: Optional[torch.Tensor],
                           n_rows: int, scale: float, tilemap: torch.Tensor, lse: Optional[torch.Tensor] = None,
                           scores: Optional[torch.Tensor] = None, kl_rows: Optional[torch.Tensor] = None,
                           kl_out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    _check(_lib.veda_full_attn_tilemax(layer.ref, _ptr(qp), _ptr(kp), _host_i32(heads_sel), len(heads_sel),
                                       _ptr(qtile_rows), int(n_rows), float(scale), _ptr(tilemap), _ptr(lse),
                                       _ptr(scores), _ptr(kl_rows), _ptr(kl_out), _ptr(ws), _stream(stream)))


def veda_tilemap_kl(layer: Layer, heads_sel: Sequence[int], qtile_rows: Optional[torch.Tensor], n_rows: int,
                    tilemap: torch.Tensor, scores: torch.Tensor, kl_rows: torch.Tensor, kl_out: torch.Tensor,
                    stream=None):
    _check(_lib.veda_tilemap_kl(layer.ref, _host_i32(heads_sel), len(heads_sel), _ptr(qtile_rows), int(n_rows),
                                _ptr(tilemap), _ptr(scores), _ptr(kl_rows), _ptr(kl_out), _stream(stream)))


def veda_tilemap_recall(layer: Layer, heads_sel: Sequence[int], qtile_rows: Optional[torch.Tensor], n_rows: int,
                        tilemap: torch.Tensor, idx: torch.Tensor, k: Sequence[int], k_cap: int, hits: torch.Tensor,
                        recall: torch.Tensor, map_idx: Optional[torch.Tensor] = None, stream=None):
    """hits [n_heads_sel, n_rows] int32, recall [n_heads_sel + 1] fp32 (per
    head, then their mean); map_idx (optional) the map's own top-k lists."""
    _check(_lib.veda_tilemap_recall(layer.ref, _host_i32(heads_sel), len(heads_sel), _ptr(qtile_rows), int(n_rows),
                                    _ptr(tilemap), _ptr(idx), _host_i32(k), int(k_cap), _ptr(hits), _ptr(map_idx),
                                    _ptr(recall), _stream(stream)))


def veda_full_attn_tilemax_ws_bytes(layer: Layer, n_heads_sel: int, n_rows: int) -> int:
    return int(_lib.veda_full_attn_tilemax_ws_bytes(layer.ref, n_heads_sel, n_rows))


def veda_estimator_grad_ws_bytes(layer: Layer, n_heads_sel: int, n_rows: int, hidden: int, out_dim: int) -> int:
    return int(_lib.veda_estimator_grad_ws_bytes(layer.ref, n_heads_sel, n_rows, hidden, out_dim))


def veda_estimator_grad(layer: Layer, dq, dk, weights: Sequence[torch.Tensor], hidden: int, out_dim: int,
                        scale: float, heads_sel: Sequence[int], qtile_rows: Optional[torch.Tensor], n_rows: int,
                        tilemap: torch.Tensor, grads: Sequence[torch.Tensor], ws: torch.Tensor,
                        loss: Optional[torch.Tensor] = None, stream=None):
    """weights and grads: (w1q, b1q, w2q, b2q, w1k, b1k, w2k, b2k)."""
    _check(_lib.veda_estimator_grad(layer.ref, _ptr(dq), _ptr(dk), *[_ptr(t) for t in weights], hidden, out_dim,
                                    float(scale), _host_i32(heads_sel), len(heads_sel), _ptr(qtile_rows),
                                    int(n_rows), _ptr(tilemap), *[_ptr(t) for t in grads], _ptr(loss), _ptr(ws),
                                    _stream(stream)))


def veda_output_sq_error(layer: Layer, a: torch.Tensor, b: torch.Tensor, err: torch.Tensor, stream=None):
    _check(_lib.veda_output_sq_error(layer.ref, _ptr(a), _ptr(b), _ptr(err), _stream(stream)))


def veda_check_status(layer: Layer, stream=None):
    _check(_lib.veda_check_status(layer.ref, _stream(stream)))


def veda_selftest_wait_timeout(layer: Layer, limit_ms: int, stream=None):
    _check(_lib.veda_selftest_wait_timeout(layer.ref, int(limit_ms), _stream(stream)))


class KVCache:
    """An 8-bit K/V tile cache (veda_kv_cache) and the tensors it is made of:
    k8, v8 [n_slots, tile, d] float8_e4m3fn; table, pos (int32), k_scale,
    v_scale, weight (fp32) [B, heads_kv, nb_cap]; len [B, heads_kv] and
    next_pos [B] (int32). Those not given are allocated: an empty cache whose
    table names slot (b * heads_kv + h) * nb_cap + i for tile i. Tensors are
    used where they are (no copy) and are the caller's to look at and to
    change, in place, between calls. tail_codes [B, heads_kv, 2, tile, d],
    tail_key and tail_scale are the library's own: what the tail tiles were
    before pending tokens raised their scales (veda_kv_tail)."""

    _META = (("table", torch.int32), ("pos", torch.int32), ("k_scale", torch.float32), ("v_scale", torch.float32),
             ("weight", torch.float32))

    def __init__(self, B: int, heads_kv: int, d: int, tile: int, nb_cap: int, device, k8=None, v8=None, table=None,
                 pos=None, k_scale=None, v_scale=None, weight=None, len=None, next_pos=None):
        self.B, self.heads_kv, self.d, self.tile, self.nb_cap = B, heads_kv, d, tile, nb_cap
        if min(B, heads_kv, d, tile, nb_cap) < 1:
            raise ValueError("B, heads_kv, d, tile and nb_cap must be positive")
        device = torch.device(device)
        given = dict(k8=k8, v8=v8, table=table, pos=pos, k_scale=k_scale, v_scale=v_scale, weight=weight, len=len,
                     next_pos=next_pos)
        n_slots = B * heads_kv * nb_cap
        for name in ("k8", "v8"):
            if given[name] is not None:
                n_slots = given[name].shape[0]
        shape = (B, heads_kv, nb_cap)
        spec = {"k8": ((n_slots, tile, d), torch.float8_e4m3fn), "v8": ((n_slots, tile, d), torch.float8_e4m3fn),
                "len": (shape[:2], torch.int32), "next_pos": (shape[:1], torch.int32)}
        spec.update({name: (shape, dtype) for name, dtype in self._META})
        for name, (shp, dtype) in spec.items():
            t = given[name]
            if t is None:
                if name == "table":
                    if n_slots < B * heads_kv * nb_cap:
                        raise ValueError("a pool smaller than B * heads_kv * nb_cap slots needs a table")
                    t = torch.arange(B * heads_kv * nb_cap, dtype=dtype, device=device).view(shape)
                elif name in ("k8", "v8"):
                    t = torch.zeros(shp, dtype=torch.uint8, device=device).view(dtype)
                else:
                    t = torch.zeros(shp, dtype=dtype, device=device)
            _expect(t, name, shp, dtype, None)
            if device.type == "cuda" and device.index is None and t.device.type == "cuda":
                device = t.device
            if t.device != device:
                raise ValueError(f"{name} is on {t.device}, not on {device}")
            setattr(self, name, t)
        self.device = device
        self.n_slots = n_slots
        # one allocation, its parts at multiples of 16 bytes
        bh = B * heads_kv
        words = torch.zeros(4 + 13 * bh, dtype=torch.int32, device=device)
        self.status, self.tail_key = words[:4], words[4:4 + 8 * bh].view(B, heads_kv, 2, 4)
        self.tail_scale = words[4 + 8 * bh:4 + 12 * bh].view(torch.float32).view(B, heads_kv, 2, 2)
        self._arrive = words[4 + 12 * bh:]
        self.tail_codes = torch.zeros((B, heads_kv, 2, tile, d), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
        self._tail = _KvTail(self.tail_codes.data_ptr(), self.tail_key.data_ptr(), self.tail_scale.data_ptr())
        self.tail_ref = ctypes.byref(self._tail)
        self._c = _KvCache(B, heads_kv, d, tile, n_slots, nb_cap,
                           *[getattr(self, n).data_ptr() for n in ("k8", "v8", "table", "pos", "k_scale", "v_scale",
                                                                   "weight", "len", "next_pos", "_arrive",
                                                                   "status")])
        self._ws_bytes = {}  # of veda_kv_attn, by (heads, n_q, with weights)
        self.ref = ctypes.byref(self._c)

    def tensors(self):
        """All the device memory that a call on the cache may use."""
        return [getattr(self, n) for n in ("k8", "v8", "table", "pos", "k_scale", "v_scale", "weight", "len", "next_pos",
                                           "status", "tail_codes")]  # (with status all counters)

    def __setattr__(self, name, value):
        # the kernels have the tensors' addresses: another tensor would be
        # ignored, and the one they use freed
        if "ref" in self.__dict__:
            raise AttributeError(f"KVCache.{name} cannot be given another value; change the tensor in place")
        object.__setattr__(self, name, value)


def _expect(t, name: str, shape, dtype, device, contiguous: bool = True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _checked(t, name: str, shape, dtype, device) -> int:
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and
            t.is_contiguous()):
        _expect(t, name, shape, dtype, device)
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, shape, cache: KVCache):
    """Pointer and strides (None: contiguous) of a [B, n, heads, d] bf16
    tensor whose last dimension is contiguous."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.shape != shape or t.device != cache.device:
        _expect(t, name, shape, torch.bfloat16, cache.device, contiguous=False)
    if t.is_contiguous():
        return t.data_ptr(), None
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), _Strides(*[s if n > 1 else 0 for s, n in zip(st[:3], shape)])


_Strides = ctypes.c_int64 * 3


def _kv_call(cache: KVCache, stream, fn, *args):
    """fn(*args, stream pointer) on the cache's device, on `stream` or that
    device's current one."""
    index = cache.device.index
    if index is None:
        raise ValueError("the cache is not on a CUDA device")
    if stream is not None and stream.device != cache.device:
        raise ValueError(f"the stream is on {stream.device}, the cache on {cache.device}")
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc != VEDA_OK:
        _check(rc)


def _i32(x, name: str) -> int:
    """x as the calls take it; ctypes would drop the bits above."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name}={x} does not fit 32 bits")
    return x


def _n_new(cache: KVCache, n_new):
    return None if n_new is None else _checked(n_new, "n_new", (cache.B,), torch.int32, cache.device)


def veda_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, n_new: Optional[torch.Tensor] = None,
                   stream=None):
    """K and V [B, n, heads_kv, d] of n new tokens into the cache, as pending
    tokens behind those it holds (n_new [B]: how many of each sequence's rows
    are real), in the place of those that are pending."""
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a [B, n, heads_kv, d] tensor")
    n = k.shape[1]
    shape = (cache.B, n, cache.heads_kv, cache.d)
    kp, ks = _rows(k, "k", shape, cache)
    vp, vs = _rows(v, "v", shape, cache)
    _kv_call(cache, stream, _lib.veda_kv_append_pending, cache.ref, cache.tail_ref, kp, ks, vp, vs, n,
             _n_new(cache, n_new))


def veda_kv_advance(cache: KVCache, n: int, n_new: Optional[torch.Tensor] = None, stream=None):
    """Take the n (or n_new[b]) pending tokens in."""
    _kv_call(cache, stream, _lib.veda_kv_advance, cache.ref, _i32(n, "n"), _n_new(cache, n_new))


def veda_kv_attn_ws_bytes(cache: KVCache, heads: int, n_q: int, with_weight: bool = False) -> int:
    return int(_lib.veda_kv_attn_ws_bytes(cache.ref, _i32(heads, "heads"), _i32(n_q, "n_q"), int(with_weight)))


def veda_kv_attn(cache: KVCache, q: torch.Tensor, o: torch.Tensor, scale: float, ws: torch.Tensor,
                 causal: bool = True, window: int = 0, sinks: int = 0, n_new: Optional[torch.Tensor] = None,
                 pending: bool = True, lse: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                 decay: float = 1.0, fill: bool = False, stream=None):
    """Attention of q [B, n_q, heads, d] over the cache, into o. ws: device
    scratch of veda_kv_attn_ws_bytes(cache, heads, n_q, weight is not None)
    bytes. weight: [B, heads_kv, nb_cap], e.g. cache.weight. fill: rows of o and
    lse without a query get zeros and -inf, else they are left as they are."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a [B, n_q, heads, d] tensor")
    _, n, heads, _ = q.shape
    shape = (cache.B, n, heads, cache.d)
    qp, qs = _rows(q, "q", shape, cache)
    op, os_ = _rows(o, "o", shape, cache)
    dev = cache.device
    lp = None if lse is None else _checked(lse, "lse", (cache.B, heads, n), torch.float32, dev)
    wp = None if weight is None else _checked(weight, "weight", (cache.B, cache.heads_kv, cache.nb_cap), torch.float32, dev)
    key = (heads, n, wp is not None)
    need = cache._ws_bytes.get(key)
    if need is None:
        need = cache._ws_bytes[key] = _lib.veda_kv_attn_ws_bytes(cache.ref, *key)
    if not isinstance(ws, torch.Tensor) or ws.device != dev or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor on the cache's device")
    if ws.nbytes < need:
        raise ValueError(f"ws holds {ws.nbytes} bytes, {need} are needed")
    _kv_call(cache, stream, _lib.veda_kv_attn_fill if fill else _lib.veda_kv_attn, cache.ref, qp, qs, heads, n, _n_new(cache, n_new), bool(pending),
             bool(causal), _i32(window, "window"), _i32(sinks, "sinks"), float(scale), op, os_, lp, wp, float(decay),
             ws.data_ptr())


def veda_kv_evict(cache: KVCache, keep: Sequence[int], sink: int, recent: int, out: Optional[KVCache] = None,
                  stream=None):
    """Drop each head's least attended tiles, down to keep[h] (one per K/V
    head), in place or into `out`, whose arrays of tiles are others. Their
    slots are the next to be written to: entries behind the tiles in use whose
    slot is shared have to be given another before the next append."""
    if len(keep) != cache.heads_kv:
        raise ValueError(f"keep must have {cache.heads_kv} entries, not {len(keep)}")
    if out is not None and out.device != cache.device:
        raise ValueError(f"out is on {out.device}, the cache on {cache.device}")
    try:
        keeps = array("i", keep)
    except OverflowError:
        raise ValueError("keep does not fit 32 bits") from None
    _kv_call(cache, stream, _lib.veda_kv_evict, cache.ref, keeps.buffer_info()[0], _i32(sink, "sink"), _i32(recent, "recent"),
             None if out is None else out.ref)


def veda_kv_check_status(cache: KVCache, stream=None):
    _kv_call(cache, stream, _lib.veda_kv_check_status, cache.ref)


def library_path() -> str:
    return _LIB_PATH
