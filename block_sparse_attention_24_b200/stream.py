"""One attention layer over a stream: tokens or chunks of video arrive, attend
to what the 8-bit K/V tile cache holds and to themselves, and join it.

    append (K, V) -> attention -> [advance -> evict]

The last two only where a chunk is final: while it is being denoised, step()
with commit=False replaces the chunk's pending keys and values each time.
Only marshalling and buffer management live here; every step is a libveda
kernel.
"""
from __future__ import annotations

import math
from typing import List, Optional

import torch

from . import (KVCache, veda_kv_advance, veda_kv_append, veda_kv_attn, veda_kv_attn_ws_bytes, veda_kv_check_status,
               veda_kv_evict)


class VedaStream:
    """heads query heads over heads_kv K/V heads of a cache of max_tokens per
    sequence. `causal`, `window` and `sinks` as in veda_kv_attn. `keep` (tiles,
    one number or one per K/V head): a head that holds more after a committed
    step drops the least attended ones, all but its first `sink_tiles` and
    last `recent_tiles`; None: nothing is dropped. Attention weights are summed
    over committed steps, those before with a factor `decay` for every step.

    max_tokens has to hold what is kept and a step's tokens together: a step
    that finds less room in any head of a sequence leaves that sequence as it
    was and gives it zeros. Only the device knows; check_status() tells.

    A captured step uses the layer's memory: the layer has to live as long as
    the graph."""

    def __init__(self, B: int, heads: int, heads_kv: int, d: int, tile: int, max_tokens: int, device,
                 causal: bool = True, window: int = 0, sinks: int = 0, keep=None, sink_tiles: int = 1,
                 recent_tiles: int = 1, decay: float = 1.0, scale: Optional[float] = None):
        self.cache = KVCache(B, heads_kv, d, tile, -(-max_tokens // tile), device)
        if heads < 1 or heads % heads_kv:
            raise ValueError(f"heads={heads} must be a multiple of heads_kv={heads_kv}")
        if window < 0 or sinks < 0:
            raise ValueError(f"window={window} and sinks={sinks} must be >= 0")
        self.heads = heads
        self.causal, self.window, self.sinks = causal, window, sinks
        self.scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        self.keep: Optional[List[int]] = None
        if keep is not None:
            self.keep = [int(keep)] * heads_kv if isinstance(keep, int) else [int(k) for k in keep]
            # here, not behind a step's append and attention
            if len(self.keep) != heads_kv:
                raise ValueError(f"keep must have {heads_kv} entries, not {len(self.keep)}")
            if sink_tiles < 0 or recent_tiles < 1 or min(self.keep) < sink_tiles + recent_tiles:
                raise ValueError(f"keep={self.keep} must be at least sink_tiles={sink_tiles} (>= 0) + "
                                 f"recent_tiles={recent_tiles} (>= 1)")
        self.sink_tiles, self.recent_tiles, self.decay = sink_tiles, recent_tiles, decay
        self._ws = {}
        self._recorded = set()

    def workspace(self, n: int, weight: bool) -> torch.Tensor:
        """Scratch of a step of n tokens, allocated at the first one. Sizes are
        powers of two, so steps of many lengths share a few; none is freed, as a
        captured step may use it."""
        size = veda_kv_attn_ws_bytes(self.cache, self.heads, n, weight)
        if size == 0:
            raise ValueError(f"a step of {n} tokens and {self.heads} heads is outside the library's limits")
        size = 1 << (size - 1).bit_length()
        if size not in self._ws:
            self._ws[size] = torch.empty(size, dtype=torch.uint8, device=self.cache.device)
        return self._ws[size]

    def step(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_new: Optional[torch.Tensor] = None,
             commit: bool = True, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None):
        """q [B, n, heads, d], k, v [B, n, heads_kv, d] bf16; n_new [B] int32:
        the real rows of each sequence (None: all). Returns the output, like q:
        `out`, whose rows (and those of lse) that are not real, or not of a
        sequence that fits, are left as they are; or if it is not given a tensor
        allocated on `stream`, where they are zero (and -inf in lse)."""
        if stream is not None:
            # the step's tensors belong to the stream that uses them
            with self._on(stream):
                return self.step(q, k, v, n_new, commit, out, lse)
        n, c = self._tokens(q, k, v), self.cache
        if n_new is None and n > c.nb_cap * c.tile:
            raise ValueError(f"a step of {n} tokens does not fit a cache of {c.nb_cap * c.tile}")
        fill = out is None
        if fill:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if n == 0:
            return out
        weigh = commit and self.keep is not None
        ws = self.workspace(n, weigh)
        self._record(ws)
        veda_kv_append(c, k, v, n_new=n_new)
        veda_kv_attn(c, q, out, self.scale, ws, causal=self.causal, window=self.window,
                     sinks=self.sinks, n_new=n_new, lse=lse, weight=c.weight if weigh else None, decay=self.decay, fill=fill)
        if commit:
            veda_kv_advance(c, n, n_new=n_new)
            if self.keep is not None:
                veda_kv_evict(c, self.keep, self.sink_tiles, self.recent_tiles)
        return out

    def _tokens(self, q, k, v) -> int:
        """The tokens of a step: append, attention and advance have to agree."""
        c = self.cache
        shapes = [t.shape if isinstance(t, torch.Tensor) else () for t in (q, k, v)]
        n = shapes[0][1] if len(shapes[0]) == 4 else 0
        kv = (c.B, n, c.heads_kv, c.d)
        if shapes == [(c.B, n, self.heads, c.d), kv, kv]:
            return n
        for shape, name, heads in zip(shapes, "qkv", (self.heads, c.heads_kv, c.heads_kv)):
            if len(shape) != 4 or (shape[0], shape[2], shape[3]) != (c.B, heads, c.d):
                raise ValueError(f"{name} must be a [{c.B}, n, {heads}, {c.d}] tensor")
        raise ValueError(f"q, k and v must have as many tokens each, not {[s[1] for s in shapes]}")

    def _record(self, ws: Optional[torch.Tensor] = None):
        """The current stream uses the layer's memory: dropped meanwhile, it is
        not to be handed out again before that stream is through."""
        c = self.cache
        if c.device.type != "cuda":
            return
        key = (torch._C._cuda_getCurrentRawStream(c.device.index), None if ws is None else ws.nbytes)
        if key not in self._recorded:
            stream = torch.cuda.current_stream(c.device)
            for t in c.tensors() if ws is None else [*c.tensors(), ws]:
                t.record_stream(stream)
            self._recorded.add(key)

    def _on(self, stream):
        if stream is not None and stream.device != self.cache.device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {self.cache.device}")
        return torch.cuda.stream(stream)

    def reset(self, stream=None):
        """Empty the cache (its next tokens are at position 0 again)."""
        with self._on(stream):
            self._record()
            self.cache.len.zero_()
            self.cache.next_pos.zero_()

    def check_status(self, stream=None):
        veda_kv_check_status(self.cache, stream=stream)
