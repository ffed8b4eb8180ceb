"""Plain fp64 CPU form of the 8-bit K/V tile cache (test-only): the state as
numpy arrays of the values the codes stand for, and the four operations on it,
written from their definitions one tile or one query at a time."""
from __future__ import annotations

import math

import numpy as np

# the finite non-negative e4m3 values, by code
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)]
                + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])


def nearest_e4m3(y: np.ndarray) -> np.ndarray:
    """The e4m3 value nearest to y (|y| <= 448), ties to the even code."""
    a = np.abs(y)
    hi = np.clip(np.searchsorted(E4M3, a), 0, len(E4M3) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.copysign(E4M3[code], y)


def scale_of(amax: float) -> float:
    """Least power of two s >= 2^-40 with 448 s >= amax; NaN if not finite or
    s would pass 2^80."""
    if not np.isfinite(amax):
        return math.nan
    s = 2.0 ** -40
    while 448.0 * s < amax:
        s *= 2.0
    return s if s <= 2.0 ** 80 else math.nan


class Cache:
    """codes k8/v8 [n_slots, tile, d] as fp64 values of the codes. tail_*: of
    each head's K and V, the codes and the scale of the tail tile's committed
    tokens as they were before pending ones raised its scale, the raised scale,
    and (rows, slot, next_pos, 0) to know that tile by (zeros: nothing)."""

    FIELDS = ("k8", "v8", "table", "pos", "k_scale", "v_scale", "weight", "len", "next_pos", "tail_codes", "tail_key",
              "tail_scale")
    FLOATS = ("k8", "v8", "k_scale", "v_scale", "weight", "tail_codes", "tail_scale")

    def __init__(self, tile: int, **arrays):
        self.tile = tile
        self.B, self.hkv, self.nb_cap = np.shape(arrays["table"])
        tails = {"tail_codes": (tile, np.shape(arrays["k8"])[-1]), "tail_key": (4,), "tail_scale": (2,)}
        for f, shape in tails.items():
            arrays.setdefault(f, np.zeros((self.B, self.hkv, 2) + shape))
        for f in self.FIELDS:
            setattr(self, f, np.array(arrays[f]).astype(np.float64 if f in self.FLOATS else np.int64))

    def count(self, b, h, n):
        """Tokens of the head with n more; None where the sequence is refused:
        one of its heads cannot hold them."""
        held = self.len[b]
        fits = n >= 0 and (held >= 0).all() and (held + n <= self.nb_cap * self.tile).all()
        return int(held[h] + n) if fits else None

    def committed(self, b, h, x, codes, scale):
        """Codes of the committed rows of the head's tail tile and their scale,
        without what pending tokens did to them; whether those had done any."""
        i, r0 = divmod(int(self.len[b, h]), self.tile)
        slot, now = self.table[b, h, i], scale[b, h, i]
        (rows, at, pos, _), (was, raised) = self.tail_key[b, h, x], self.tail_scale[b, h, x]
        if (rows, at, pos) == (r0, slot, self.next_pos[b]) and np.array_equal(raised, now, equal_nan=True):
            kept = self.tail_codes[b, h, x, :r0]
            moved = kept if math.isnan(raised) else nearest_e4m3(kept * (was / raised))
            if np.array_equal(moved, codes[slot, :r0], equal_nan=True):
                return kept, was, True
        return codes[slot, :r0].copy(), now, False

    def append(self, k, v, news):
        """k, v [B, n, hkv, d] fp64."""
        T = self.tile
        for b in range(self.B):
            for h in range(self.hkv):
                total = self.count(b, h, news[b])
                if total is None or news[b] > k.shape[1]:
                    continue
                held = int(self.len[b, h])
                if news[b] == 0:
                    i, r0 = divmod(held, T)
                    slot = self.table[b, h, i] if r0 else -1
                    if not 0 <= slot < len(self.k8):
                        continue
                    for x, codes, scale in ((0, self.k8, self.k_scale), (1, self.v8, self.v_scale)):
                        kept, was, some = self.committed(b, h, x, codes, scale)
                        if some:
                            codes[slot, :r0], codes[slot, r0:], scale[b, h, i] = kept, 0.0, was
                            self.tail_key[b, h, x] = 0
                    continue
                for i in range(held // T, -(-total // T)):
                    lo, hi = max(held, i * T), min(total, (i + 1) * T)
                    slot = self.table[b, h, i]
                    fresh = lo == i * T
                    if not 0 <= slot < len(self.k8):
                        if fresh:
                            self.pos[b, h, i] = self.next_pos[b] + lo - held
                        continue
                    for x, new, codes, scale in ((0, k, self.k8, self.k_scale), (1, v, self.v8, self.v_scale)):
                        rows = new[b, lo - held:hi - held, h]
                        with np.errstate(invalid="ignore"):
                            amax = np.max(np.abs(rows))
                        s = scale_of(amax)
                        r0, r1 = lo - i * T, hi - i * T
                        if i == held // T:
                            key = np.zeros(4, np.int64)
                        if not fresh:
                            kept, old, _ = self.committed(b, h, x, codes, scale)
                            s = math.nan if math.isnan(s) or math.isnan(old) else max(s, old)
                            if s != old and not math.isnan(old):
                                self.tail_codes[b, h, x, :r0], self.tail_scale[b, h, x] = kept, (old, s)
                                key[:3] = r0, slot, self.next_pos[b]
                            codes[slot, :r0] = kept if math.isnan(s) or s == old else nearest_e4m3(kept * (old / s))
                        if i == held // T:
                            self.tail_key[b, h, x] = key
                        codes[slot, r0:r1] = 0.0 if math.isnan(s) else nearest_e4m3(rows / s)
                        codes[slot, r1:] = 0.0
                        scale[b, h, i] = s
                    if fresh:
                        self.pos[b, h, i] = self.next_pos[b] + lo - held
                        self.weight[b, h, i] = 0.0

    def advance(self, news):
        for b in range(self.B):
            if self.count(b, 0, news[b]) is not None:
                self.len[b] += news[b]
                self.next_pos[b] += news[b]

    def keys(self, b, h, total):
        """(K, V, positions) of the head's first `total` tokens; tiles with a
        slot outside the pool are left out (mask in the fourth)."""
        T, nb = self.tile, -(-total // self.tile)
        slot = self.table[b, h, :nb]
        there = (slot >= 0) & (slot < len(self.k8))
        slot = np.where(there, slot, 0)
        K = (self.k8[slot] * self.k_scale[b, h, :nb, None, None]).reshape(-1, self.k8.shape[-1])[:total]
        V = (self.v8[slot] * self.v_scale[b, h, :nb, None, None]).reshape(-1, self.k8.shape[-1])[:total]
        at = (self.pos[b, h, :nb, None] + np.arange(T)).reshape(-1)[:total]
        return K, V, at, np.repeat(there, T)[:total]

    def attend(self, q, news, scale, causal, window, sinks, pending=True):
        """Returns per query O, lse and the tile weights, and for tolerances
        A = sum p |v| and S = scale * sum |q| |k| (largest over its keys):
        o [B, n, heads, d], lse [B, heads, n], weight [B, hkv, nb_cap] (NaN
        where not written), A like o, S like lse, and R like lse: the largest
        p_j times its tile's V scale; Q likewise, scale * max |q| * sum |k|
        (largest over its keys)."""
        B, n, heads, d = q.shape
        g = heads // self.hkv
        o, A = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
        lse, S, R = np.full((B, heads, n), np.nan), np.zeros((B, heads, n)), np.zeros((B, heads, n))
        Q = np.zeros((B, heads, n))
        weight = np.full(self.table.shape, np.nan)
        written = np.zeros(self.table.shape, bool)
        for b in range(B):
            for h in range(self.hkv):
                total = self.count(b, h, news[b] if pending else 0)
                if total is None or news[b] <= 0 or news[b] > n:
                    continue
                m, nb = int(news[b]), -(-total // self.tile)
                K, V, at, there = self.keys(b, h, total)
                t = int(self.next_pos[b]) + np.arange(m)[:, None]
                see = np.broadcast_to(there[None, :], (m, total)).copy()
                if causal:
                    see &= at[None, :] <= t
                if window > 0:
                    see &= (at[None, :] > t - window) | (at[None, :] < sinks)
                acc = np.zeros(nb * self.tile)
                for j in range(h * g, (h + 1) * g):
                    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
                        s = np.where(see, q[b, :m, j] @ K.T * scale, -np.inf)
                        s = np.where(see & np.isnan(K).any(-1)[None, :], np.nan, s)
                        mx = np.max(s, axis=1, keepdims=True, initial=-np.inf)
                        mx = np.where(mx == -np.inf, 0.0, mx)
                        e = np.where(see, np.exp(s - mx), 0.0)
                        z = e.sum(1, keepdims=True)
                        p = np.where(z == 0, 0.0, e / np.where(z == 0, 1.0, z))
                        lse[b, j, :m] = (mx + np.log(z))[:, 0]
                        bad = np.isnan(V).any(-1)
                        Vf = np.where(bad[:, None], 0.0, V)
                        o[b, :m, j] = p @ Vf
                        A[b, :m, j] = p @ np.abs(Vf)
                        sv = np.repeat(self.v_scale[b, h, :nb], self.tile)[:total]
                        R[b, j, :m] = np.max(np.where(see & ~bad[None, :], p * sv, 0.0), axis=1, initial=0.0)
                        sick = (see & bad[None, :]).any(1)
                        o[b, :m, j][sick] = np.nan
                        S[b, j, :m] = np.max(np.where(see, np.abs(q[b, :m, j]) @ np.abs(K).T, 0.0), axis=1, initial=0.0) * abs(scale)
                        top = np.abs(q[b, :m, j]).max(-1) * abs(scale)
                        Q[b, j, :m] = top * np.max(np.where(see, np.abs(K).sum(-1)[None, :], 0.0), axis=1, initial=0.0)
                        # a V tile without a scale also spoils the row's sum
                        lse[b, j, :m][sick] = np.nan
                        p = np.where(sick[:, None], np.nan, p)
                        acc[:total] += np.where(see, p, 0.0).sum(0)
                weight[b, h, :nb] = acc.reshape(nb, self.tile).sum(1)
                written[b, h, :nb] = True
        return o, lse, weight, written, A, S, R, Q

    def evict(self, keep, sink, recent):
        for b in range(self.B):
            for h in range(self.hkv):
                nb = -(-int(self.len[b, h]) // self.tile)
                if nb <= keep[h]:
                    continue
                w = self.weight[b, h]
                rank = sorted(range(sink, nb - recent),
                              key=lambda i: (0 if math.isnan(w[i]) else 1, 0.0 if math.isnan(w[i]) else -w[i], i))
                stay = sorted(list(range(sink)) + rank[:keep[h] - sink - recent] + list(range(nb - recent, nb)))
                kept = set(stay)
                order = stay + [i for i in range(nb) if i not in kept] + list(range(nb, self.nb_cap))
                for f in ("table", "pos", "k_scale", "v_scale", "weight"):
                    a = getattr(self, f)
                    a[b, h] = a[b, h][order]
                self.len[b, h] -= (nb - keep[h]) * self.tile
