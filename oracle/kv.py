"""Float64 oracle of the attention side of a layer: norm and rotation of query and key heads,
the paged NVFP4 key/value cache, and attention over it.

The Basalt pages define none of these; the readings are the plainest:
  K1 norm: y = x / sqrt(mean(x^2) + eps) * w over a head's D elements.
  K2 rotation: pair p of a token at position pos turns by pos * f_p; pairs are (p, p + R/2) or
     (2p, 2p + 1) of the first R elements, sine and cosine times a factor m; the result is
     rounded to float32 and then to bf16.
  K3 cache: the NVFP4 quantisation (R1-R3) of the bf16 rows, blocks of 16 along D, a static
     tensor scale per key/value head; a token's slot s is row s % page_size of page s // page_size.
  K4 attention: softmax(scale q k) v over the keys a query sees; query i of n at position
     ctx - n + i; no key gives 0 and -infinity.
"""
from __future__ import annotations

import numpy as np

from . import nvfp4 as onv

F32 = np.float32


def to_bf16(x) -> np.ndarray:
    """float64 -> float32 -> bf16, nearest even, as float32 values (finite input)."""
    b = np.asarray(x, dtype=np.float64).astype(F32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16
    return b.astype(np.uint32).view(F32)


def norm_rope(x, pos, weight=None, eps=0.0, inv_freq=None, interleaved=False, m=1.0) -> np.ndarray:
    """x [T][heads][D] -> float64 before rounding (K1, K2)."""
    y = np.asarray(x, dtype=np.float64).copy()
    D = y.shape[-1]
    if weight is not None:
        y = y / np.sqrt(np.sum(y * y, axis=-1, keepdims=True) / D + eps) * np.asarray(weight, np.float64)
    half = 0 if inv_freq is None else len(inv_freq)
    out = y.copy()
    for p in range(half):
        a = np.asarray(pos, np.float64) * np.float64(inv_freq[p])
        c, s = (m * np.cos(a))[:, None], (m * np.sin(a))[:, None]
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        out[..., i] = y[..., i] * c - y[..., j] * s
        out[..., j] = y[..., j] * c + y[..., i] * s
    return out


class Cache:
    """One layer's cache as numpy arrays, laid out as moe_kv_cache_t."""

    def __init__(self, n_pages, page_size, Hkv, D, k_ts=None, v_ts=None):
        self.page_size, self.Hkv, self.D = page_size, Hkv, D
        self.ts = {"k": np.ones(Hkv, F32) if k_ts is None else np.asarray(k_ts, F32),
                   "v": np.ones(Hkv, F32) if v_ts is None else np.asarray(v_ts, F32)}
        self.codes = {n: np.zeros((n_pages, Hkv, page_size, D // 2), np.uint8) for n in "kv"}
        self.scales = {n: np.zeros((n_pages, Hkv, page_size, D // 16), np.uint8) for n in "kv"}

    def write(self, name, rows, slots):
        """rows float32 (bf16 values) [T][Hkv][D]; negative slots are skipped."""
        for h in range(self.Hkv):
            codes, scales, _ = onv.quantize(np.ascontiguousarray(rows[:, h], dtype=F32), ts=self.ts[name][h])
            for t, s in enumerate(slots):
                if s >= 0:
                    at = (s // self.page_size, h, s % self.page_size)
                    self.codes[name][at], self.scales[name][at] = codes[t], scales[t]

    def read(self, name, slots) -> np.ndarray:
        """float64 [n][Hkv][D], exact."""
        slots = np.asarray(slots, dtype=np.int64)
        page, off = slots // self.page_size, slots % self.page_size
        out = np.empty((len(slots), self.Hkv, self.D))
        for h in range(self.Hkv):
            out[:, h] = onv.dequantize(self.codes[name][page, h, off], self.scales[name][page, h, off], self.ts[name][h])
        return out


def attention(q, k, v, scale, causal):
    """One sequence: q [n][Hq][D], k and v [ctx][Hkv][D] in float64. Returns out [n][Hq][D], lse
    [n][Hq], and two magnitudes for error bounds: weight [n][Hq][D] = sum_j p_j |v_j| and
    logit [n][Hq] = scale * max_j sum_i |q_i k_ij| over the seen keys (0 for none)."""
    q = np.asarray(q, dtype=np.float64)
    n, Hq, D = q.shape
    ctx, Hkv = k.shape[0], k.shape[1]
    out, weight = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, logit = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        seen = min(ctx, max(0, ctx - n + i + 1)) if causal else ctx
        if seen == 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            s = scale * (k[:seen, g] @ q[i, h])
            top = s.max()
            e = np.exp(s - top)
            lse[i, h] = top + np.log(e.sum())
            p = e / e.sum()
            out[i, h] = p @ v[:seen, g]
            weight[i, h] = p @ np.abs(v[:seen, g])
            logit[i, h] = abs(scale) * (np.abs(k[:seen, g]) @ np.abs(q[i, h])).max()
    return out, lse, weight, logit
