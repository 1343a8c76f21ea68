"""Streams of single tokens (oracle): rotary positions, the append to a paged
pool and attention over it, in fp64 and one sequence, head and token at a time.

Definitions (include/ll_api.h, "Streams of single tokens"):
- pair i of a head turns by the angle p * w_i; w_i = theta^(-2i/rot), scaled by
  f_i = r_i + (1 - r_i) * scale with r_i the ramp of the turns within the
  original length (0 without one);
- the scale of a page and head is the largest power of two asked for by the
  calls that wrote it (the smallest s with 448 s >= max|x|);
- key j is seen from position p when j < prefix, or j <= p and (no window, or
  p - j < window, or j < n_sink).
"""
from __future__ import annotations

import math

import numpy as np

from oracle import fp8


def frequencies(rot: int, theta0: float = 10000.0, scale: float = 1.0, original_len: float = 0.0,
                beta_fast: float = 32.0, beta_slow: float = 1.0) -> np.ndarray:
    w = np.array([theta0 ** (-2.0 * i / rot) for i in range(rot // 2)])
    keep = np.zeros_like(w)
    if original_len > 0:
        turns = original_len * w / (2 * math.pi)
        keep = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
    return w * (keep + (1.0 - keep) * scale)


def rotate(x: np.ndarray, pos, w: np.ndarray, layout: str, amplitude: float = 1.0, transpose: bool = False):
    """x [T][H][D] at positions pos [T]."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    n = len(w)
    for t, p in enumerate(pos):
        z = amplitude * np.exp((-1j if transpose else 1j) * float(p) * w)
        if layout == "half":
            a, b = x[t, :, :n], x[t, :, n:2 * n]
        else:
            a, b = x[t, :, 0:2 * n:2], x[t, :, 1:2 * n:2]
        c = (a + 1j * b) * z
        if layout == "half":
            y[t, :, :n], y[t, :, n:2 * n] = c.real, c.imag
        else:
            y[t, :, 0:2 * n:2], y[t, :, 1:2 * n:2] = c.real, c.imag
    return y


def two_power_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with 448 s >= amax; 0 for 0."""
    if not amax > 0:
        return 0.0
    s = 2.0 ** -126
    e = max(-126, math.floor(math.log2(amax / 448.0)) - 1)
    s = 2.0 ** e
    while 448.0 * s < amax:
        s *= 2.0
    return s


class Pool:
    """[n_pages][H][page_size][D] values (bf16 pool: what is stored; e4m3: codes and scales)."""

    def __init__(self, n_pages, page_size, H, D, dtype):
        self.n_pages, self.page_size, self.H, self.D, self.dtype = n_pages, page_size, H, D, dtype
        shape = (n_pages, H, page_size, D)
        self.k, self.v = np.zeros(shape), np.zeros(shape)          # bf16: values; fp8: decoded codes
        self.ks, self.vs = np.zeros(shape[:2]), np.zeros(shape[:2])

    def values(self, which):
        x, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        return x * s[..., None, None] if self.dtype == "fp8" else x

    def append(self, table, length, k, v):
        """k, v [n][H][D] (already rotated) are the last tokens of a sequence of `length` tokens."""
        n, ps = k.shape[0], self.page_size
        first = length - n
        pages = sorted({p // ps for p in range(max(first, 0), length)})
        for pg in pages:
            if pg >= len(table) or not 0 <= table[pg] < self.n_pages:
                continue
            page = table[pg]
            new = [p for p in range(max(first, pg * ps, 0), min(length, (pg + 1) * ps))]
            off = new[0] - pg * ps
            for h in range(self.H):
                for x, pool, scales in ((k, self.k, self.ks), (v, self.v, self.vs)):
                    rows = np.stack([x[p - first, h] for p in new])
                    at = slice(off, off + len(new))
                    if self.dtype != "fp8":
                        pool[page, h, at] = rows
                        continue
                    was = scales[page, h] if off else 0.0
                    s = max(was, two_power_scale(float(np.max(np.abs(rows)))))
                    if s > was and off:
                        pool[page, h, :off] = fp8.e4m3_decode_array(fp8.e4m3_encode(pool[page, h, :off] * was / s))
                    pool[page, h, at] = fp8.e4m3_decode_array(fp8.e4m3_encode(rows / s)) if s else 0.0
                    scales[page, h] = s


def attend(q, k, v, length, *, scale=None, cap=0.0, slopes=None, window=0, n_sink=0, prefix=0, exists=None):
    """q [n][Hq][D], the (rotated) last n tokens of a sequence of `length` keys k, v
    [length][H][D]; exists [length]: keys in mapped pages. Returns out, lse and, for
    tolerances, sum_j p_j |v_j| and the largest sum_d |q_d k_d| * scale of a row's seen keys."""
    n, Hq, D = q.shape
    group = Hq // k.shape[1] if k.shape[1] else 1
    scale = D ** -0.5 if not scale else scale
    out, mag = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, dots = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    j = np.arange(k.shape[0])
    for i in range(n):
        p = length - n + i
        seen = j <= p
        if window:
            seen = seen & ((p - j < window) | (j < n_sink))
        seen = seen | (j < prefix)
        if exists is not None:
            seen = seen & exists
        if not seen.any():
            continue
        for h in range(Hq):
            kk, vv = k[seen, h // group], v[seen, h // group]
            x = kk @ q[i, h] * scale
            dots[i, h] = np.max(np.abs(kk) @ np.abs(q[i, h])) * scale
            if cap:
                x = cap * np.tanh(x / cap)
            if slopes is not None:
                x = x - slopes[h] * np.abs(p - j[seen])
            m = x.max()
            e = np.exp(x - m)
            out[i, h] = e @ vv / e.sum()
            mag[i, h] = e @ np.abs(vv) / e.sum()
            lse[i, h] = m + math.log(e.sum())
    return out, lse, mag, dots
