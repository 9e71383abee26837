"""Plain CPU oracle of the operators around the 4-bit paged cache (numpy, fp64).

TEST INFRASTRUCTURE ONLY.  It shares no code, table or constant with the CUDA
library and never imports it.

The definitions are those of include/fm.h ("4-bit paged cache"): the e2m1 /
e8m0 record, the append with its rotation, the attention with its cap, bias,
window, start and list, the indexer key's record and the residual RMSNorm with
an e4m3 output.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import retriever as R

D = 128


# ------------------------------------------------------------- the 4-bit record


def e2m1(code: np.ndarray) -> np.ndarray:
    """4-bit code -> value: sign, two exponent bits (bias 1), one mantissa bit."""
    c = np.asarray(code).astype(np.int64)
    e, m = (c >> 1) & 3, (c & 1).astype(np.float64)
    mag = np.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * 2.0 ** (e - 1.0))
    return np.where(c & 8, -mag, mag)


def e8m0(byte: np.ndarray) -> np.ndarray:
    b = np.asarray(byte).astype(np.float64)
    return np.where(b == 255, np.nan, np.exp2(b - 127.0))


def dequant4(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """codes [..., 64], scales [..., 4] bytes -> [..., 128] fp64."""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], D)
    return e2m1(c) * np.repeat(e8m0(scales), 32, axis=-1)


def quant4(x: np.ndarray):
    """fp64 [..., 128] -> codes [..., 64], scales [..., 4] uint8, from the
    definition: the least power of two with amax <= 6 * 2^e, then the nearest
    of the eight magnitudes by search, ties to the even code."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], 4, 32)
    bad = ~np.isfinite(g).all(axis=-1)
    g = np.where(bad[..., None], 0.0, g)
    amax = np.abs(g).max(axis=-1)
    e = np.full(amax.shape, -126)
    pos = amax > 0
    guess = np.floor(np.log2(np.where(pos, amax, 1.0))).astype(np.int64) - 4
    for _ in range(4):
        guess = np.where(amax > 6.0 * np.exp2(guess.astype(np.float64)), guess + 1, guess)
    e = np.clip(np.where(pos, guess, -126), -126, 125)
    y = np.abs(g) / np.exp2(e.astype(np.float64))[..., None]
    mags = e2m1(np.arange(8))
    dist = np.abs(y[..., None] - mags)
    best = dist.min(axis=-1, keepdims=True)
    near = dist == best
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    code = code + 8 * ((g < 0) & (code > 0))
    code = np.where(bad[..., None], 0, code).reshape(*x.shape[:-1], 64, 2)
    scale = np.where(bad, 255, np.where(pos, e + 127, 0))
    return (code[..., 0] | (code[..., 1] << 4)).astype(np.uint8), scale.astype(np.uint8)


def rotate(x: np.ndarray, positions: np.ndarray, inv_freq) -> np.ndarray:
    """[T, heads, 128] rotated by positions [T] in half-split pairs of the last
    2 * len(inv_freq) dims; cosines and sines rounded to fp32 once."""
    x = np.array(x, np.float64, copy=True)
    if inv_freq is None:
        return x
    half = len(inv_freq)
    th = np.asarray(positions).astype(np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c = np.cos(th).astype(np.float32).astype(np.float64)
    s = np.sin(th).astype(np.float32).astype(np.float64)
    a, b = x[..., D - 2 * half:D - half].copy(), x[..., D - half:].copy()
    x[..., D - 2 * half:D - half] = a * c - b * s
    x[..., D - half:] = b * c + a * s
    return x


def read_cache(pages: np.ndarray, page_table: np.ndarray, page_size: int):
    """pages [n_pages, heads, page_size * 68] -> ([B, heads, max_pages * page_size, 128] fp64,
    there [B, max_pages * page_size] bool)."""
    n_pages, H, _ = pages.shape
    B, mp = page_table.shape
    there = (page_table >= 0) & (page_table < n_pages)
    blk = pages[np.where(there, page_table, 0)]  # [B, mp, H, block]
    codes = blk[..., :page_size * 64].reshape(B, mp, H, page_size, 64)
    scales = blk[..., page_size * 64:].reshape(B, mp, H, page_size, 4)
    x = dequant4(codes, scales).transpose(0, 2, 1, 3, 4).reshape(B, H, mp * page_size, D)
    return x, np.repeat(there, page_size, axis=1)


# ------------------------------------------------------------------- attention


def attention(q, k, v, there, kv_len, scale=None, softcap=0.0, slopes=None, window=0, kv_start=None, idx=None,
              count=None):
    """q [B, Tq, Hq, 128]; k, v [B, Hkv, n, 128] fp64; there [B, n].  Returns
    (out, err_x, abs_v, top_v): the output; what a logit's rounding error
    scales with, the largest |scale| * (sum |q||k| + sum |q| * max |k| / 16) + |x|
    over what a query sees; what the output's scales with, sum p |v|; and what
    the smallest weights' and values' absolute steps scale with,
    2^-33 * 12 n max(p max|v|) + 2^-24 sum p max|v|; each [B, Tq, Hq, 128 or 1]."""
    q = np.asarray(q, np.float64)
    B, Tq, Hq, _ = q.shape
    Hkv = k.shape[1]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = np.zeros(q.shape)
    abs_v = np.zeros(q.shape)
    err_x = np.zeros((B, Tq, Hq, 1))
    top_v = np.zeros((B, Tq, Hq, 1))
    for b in range(B):
        n = int(min(max(kv_len[b], 0), there.shape[1]))
        lo = max(0, int(kv_start[b])) if kv_start is not None else 0
        if idx is None:
            at = np.arange(n)
        else:
            at = np.asarray(idx[b, :max(0, min(int(count[b]), idx.shape[1]))], np.int64)
            at = at[(at >= 0) & (at < n)]
        at = at[there[b, at]]
        for t in range(Tq):
            p = n - Tq + t
            ok = (at <= p) & (at >= lo)
            if window > 0:
                ok &= p - at < window
            j = at[ok]
            if j.size == 0:
                continue
            for h in range(Hq):
                kh = h // (Hq // Hkv)
                x = scale * (k[b, kh, j] @ q[b, t, h])
                e = abs(scale) * (np.abs(k[b, kh, j]) @ np.abs(q[b, t, h])
                                  + np.abs(q[b, t, h]).sum() * np.abs(k[b, kh, j]).max(axis=1) / 16)
                if softcap > 0:
                    x = softcap * np.tanh(x / softcap)
                    e = e + softcap
                if slopes is not None:
                    x = x + float(slopes[h]) * (j - p)
                    e = e + np.abs(float(slopes[h]) * (j - p))
                w = np.exp(x - x.max())
                w = w / w.sum()
                out[b, t, h] = w @ v[b, kh, j]
                abs_v[b, t, h] = w @ np.abs(v[b, kh, j])
                err_x[b, t, h] = (e + np.abs(x)).max()
                pv = w * np.abs(v[b, kh, j]).max(axis=1)
                top_v[b, t, h] = 2.0 ** -33 * 12 * j.size * pv.max() + 2.0 ** -24 * pv.sum()
    return out, err_x, abs_v, top_v


# --------------------------------------------------- indexer keys and the norm


def index_vector(k, positions=None, inv_freq=None, hadamard=True) -> np.ndarray:
    x = rotate(k, positions, inv_freq)
    return R.hadamard_transform(x) if hadamard else x


def add_rmsnorm(x, residual=None, gain=None, eps=1e-6):
    """(z, y) in fp64."""
    z = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    y = R.rms_norm(z, np.ones(z.shape[-1]) if gain is None else np.asarray(gain, np.float64), eps)
    return z, y
