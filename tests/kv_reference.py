"""The paged 4-bit cache and attention in float64 numpy, from the formulas of
include/zt_q4.h: quantization, the place of every code and scale, rotary
embedding, softmax attention.  Shares no code with the library."""
from __future__ import annotations

import numpy as np


def quantize(x):
    """fp16 [..., D] -> (codes uint8 [..., D], scales fp16 [..., D/32])."""
    g = x.astype(np.float64).reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(g).all(-1)
    with np.errstate(all="ignore"):
        s = np.maximum(g.max(-1) / 8, -g.min(-1) / 7).astype(np.float16)
        s = s + np.float16(0)                            # no negative zero
        s[bad] = np.nan
        q = np.clip(np.rint(g / s.astype(np.float64)[..., None]), -7, 8) + 7
    q = np.where((s > 0)[..., None], q, 7)
    return q.reshape(x.shape).astype(np.uint8), s


def dequantize(q, s):
    """(code - 7) * scale in float64."""
    return (q.astype(np.float64) - 7) * np.repeat(s.astype(np.float64), 32, -1)


def tile_bytes(D):
    return 18 * D


def k_code(t, d, D):
    """(byte, nibble) of a K code within its tile."""
    G, g, j, n = D // 32, d // 32, d % 32 // 8, d % 8
    return (t * D // 8 + j * G + g) * 4 + n // 2, n % 2


def v_code(t, d, D):
    h, j, e = t // 8, t % 8 // 2, t % 2
    m, i, r = d // 16, d % 16 // 8, d % 8
    return 8 * D + ((m // 2) * 64 + (4 * r + j) * 2 + m % 2) * 4 + 2 * e + h, i


def k_scale(t, g, D):
    """byte of a K scale within its tile."""
    return 16 * D + 2 * ((t % 8 * (D // 32) + g) * 2 + t // 8)


def v_scale(t, g, D):
    h, j, e = t // 8, t % 8 // 2, t % 2
    return 17 * D + 2 * (((j * (D // 32) + g) * 2 + h) * 2 + e)


def _maps(D):
    t, d, g = np.arange(16)[:, None], np.arange(D)[None], np.arange(D // 32)[None]
    return [np.broadcast_arrays(*k_code(t, d, D)), np.broadcast_arrays(*v_code(t, d, D)), k_scale(t, g, D), v_scale(t, g, D)]


class Pool:
    """A pool of pages as bytes [n_pages, kv_heads, page_size / 16, 18 D] (a view of the library's buffer)."""

    def __init__(self, raw, page, heads, D):
        self.raw = raw.reshape(raw.shape[0], heads, page // 16, 18 * D)
        self.page, self.heads, self.D = page, heads, D

    def write(self, page, pos, k, v):
        """Quantized rows k, v [heads, D] to position pos of page `page` (pos within the page)."""
        D, t = self.D, pos % 16
        (kb, kn), (vb, vn), ks, vs = _maps(D)
        tile = self.raw[page, :, pos // 16]
        for x, b, nib, sc in ((k, kb, kn, ks), (v, vb, vn, vs)):
            q, s = quantize(x)
            for nibble in (0, 1):
                at = nib[t] == nibble
                keep = tile[:, b[t][at]] & (0xF0 >> (4 * nibble))
                tile[:, b[t][at]] = keep | (q[:, at] << (4 * nibble))
            for c in (0, 1):
                tile[:, sc[t] + c] = s.view(np.uint16) >> (8 * c) & 255

    def values(self, pages, n):
        """float64 (K, V) [n, heads, D] of the first n tokens of a sequence on `pages`."""
        D = self.D
        (kb, kn), (vb, vn), ks, vs = _maps(D)
        tiles = self.raw[np.asarray(pages, int)].transpose(0, 2, 1, 3).reshape(-1, self.heads, 18 * D)   # tile, head
        out = []
        for b, nib, sc in ((kb, kn, ks), (vb, vn, vs)):
            q = tiles[:, :, b] >> (4 * nib).astype(np.uint8) & 15                   # tile, head, t, d
            s = (tiles[:, :, sc].astype(np.uint16) | tiles[:, :, sc + 1].astype(np.uint16) << 8).view(np.float16)
            out.append(dequantize(q, s).transpose(0, 2, 1, 3).reshape(-1, self.heads, D)[:n])
        return out


def rotate(x, pos, theta):
    """Rotary embedding of x [T, H, D] at positions pos, in float64."""
    D = x.shape[-1]
    phi = np.asarray(pos, np.float64)[:, None] * float(np.float32(theta)) ** (-2.0 * np.arange(D // 2) / D)
    c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
    a, b = x[..., : D // 2].astype(np.float64), x[..., D // 2:].astype(np.float64)
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def attention(q, k, v, seen, scale):
    """(out, weighted) float64: softmax attention of q [n, Hq, D] over k, v [m, Hkv, D]; query i sees the first seen[i]
    keys; a query that sees none gives zeros.  weighted = sum_t w_t |v_t|, for error bounds."""
    n, Hq, D = q.shape
    group = Hq // k.shape[1]
    out, mag = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    for i in range(n):
        m = int(min(max(seen[i], 0), k.shape[0]))
        if m == 0:
            continue
        for h in range(Hq):
            kk, vv = k[:m, h // group], v[:m, h // group]
            s = kk @ q[i, h].astype(np.float64) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h], mag[i, h] = w @ vv, w @ np.abs(vv)
    return out, mag
