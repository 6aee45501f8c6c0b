"""Plain 64-bit forms of the operators of include/pkv_ops.h, in numpy, for the tests."""
from __future__ import annotations

import math

import numpy as np

import workloads as W

BLOCK = 16


def bf16(x):
    """float64 / float32 values rounded to bf16, as their bit patterns."""
    return W.f32_to_bf16_bits(np.array(x, dtype=np.float32))


def value(bits):
    return W.bf16_bits_to_f32(bits).astype(np.float64)


# ---------------------------------------------------------------- rotation
def turn_fractions(positions, turns):
    """The angle of every (row, pair) as a fraction of a turn, exact in Python integers."""
    out = np.empty((len(positions), len(turns)))
    for i, p in enumerate(positions):
        for j, t in enumerate(turns):
            out[i, j] = ((int(p) * int(t)) % (1 << 64)) / 2.0 ** 64
    return out


def rotate(x, positions, turns, interleaved, scale=1.0):
    """``x`` float64 [n, heads, D], its first 2 * len(turns) dims rotated; also the
    magnitude |x| + |y| of each pair (0 where nothing turns), for error bounds."""
    h = len(turns)
    a = 2 * math.pi * turn_fractions(positions, turns)
    c, s = np.cos(a)[:, None, :] * scale, np.sin(a)[:, None, :] * scale
    lo = np.arange(h) * 2 if interleaved else np.arange(h)
    hi = lo + 1 if interleaved else lo + h
    out, mag = x.copy(), np.zeros_like(x)
    out[..., lo] = x[..., lo] * c - x[..., hi] * s
    out[..., hi] = x[..., hi] * c + x[..., lo] * s
    both = (np.abs(x[..., lo]) + np.abs(x[..., hi])) * abs(scale)
    mag[..., lo], mag[..., hi] = both, both
    return out, mag


# ---------------------------------------------------------------- E4M3
_CODES = np.array([(-1.0 if c & 128 else 1.0) *
                   (math.ldexp(8 + (c & 7), ((c >> 3) & 15) - 10) if (c >> 3) & 15
                    else math.ldexp(c & 7, -9)) for c in range(256)])
_CODES[[127, 255]] = np.nan


def e4m3_value(codes):
    return _CODES[np.asarray(codes, np.uint8)]


_MAGS = _CODES[:127]


def e4m3_code(x):
    """Nearest E4M3 code, ties to even, saturating at 448; NaN is 0x7f."""
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e9, neginf=1e9)), 448.0)
    up = np.clip(np.searchsorted(_MAGS, mag), 1, 126)
    dn = up - 1
    du, dd = _MAGS[up] - mag, mag - _MAGS[dn]
    code = np.where((dd < du) | ((dd == du) & (dn % 2 == 0)), dn, up).astype(np.uint8)
    code = code | np.where(np.signbit(x), 128, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(127), code)


def scale_byte(amax):
    """The smallest byte b >= 1 with amax <= 448 * 2^(b - 127)."""
    b = 1
    while amax > math.ldexp(448.0, b - 127):
        b += 1
    return b


def append_block(x, slots, codes, scale):
    """Rows x (float64 [n, heads, D]) into block-scaled codes and scale bytes, in place."""
    n, heads, _ = x.shape
    i = 0
    while i < n:
        if slots[i] < 0 or slots[i] >= codes.shape[0] * BLOCK:
            i += 1
            continue
        b = slots[i] // BLOCK
        e = i
        while e < n and slots[e] >= 0 and slots[e] // BLOCK == b:
            e += 1
        offs = slots[i:e] % BLOCK
        for h in range(heads):
            run = x[i:e, h]
            fin = np.abs(run[np.isfinite(run)])
            new = scale_byte(fin.max() if fin.size else 0.0)
            old = 0 if (offs == 0).any() else int(scale[b, h])
            s = max(old, new)
            if old and s > old:
                codes[b, :, h] = e4m3_code(np.ldexp(e4m3_value(codes[b, :, h]), old - s))
            scale[b, h] = s
            codes[b, offs, h] = e4m3_code(np.ldexp(run, 127 - s))
        i = e


def pool_values(codes, scale):
    return e4m3_value(codes) * np.ldexp(1.0, scale.astype(np.int64) - 127)[:, None, :, None]


# ---------------------------------------------------------------- attention
def attention(q, k, v, tables, lens, nq, scale, softcap=0.0, slopes=None, window=0, v_exp=None):
    """float64 q [S*nq, Hq, D], pools k, v [NB, 16, Hkv, D]: the output; the same with
    |v| in place of v (what the weights' relative errors scale with); per row the
    largest sum |q||k| * scale over its visible positions; and with v_exp (the scale
    exponents of a block-scaled v) the sum over the visible positions of |v| 2^(E - e),
    E the largest exponent among them, over the sum of the weights relative to the
    largest (what an absolute error of every scaled weight scales with)."""
    S, Hkv, D = len(lens), k.shape[2], k.shape[3]
    Hq = q.shape[1]
    G = Hq // Hkv
    out = np.zeros(q.shape)
    mag = np.zeros(q.shape)
    big = np.zeros(q.shape[:2])
    low = np.zeros(q.shape)
    for s in range(S):
        T = int(min(max(lens[s], 0), tables.shape[1] * BLOCK))
        first = max(0, T - nq - window + 1) if window else 0
        at = np.arange(first, T)
        rows = tables[s][at // BLOCK].astype(np.int64)
        ks, vs = k[rows, at % BLOCK], v[rows, at % BLOCK]         # [t, Hkv, D]
        for j in range(nq):
            pos = T - nq + j
            see = (at <= pos) & ((at > pos - window) if window else True)
            if pos < 0 or not see.any():
                continue
            qr = q[s * nq + j].reshape(Hkv, G, D)
            x = np.einsum("hgd,thd->hgt", qr, ks[see]) * scale
            big[s * nq + j] = (np.einsum("hgd,thd->hgt", np.abs(qr), np.abs(ks[see])).max(-1)
                               * scale).reshape(-1)
            if softcap:
                x = softcap * np.tanh(x / softcap)
            if slopes is not None:
                x = x + slopes.reshape(Hkv, G, 1) * (at[see] - pos)
            p = np.exp(x - x.max(-1, keepdims=True))
            if v_exp is not None:
                e = v_exp[rows].astype(np.int64)                  # [t, Hkv]
                scaled = np.abs(vs) * np.ldexp(1.0, e.max(0) - e)[..., None]
                low[s * nq + j] = (scaled.sum(0)[:, None] /
                                   p.sum(-1)[..., None]).reshape(Hq, D)
            p /= p.sum(-1, keepdims=True)
            out[s * nq + j] = np.einsum("hgt,thd->hgd", p, vs[see]).reshape(Hq, D)
            mag[s * nq + j] = np.einsum("hgt,thd->hgd", p, np.abs(vs[see])).reshape(Hq, D)
    return out, mag, big, low
