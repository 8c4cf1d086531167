"""Oracle of the attention sub-layer between the QKV projection and the output
projection: rotary positions, the append to a paged key-value cache, and the
attention of one token per sequence over it.

TEST INFRASTRUCTURE ONLY: plain float64 statements of the definitions, one
sequence and head at a time.  The pages name the attention sub-layer of a
block ("[Feature] Async Tensor Parallelism for Archon Engine", "Potential
Solution") and leave its inside open; the readings are the usual definitions
(rotary positions, scaled dot products, softmax).

Parity status: the rotation is pinned by closed forms (norms, composition of
positions, a transposed rotation as inverse), the attention by uniform and
one-hot weights and by splitting a row.
"""
from __future__ import annotations

import math

import numpy as np

from . import fp8_oracle


def rope_frequencies(rot, theta, scaling="none", factor=1.0, orig_len=0.0, alpha=1.0, beta=32.0):
    """Radians per position of the rot/2 pairs."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "parts":
        turns = orig_len * f / (2 * math.pi)
        keep = np.clip((turns - alpha) / (beta - alpha), 0.0, 1.0)
        return keep * f + (1 - keep) * f / factor
    return f


def angles_from_turns(positions, turns):
    """Angles [M, rot/2] in radians from the integer table, without rounding
    before the last step: the product modulo one turn is exact."""
    a = np.empty((len(positions), len(turns)))
    for m, pos in enumerate(positions):
        for i, u in enumerate(turns):
            r = (int(pos) * int(u)) % (1 << 64)
            if r >= 1 << 63:
                r -= 1 << 64
            a[m, i] = r / 2.0 ** 64 * 2 * math.pi
    return a


def rope(x, angles, Hr, interleaved=False, transpose=False, gain=1.0):
    """x [P, M, H, D] with the first Hr heads' pairs turned by angles [M, rot/2]."""
    n = angles.shape[1]
    y = np.array(x, dtype=np.float64)
    c, s = gain * np.cos(angles)[:, None, :], gain * np.sin(angles)[:, None, :]
    if transpose:
        s = -s
    ia, ib = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    a, b = y[:, :, :Hr, ia], y[:, :, :Hr, ib]
    out = y.copy()
    out[:, :, :Hr, ia] = a * c - b * s
    out[:, :, :Hr, ib] = a * s + b * c
    return out


def rope_pair_sizes(x, n, Hr, interleaved=False):
    """|a| + |b| of every element's pair (0 where nothing turns), for error bounds."""
    w = np.zeros(x.shape)
    ia, ib = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    t = np.abs(x[:, :, :Hr, ia]) + np.abs(x[:, :, :Hr, ib])
    w[:, :, :Hr, ia] = t
    w[:, :, :Hr, ib] = t
    return w


def dequantised(codes, scale):
    """Values of E4M3 codes (uint8) times their rows' scales."""
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.ldexp(1.0, e - 10))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >> 7 == 1, -v, v) * scale[..., None].astype(np.float64)


def quantise_rows(a):
    """(codes uint8, scale) of bf16-valued rows along the last axis."""
    flat = a.reshape(-1, a.shape[-1])
    q, e = fp8_oracle.quantize_rows_e4m3(flat)
    return fp8_oracle.e4m3_encode(q).reshape(a.shape), np.ldexp(1.0, e).reshape(a.shape[:-1])


def paged_attn_decode(q, k, v, page_table, seq_lens, scale, window=0):
    """q [P, B, Hq, D]; k, v [P, pages, Hkv, page, D] in float64.  Returns out
    [P, B, Hq, D], lse [P, B, Hq], and two sizes for error bounds: the weighted
    mean of |v| (like out) and the largest sum of |scale q_i k_i| of a row's
    keys (like lse)."""
    P, B, Hq, D = q.shape
    Hkv, page = k.shape[2], k.shape[3]
    group = Hq // Hkv
    out, mean = np.zeros(q.shape), np.zeros(q.shape)
    lse, dots = np.full((P, B, Hq), -np.inf), np.zeros((P, B, Hq))
    for b in range(B):
        n = int(seq_lens[b])
        at = np.arange(max(0, n - window) if window > 0 else 0, n)
        if at.size == 0:
            continue
        pages, off = page_table[b][at // page], at % page
        for p in range(P):
            for h in range(Hq):
                K, V = k[p, pages, h // group, off], v[p, pages, h // group, off]
                z = (K @ q[p, b, h]) * scale
                top = z.max()
                w = np.exp(z - top)
                total = w.sum()
                out[p, b, h] = w @ V / total
                mean[p, b, h] = w @ np.abs(V) / total
                lse[p, b, h] = top + math.log(total)
                dots[p, b, h] = (np.abs(K) @ np.abs(q[p, b, h])).max() * abs(scale)
    return out, lse, mean, dots
