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


def modified_scores(z, cap, slope, distance):
    """cap tanh(z / cap) (cap 0: z) - slope |distance|."""
    if cap:
        z = cap * np.tanh(z / cap)
    return z - slope * np.abs(distance)


def paged_attn_prompt(q, k, v, page_table, seq_lens, row_starts, scale, window=0, cap=0.0, slopes=None, prefix_lens=None):
    """q [P, M, Hq, D]; k, v [P, pages, Hkv, page, D] in float64; a row sees keys of
    its own sequence only.  Returns out [P, M, Hq, D], lse [P, M, Hq] (NaN in the rows
    of no sequence), the weighted mean of |v|, and an error bound's three sizes per
    row and head: the largest sum of |scale q_i k_ji|, the largest |bias|, and the
    keys seen."""
    P, M, Hq, D = q.shape
    Hkv, page = k.shape[2], k.shape[3]
    out, mean = np.full(q.shape, np.nan), np.zeros(q.shape)
    lse = np.full((P, M, Hq), np.nan)
    dots, far, keys = np.zeros((P, M, Hq)), np.zeros((P, M, Hq)), np.zeros((P, M, Hq))
    for b in range(len(seq_lens)):
        n, length = int(row_starts[b + 1] - row_starts[b]), int(seq_lens[b])
        prefix = 0 if prefix_lens is None else min(max(int(prefix_lens[b]), 0), length)
        for r in range(n):
            m, pos = int(row_starts[b]) + r, length - n + r
            out[:, m], lse[:, m] = 0.0, -np.inf
            if pos < 0:
                continue
            lo = max(0, pos + 1 - window) if window else 0
            at = np.arange(lo, max(pos + 1, prefix))
            pages, off = page_table[b][at // page], at % page
            for p in range(P):
                for h in range(Hq):
                    K, V = k[p, pages, h * Hkv // Hq, off], v[p, pages, h * Hkv // Hq, off]
                    slope = 0.0 if slopes is None else float(slopes[p, h])
                    z = modified_scores((K @ q[p, m, h]) * scale, cap, slope, pos - at)
                    top = z.max()
                    w = np.exp(z - top)
                    out[p, m, h], mean[p, m, h] = w @ V / w.sum(), w @ np.abs(V) / w.sum()
                    lse[p, m, h] = top + math.log(w.sum())
                    dots[p, m, h] = (np.abs(K) @ np.abs(q[p, m, h])).max() * abs(scale)
                    far[p, m, h] = abs(slope) * np.abs(pos - at).max()
                    keys[p, m, h] = at.size
    return out, lse, mean, (dots, far, keys)


def lora(x, A, B, ids, base, gains=None):
    """base[p][m] + gains[a] B_a (A_a x_m), a = ids[m] (< 0: none), in float64.  x [M, K]
    with base [P, M, N / P], or x [P, M, K / P] with base [P, M, N].  Returns the sum
    and its terms' absolute sum."""
    P, M, n = base.shape
    out, size = np.array(base, dtype=np.float64), np.abs(np.array(base, dtype=np.float64))
    for m in range(M):
        a = int(ids[m])
        if a < 0:
            continue
        gain = 1.0 if gains is None else float(gains[a])
        for p in range(P):
            if x.ndim == 2:
                t, tt = A[a] @ x[m], np.abs(A[a]) @ np.abs(x[m])
                up = B[a][p * n:(p + 1) * n]
            else:
                f = x.shape[2]
                Ap = A[a][:, p * f:(p + 1) * f]
                t, tt = Ap @ x[p, m], np.abs(Ap) @ np.abs(x[p, m])
                up = B[a]
            out[p, m] += gain * (up @ t)
            size[p, m] += abs(gain) * (np.abs(up) @ tt)
    return out, size
