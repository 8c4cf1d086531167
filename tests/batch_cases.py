"""Cases of prompts' attention for the GPU tests: host values, device tensors, and the
comparison with the float64 oracle."""
import numpy as np
import torch

import sequence_tensor_transformer_gb300 as st
from oracle import attn_oracle as ao
from sequence_tensor_transformer_gb300 import synth

from helpers import dev_tensor, host_f64, nan_workspace, to_f64

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
TD = {"bf16": torch.bfloat16, "fp32": torch.float32}


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def make(P, rows, lens, Hq, Hkv, D, page, kind, seed=0, q_std=1.0, window=0, prefix=None, cap=0.0, slopes=None, first=0, pad=0,
         spread=0.0, scale=None, holes=True):
    """Sequences of rows[b] new rows and lens[b] keys, `first` rows of none before them and
    `pad` behind.  Cache slots that no row of a sequence sees hold NaN, or NaN codes
    and scales (holes=False: values, for calls with other rows and lengths)."""
    rng = np.random.default_rng(seed + D + Hq)
    dtype = "fp32" if kind == "fp32" else "bf16"
    rows, lens = np.asarray(rows), np.asarray(lens)
    B, starts = len(rows), first + np.concatenate([[0], np.cumsum(rows)])
    M = int(starts[-1]) + pad
    max_pages = max(1, max(-(-int(n) // page) for n in lens)) + 1
    num_pages = B * max_pages + 1
    table = rng.permutation(num_pages)[: B * max_pages].reshape(B, max_pages)
    q = synth._cast(rng.standard_normal((P, M, Hq, D)) * q_std, dtype)
    shape = (P, num_pages, Hkv, page, D)
    mags = np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    used = np.zeros((num_pages, page), bool)
    for b in range(B):
        if rows[b] == 0:
            continue
        pos = max(0, lens[b] - rows[b])
        at = np.arange(max(0, pos + 1 - window) if window else 0, lens[b])
        used[table[b][at // page], at % page] = True
    hole = ~used[None, :, None, :] & np.full((P, 1, Hkv, 1), holes)
    c = dict(P=P, M=M, B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, rows=rows, lens=lens, starts=starts, table=table, kind=kind,
             dtype=dtype, window=window, cap=cap, prefix=prefix, scale=D ** -0.5 if scale is None else scale,
             slopes=None if slopes is None else np.asarray(slopes, np.float32).reshape(P, Hq), q64=to_f64(q, dtype),
             q=dev_tensor(q, dtype))
    pools, scales, wide = [], [], []
    for i in range(2):
        x = synth._cast(rng.standard_normal(shape) * mags, dtype)
        if kind == "e4m3":
            codes, s = ao.quantise_rows(to_f64(x, "bf16"))
            wide.append(ao.dequantised(codes, s))
            codes[hole], s = 0xFF, s.astype(np.float32)
            s[hole] = np.nan
            pools.append(torch.from_numpy(codes).cuda())
            scales.append(torch.from_numpy(s).cuda())
        else:
            wide.append(to_f64(x, dtype))
            t = dev_tensor(x, dtype)
            t[torch.from_numpy(hole).cuda()] = float("nan")
            pools.append(t)
            scales.append(None)
    c["k64"], c["v64"] = wide
    c["cache"] = (*pools, *scales)
    return c


def workspace(c):
    return nan_workspace(st.sptp_paged_attn_prompt_workspace_size(c["P"], c["M"], c["B"], c["Hq"], c["Hkv"], c["D"]))


def arguments(c):
    """(positional, keyword) arguments of the call."""
    return ((c["q"], c["cache"], ints(c["table"]), ints(c["lens"]), ints(c["starts"])),
            dict(scale=c["scale"], window=c["window"], cap=c["cap"],
                 slopes=None if c["slopes"] is None else torch.from_numpy(c["slopes"]).cuda(),
                 prefix_lens=None if c["prefix"] is None else ints(c["prefix"])))


def call(c, **kw):
    """The call into outputs of 7s."""
    ws = workspace(c)
    out = torch.full((c["P"], c["M"], c["Hq"] * c["D"]), 7.0, dtype=TD[c["dtype"]], device="cuda")
    lse = torch.full((c["P"], c["M"], c["Hq"]), 7.0, device="cuda")
    args, kws = arguments(c)
    got = st.sptp_paged_attn_prompt(*args, **{**kws, **kw}, out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse
    return out, lse, ws


def score_error(D, dots, far, cap):
    """How far a score may be off (natural units): D products summed in fp32 and scaled;
    the cap's tanh, 2^-22 of it; the bias, 2^-22 of itself; its weight's exponent and
    exponential, 4e-6."""
    return (D + 4) * 2.0 ** -24 * dots + 2.0 ** -21 * (cap if cap < 1e9 else 0.0) + 2.0 ** -22 * far + 4e-6


def check(c, out, lse):
    """Bounds per element, with A = sum_j w_j |v_j| / sum_j w_j and n keys: a weight's
    exponent is off by e (score_error), the sums over the keys by n 2^-24 of them: r = 2
    (e + n 2^-24) of A together; a bf16 or E4M3 cache's weights are rounded to bf16, 2^-8
    A more; the result is rounded once, half a step of it.  The log-sum-exp is off by e
    + n 2^-24 and 2^-22 of itself."""
    P, M, Hq, D = c["P"], c["M"], c["Hq"], c["D"]
    ref, rl, mean, (dots, far, keys) = ao.paged_attn_prompt(c["q64"], c["k64"], c["v64"], c["table"], c["lens"], c["starts"],
                                                            c["scale"], c["window"], c["cap"], c["slopes"], c["prefix"])
    got, gl = host_f64(out).reshape(P, M, Hq, D), host_f64(lse)
    none = np.isnan(rl)
    assert (got[none] == 7.0).all() and (gl[none] == 7.0).all(), "a row of no sequence was written"
    got, gl, ref, rl, mean = (x[~none] for x in (got, gl, ref, rl, mean))
    es = (score_error(D, dots, far, c["cap"]) + keys * 2.0 ** -24)[~none]
    assert not np.isnan(got).any() and not np.isnan(gl).any()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty) and not got[empty].any()
    rounded = 0.0 if c["kind"] == "fp32" else 2.0 ** -8
    tol = (rounded + 2 * es)[..., None] * mean + HALF[c["dtype"]] * np.abs(ref) * (1 + 2.0 ** -7)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], (np.abs(got - ref) / np.maximum(tol, 1e-30)).max())
    gl, rl, es = gl[~empty], rl[~empty], es[~empty]
    assert (np.abs(gl - rl) <= es + 2.0 ** -22 * np.abs(rl)).all(), np.abs(gl - rl).max()
