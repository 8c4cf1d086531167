"""The one-token attention over an E4M3 cache, held to the bound of its own
arithmetic (fp16 operands), and at the scores and scales where it can go wrong.

Bounds, per element, with w_j the weights e^(s_j - m), l their sum, vs_j the
scales of v and A = sum_j w_j |v_j| / l.  A score is off by
    e_s = (D + 4) 2^-24 max_j sum_i |scale q_i k_ji| + 2^-39 |scale| max|q| max_j sum_i |k_ji|
(q is scaled so that its largest element is 2^14 or more and held in fp16,
whose least step is 2^-24: half of it is 2^-39 of the largest), a weight by
4e-6 more and by the rounding of its exponent, s_j plus the scale's exponent
minus a reference, numbers below |s_j| + 256 together: 2^-22 (256 + |s|).  Over
n keys, numerator and denominator together: r = 2 (e_s + n 2^-24 + 4e-6) + 2^-22 (256 + |s|) of A.
A weight times scale is rounded to fp16: 2^-11 A, and 2^-25 where it is below
2^-14, with the row's largest at 2^12 or more: n 2^-37 448 max_j w_j vs_j / l.
The result is rounded to bf16 once, half a step of it (2^-8), and may be below
bf16's least normal number.  The log-sum-exp is off by e_s + n 2^-24 + 4e-6 and
2^-22 of itself."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st
from oracle import attn_oracle as ao

import test_gpu_paged_attn as ta
from helpers import dev_tensor, host_f64, to_f64
from sequence_tensor_transformer_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


def check(c, out, lse):
    """As test_gpu_paged_attn.check, with the bound above."""
    P, B, Hq, D = c["P"], c["B"], c["Hq"], c["D"]
    ref, rl, mean, dots = ao.paged_attn_decode(c["q64"], c["k64"], c["v64"], c["table"], c["lens"], c["scale"], c["window"])
    got, gl = host_f64(out).reshape(P, B, Hq, D), host_f64(lse)
    assert not np.isnan(got).any() and not np.isnan(gl).any()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty) and not got[empty].any()
    vs = c["cache"][3].cpu().double().numpy()
    group, page = Hq // (c["k64"].shape[2]), c["page"]
    for b in range(B):
        n = int(c["lens"][b])
        at = np.arange(max(0, n - c["window"]) if c["window"] else 0, n)
        pages, off = c["table"][b][at // page], at % page
        for p in range(P):
            for h in range(Hq):
                if empty[p, b, h]:
                    continue
                K, q = c["k64"][p, pages, h // group, off], c["q64"][p, b, h]
                s = K @ q * c["scale"]
                es = (D + 4) * 2.0 ** -24 * dots[p, b, h] + 2.0 ** -39 * abs(c["scale"]) * np.abs(q).max() * np.abs(K).sum(-1).max()
                es += at.size * 2.0 ** -24 + 4e-6
                far = 2.0 ** -22 * (256 + np.abs(s).max())
                flush = at.size * 2.0 ** -37 * 448 * (np.exp(s - rl[p, b, h]) * np.abs(vs[p, pages, h // group, off])).max()
                r = ref[p, b, h]
                tol = (2.0 ** -11 + 2 * es + far) * mean[p, b, h] + flush + 2.0 ** -8 * np.abs(r) * (1 + 2.0 ** -7) + 2.0 ** -126
                err = np.abs(got[p, b, h] - r)
                assert (err <= tol).all(), (p, b, h, (err / tol).max(), got[p, b, h][:4], r[:4])
                assert abs(gl[p, b, h] - rl[p, b, h]) <= es + 2.0 ** -22 * abs(rl[p, b, h]), (p, b, h)


@pytest.mark.parametrize("P,lens,Hq,Hkv,D,page,window", [
    (4, [333, 0, 1], 7, 1, 128, 16, 0), (2, [15, 16, 17, 63, 64, 65, 129], 8, 2, 128, 16, 0), (1, [1000, 3, 2000], 32, 1, 128, 32, 0),
    (2, [700, 90], 48, 1, 64, 16, 100), (1, [400, 37], 12, 2, 256, 16, 0), (2, [130, 64, 1], 6, 3, 80, 112, 0), (1, [257], 9, 9, 96, 256, 0),
    (8, [40, 41], 3, 1, 16, 16, 0), (1, [600], 66, 2, 144, 16, 0), (1, [12000, 7], 4, 2, 64, 64, 0), (1, [500, 300], 20, 1, 256, 16, 0)])
def test_parity_within_fp16(P, lens, Hq, Hkv, D, page, window):
    for spread in (0.0, 2.0):
        c = ta.make(P, lens, Hq, Hkv, D, page, "e4m3", spread=spread, window=window)
        out, lse, ws = ta.call(c)
        assert st.sptp_read_device_status(ws) == 0
        check(c, out, lse)


def case(n, Hq, D, q, k, v, scale, page=16):
    """One sequence of n keys, one key/value head, with these float64 rows of q
    [Hq, D], k and v [n, D] (k and v quantised as an append would)."""
    max_pages = -(-n // page)
    num_pages = max_pages + 2
    table = np.random.default_rng(n + D).permutation(num_pages)[:max_pages].reshape(1, max_pages)
    q = synth._cast(q.reshape(1, 1, Hq, D), "bf16")
    c = dict(P=1, B=1, Hq=Hq, Hkv=1, D=D, page=page, lens=np.array([n]), table=table, kind="e4m3", dtype="bf16", window=0, scale=scale,
             q64=to_f64(q, "bf16"), q=dev_tensor(q, "bf16"))
    pools, scales, wide = [], [], []
    at = np.arange(n)
    for x in (k, v):
        full = np.zeros((1, num_pages, 1, page, D))
        full[0, table[0][at // page], 0, at % page] = to_f64(synth._cast(x, "bf16"), "bf16")
        codes, s = ao.quantise_rows(full)
        wide.append(ao.dequantised(codes, s))
        pools.append(torch.from_numpy(codes).cuda())
        scales.append(torch.from_numpy(s.astype(np.float32)).cuda())
    c["k64"], c["v64"] = wide
    c["cache"] = (*pools, *scales)
    return c


def scored(n, Hq, D, scores, v):
    """Keys whose scores are exactly `scores` (of four significant bits) for every head."""
    q, k = np.zeros((Hq, D)), np.zeros((n, D))
    q[:, 0] = 16.0
    k[:, 0] = np.asarray(scores) / 16.0
    return case(n, Hq, D, q, k, v, 1.0)


@pytest.mark.parametrize("Hq,D", [(4, 64), (7, 128), (16, 128), (32, 64), (4, 256)])
@pytest.mark.parametrize("n,top,other", [(40, 3, 20), (300, 2, 299), (300, 299, 2), (5000, 10, 4000), (5000, 4000, 10)])
def test_a_large_value_far_below_the_top_score(Hq, D, n, top, other):
    """The top score belongs to a row of zeros, and what the output consists
    of has a weight of 2^-130 and values of 2^60: nothing may be lost on the way."""
    rng = np.random.default_rng(n)
    scores, v = np.full(n, -128.0), rng.standard_normal((n, D))
    scores[top], scores[other] = 128.0, 36.0
    v[top] = 0.0
    v[other] *= 2.0 ** 60
    c = scored(n, Hq, D, scores, v)
    out, lse, ws = ta.call(c)
    assert st.sptp_read_device_status(ws) == 0
    check(c, out, lse)
    assert host_f64(out).any()


@pytest.mark.parametrize("Hq,D", [(4, 64), (7, 128), (16, 128), (32, 64), (4, 256)])
@pytest.mark.parametrize("big", [2.0 ** 12, 2.0 ** 40, 2.0 ** 100])
def test_a_zero_row_on_top_of_large_values(Hq, D, big):
    """All but a row of zeros are hundreds of powers of two below it: the
    output is (about) zero, not the product of a zero and an infinity."""
    n = 200
    for low in (-128.0, -1.0):
        scores, v = np.full(n, low), np.random.default_rng(1).standard_normal((n, D)) * big
        scores[77] = 128.0
        v[77] = 0.0
        c = scored(n, Hq, D, scores, v)
        out, lse, ws = ta.call(c)
        check(c, out, lse)


@pytest.mark.parametrize("Hq,D", [(4, 64), (7, 128), (16, 128), (32, 64), (4, 256)])
@pytest.mark.parametrize("n", [60, 500, 60001])
@pytest.mark.parametrize("gap", [12.0, 16.0, 18.0, 20.0])
def test_a_tail_below_one_key(Hq, D, n, gap):
    """One key on top and many that are e^-gap of it each, in an element of
    their own: what they add up to is kept, whichever share of the keys the one
    on top is in."""
    scores, v = np.zeros(n), np.zeros((n, D))
    scores[n // 5] = gap
    v[:, 1] = 1.0
    v[n // 5] = 0.0
    v[n // 5, 0] = 1.0
    c = scored(n, Hq, D, scores, v)
    out, lse, ws = ta.call(c)
    check(c, out, lse)


@pytest.mark.parametrize("Hq,D", [(4, 64), (7, 128), (16, 128), (32, 64), (4, 256)])
@pytest.mark.parametrize("outlier", [2.0 ** 12, 2.0 ** 18, 2.0 ** 22])
def test_an_outlier_in_q_beside_ordinary_elements(Hq, D, outlier):
    """An element of q that is far larger than the others and meets zeros:
    the others count in full."""
    n, rng = 300, np.random.default_rng(4)
    q, k = rng.standard_normal((Hq, D)), rng.standard_normal((n, D))
    q[:, 5] = outlier
    k[:, 5] = 0.0
    c = case(n, Hq, D, q, k, rng.standard_normal((n, D)), D ** -0.5)
    out, lse, ws = ta.call(c)
    check(c, out, lse)


def test_scales_that_are_no_powers_of_two():
    """Scales that another quantiser chose (their logarithms are off by 2^-22
    of themselves, 2^-15 at most: less than 2^-11 leaves room for, as `far` has it)."""
    c = ta.make(1, [300, 40], 8, 2, 64, 16, "e4m3", spread=1.0)
    rng = np.random.default_rng(0)
    for i, wide in ((2, "k64"), (3, "v64")):
        f = rng.uniform(0.5, 2.0, tuple(c["cache"][i].shape)).astype(np.float32)
        old = c["cache"][i].cpu().numpy()
        new = (old * f).astype(np.float32)
        with np.errstate(invalid="ignore"):
            c[wide] = c[wide] * np.where(np.isfinite(old), new.astype(np.float64) / old, 1.0)[..., None]
        c["cache"][i].copy_(torch.from_numpy(new))
    out, lse, ws = ta.call(c)
    check(c, out, lse)
