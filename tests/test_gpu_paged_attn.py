"""GPU parity of the attention of one token over a paged key-value cache,
against the float64 oracle, and a run of the whole attention sub-layer.

Bounds, per element, with A = sum_j w_j |v_j| / sum_j w_j and n keys.  A score
is a sum of D products, times a scale: off by e_s = (D + 4) 2^-24 max_j sum_i
|scale q_i k_ji|; its weight's exponent and exp by 4e-6 more.  The sums over
the keys are off by n 2^-24 at most.  Numerator and denominator together:
r = 2 (e_s + n 2^-24 + 4e-6) of A.  With a bf16 or E4M3 cache a weight is
rounded to bf16 for its product with v: 2^-8 A more.  The result is rounded
once, half a step of it.  The log-sum-exp is off by e_s + n 2^-24 + 4e-6 and
2^-22 of itself."""
import numpy as np
import pytest
import torch

import oracle
import sequence_tensor_transformer_gb300 as st
from oracle import attn_oracle as ao
from oracle import fp8_oracle as f8
from sequence_tensor_transformer_gb300 import synth

from helpers import TOL, dev_tensor, host_f64, nan_tensor, nan_workspace, rel_err, to_f64

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
TD = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def make(P, lens, Hq, Hkv, D, page, kind, seed=0, q_std=1.0, window=0, spread=0.0):
    """A case on the host (q, k, v as float64 of what is stored) and its device
    tensors.  Cache slots that no key of a sequence (within its window)
    occupies hold NaN, or NaN codes and scales."""
    rng = np.random.default_rng(seed + D + Hq)
    dtype = "fp32" if kind == "fp32" else "bf16"
    lens = np.asarray(lens)
    B = len(lens)
    max_pages = max(1, max(-(-int(n) // page) for n in lens)) + 1
    num_pages = B * max_pages + 1
    table = rng.permutation(num_pages)[: B * max_pages].reshape(B, max_pages)
    q = synth._cast(rng.standard_normal((P, B, Hq, D)) * q_std, dtype)
    shape = (P, num_pages, Hkv, page, D)
    mags = np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    used = np.zeros((num_pages, page), bool)
    for b in range(B):
        at = np.arange(max(0, lens[b] - window) if window else 0, lens[b])
        used[table[b][at // page], at % page] = True
    hole = ~used[None, :, None, :] & np.ones((P, 1, Hkv, 1), bool)
    c = dict(P=P, B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, lens=lens, table=table, kind=kind, dtype=dtype, window=window,
             scale=D ** -0.5, q64=to_f64(q, dtype), q=dev_tensor(q, dtype))
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


def call(c, **kw):
    ws = nan_workspace(st.sptp_paged_attn_workspace_size(c["P"], c["B"], c["Hq"], c["Hkv"], c["D"]))
    out, lse = nan_tensor((c["P"], c["B"], c["Hq"] * c["D"]), TD[c["dtype"]]), nan_tensor((c["P"], c["B"], c["Hq"]), torch.float32)
    kw = {**dict(page_table=ints(c["table"]), seq_lens=ints(c["lens"])), **kw}
    got = st.sptp_paged_attn_decode(c["q"], c["cache"], scale=c["scale"], window=c["window"], out=out, lse=lse, workspace=ws, **kw)
    assert got[0] is out and got[1] is lse
    return out, lse, ws


def check(c, out, lse, rows=slice(None)):
    P, B, Hq, D = c["P"], c["B"], c["Hq"], c["D"]
    ref, rl, mean, dots = ao.paged_attn_decode(c["q64"], c["k64"], c["v64"], c["table"], c["lens"], c["scale"], c["window"])
    n = np.minimum(c["lens"], c["window"]) if c["window"] else c["lens"]
    es = (D + 4) * 2.0 ** -24 * dots + n[None, :, None] * 2.0 ** -24 + 4e-6
    got, gl = host_f64(out).reshape(P, B, Hq, D), host_f64(lse)
    assert not np.isnan(got).any() and not np.isnan(gl).any()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty) and not got[empty].any()
    rounded = 0.0 if c["kind"] == "fp32" else 2.0 ** -8
    tol = (rounded + 2 * es)[..., None] * mean + HALF[c["dtype"]] * np.abs(ref) * (1 + 2.0 ** -7)
    bad = (np.abs(got - ref) > tol)[:, rows]
    assert not bad.any(), (np.argwhere(bad)[:3], (np.abs(got - ref) / np.maximum(tol, 1e-30)).max())
    gl, rl, es = gl[~empty], rl[~empty], es[~empty]
    assert (np.abs(gl - rl) <= es + 2.0 ** -22 * np.abs(rl)).all(), np.abs(gl - rl).max()


KINDS = ["bf16", "fp32", "e4m3"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P,lens,Hq,Hkv,D,page", [
    (4, [1], 7, 1, 128, 16), (1, [0], 4, 2, 64, 16), (2, [15, 16, 17, 0, 63, 64, 65, 1], 8, 2, 128, 16), (1, [127, 128, 129, 255, 500], 5, 5, 64, 48),
    (4, [333], 7, 1, 128, 64), (1, [1000, 3, 2000], 32, 1, 128, 32), (2, [700, 90], 48, 1, 64, 16), (1, [400, 37], 12, 2, 256, 16),
    (2, [130, 64, 1], 6, 3, 80, 112), (1, [257], 9, 9, 96, 256), (8, [40, 41], 3, 1, 16, 16), (1, [600], 66, 2, 144, 16), (1, [0, 0, 0], 2, 1, 128, 16)])
def test_decode(P, lens, Hq, Hkv, D, page, kind):
    c = make(P, lens, Hq, Hkv, D, page, kind, spread=0.5)
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    check(c, out, lse)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [8, 24, 40, 72, 104, 200])
def test_decode_odd_head_sizes(D, kind):
    c = make(2, [70, 5, 129], 4, 2, D, 16, kind)
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    check(c, out, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 16, 63, 64, 200, 5000])
def test_decode_window(window, kind):
    c = make(2, [1, 16, 200, 201, 330, 1000, 0], 6, 2, 64, 32, kind, window=window)
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    check(c, out, lse)


def test_decode_window_reads_no_page_before_it():
    """Pages that lie before the window may be gone from the table."""
    c = make(1, [300, 100], 4, 1, 128, 16, "bf16", window=40)
    table = c["table"].copy()
    table[0, : (300 - 40) // 16] = -1
    table[1, : (100 - 40) // 16] = 1 << 30
    table[0, 19:], table[1, 7:] = -7, 1 << 29  # nor behind the length
    out, lse, ws = call(c, page_table=ints(table))
    assert st.sptp_read_device_status(ws) == 0
    check(c, out, lse)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_long_rows(kind):
    """Few long rows beside short ones: the length is split over many SMs."""
    c = make(1, [20011, 1, 9000, 0, 777], 4, 2, 64, 64, kind, q_std=2.0)
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    check(c, out, lse)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_many_rows(kind):
    """More rows than SMs, of every length around the tiles."""
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 150, 700)
    c = make(1, lens, 2, 1, 64, 16, kind)
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    check(c, out, lse)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_extreme_scores(kind):
    """One key far above the others; scores of large size either way; the
    largest score first or last."""
    for at in (0, 100, 299):
        c = make(1, [300], 4, 1, 64, 16, kind, q_std=30.0)
        row = c["table"][0][at // 16], at % 16
        k = c["k64"][0, row[0], 0, row[1]]
        if kind == "e4m3":
            c["cache"][2][0, row[0], 0, row[1]] *= 64
        else:
            c["cache"][0][0, row[0], 0, row[1]] *= 64
        k *= 64
        out, lse, ws = call(c)
        check(c, out, lse)


def test_decode_extreme_magnitudes_e4m3():
    """Values of far-apart scales: a row of zeros (the least scale), tiny and
    huge rows of v, each the winner of a head or not."""
    c = make(1, [200], 4, 2, 64, 16, "e4m3")
    codes, scale, v64 = c["cache"][1], c["cache"][3], c["v64"]
    page = c["table"][0]
    for j, f in ((3, 0.0), (17, 2.0 ** -90), (50, 2.0 ** 90), (120, 2.0 ** 20)):
        pg, off = page[j // 16], j % 16
        if f == 0.0:
            codes[0, pg, :, off] = 0
            scale[0, pg, :, off] = 2.0 ** -126
        else:
            scale[0, pg, :, off] *= f
        v64[0, pg, :, off] *= f
    out, lse, ws = call(c)
    check(c, out, lse)
    # every row tiny
    c = make(1, [100], 2, 1, 32, 16, "e4m3")
    c["cache"][3].mul_(2.0 ** -80)
    c["v64"] *= 2.0 ** -80
    out, lse, ws = call(c)
    check(c, out, lse)


def test_decode_scale_zero_negative_and_no_lse():
    for scale in (0.0, -0.3, 2.0):
        c = make(1, [130, 20], 4, 2, 64, 16, "bf16")
        c["scale"] = scale
        out, lse, ws = call(c)
        check(c, out, lse)
        got, none = st.sptp_paged_attn_decode(c["q"], c["cache"], ints(c["table"]), ints(c["lens"]), scale, write_lse=False)
        assert none is None and torch.equal(got, out)
    c = make(1, [130, 20], 4, 2, 64, 16, "bf16")
    out, lse, ws = call(c)
    got, l2 = st.sptp_paged_attn_decode(c["q"], c["cache"], ints(c["table"]), ints(c["lens"]))
    assert torch.equal(got, out) and torch.equal(l2, lse)  # the default scale is D^-1/2


@pytest.mark.parametrize("kind", KINDS)
def test_decode_is_deterministic(kind):
    c = make(2, [5000, 3, 1200, 0, 64], 14, 2, 128, 16, kind)
    first = call(c)[:2]
    for _ in range(5):
        again = call(c)[:2]
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("kind", KINDS)
def test_decode_bad_pages_and_lengths_are_recorded(kind):
    """A page outside the pool counts as zero keys and values, a length
    outside the table is cut; both are recorded, and the next call's status is
    its own."""
    c = make(2, [100, 60, 40], 4, 2, 64, 16, kind)
    good = c["table"].copy()
    for entry in (-1, c["cache"][0].shape[1], -2 ** 31, 2 ** 31 - 1):
        table = good.copy()
        table[1, 2] = entry
        out, lse, ws = call(c, page_table=ints(table))
        assert st.sptp_read_device_status(ws) == st.STATUS["shape"]
        zero = dict(c, k64=c["k64"].copy(), v64=c["v64"].copy())
        zero["k64"][:, good[1, 2]] = 0
        zero["v64"][:, good[1, 2]] = 0
        check(zero, out, lse)
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    check(c, out, lse)
    # a negative length is an empty row; one past the table is cut to it
    lens = c["lens"].copy()
    lens[2] = -5
    out, lse, ws = call(c, seq_lens=ints(lens))
    assert st.sptp_read_device_status(ws) == st.STATUS["shape"]
    check(dict(c, lens=np.array([100, 60, 0])), out, lse)
    full = c["table"].shape[1] * 16
    c = make(1, [full, 20], 4, 2, 64, 16, kind)
    span = c["table"].shape[1] * 16
    lens = np.array([span + 1, 20])
    cut = make(1, [span, 20], 4, 2, 64, 16, kind)
    short = cut["table"][:, : span // 16]
    assert cut["table"].shape[1] == span // 16 + 1
    out, lse, ws = call(cut, page_table=ints(short), seq_lens=ints(lens))
    assert st.sptp_read_device_status(ws) == st.STATUS["shape"]
    check(cut, out, lse)


def test_decode_cache_past_2_31_elements():
    P, Hkv, page, D, n = 1, 8, 64, 256, 150
    num_pages = (1 << 31) // (Hkv * page * D) + 40
    pools = [torch.full((P, num_pages, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    small = make(P, [n], 8, Hkv, D, page, "bf16")
    table = np.array([[num_pages - 1, 5, num_pages - 20]])
    for pool, src in zip(pools, small["cache"][:2]):
        for i, pg in enumerate(table[0]):
            pool[:, pg] = src[:, small["table"][0, i]]
    out, lse, ws = call(dict(small, cache=(*pools, None, None)), page_table=ints(table))
    check(small, out, lse)


def test_decode_on_another_stream_and_captured():
    """A call on a stream of its own, and a captured one replayed on new
    lengths, queries and keys."""
    c = make(2, [200, 31, 0, 400], 4, 2, 64, 16, "bf16")
    d = make(2, [17, 400, 100, 64], 4, 2, 64, 16, "bf16", seed=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse, ws = call(c)
    s.synchronize()
    check(c, out, lse)
    q, table, lens = c["q"].clone(), ints(c["table"]), ints(c["lens"])
    k, v = c["cache"][0].clone(), c["cache"][1].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.sptp_paged_attn_decode(q, (k, v, None, None), table, lens, c["scale"], out=out, lse=lse, workspace=ws)
    for x in (d, c, d):
        q.copy_(x["q"])
        k.copy_(x["cache"][0])
        v.copy_(x["cache"][1])
        table.copy_(ints(x["table"]))
        lens.copy_(ints(x["lens"]))
        out.fill_(float("nan"))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        check(x, out, lse)
        assert st.sptp_read_device_status(ws) == 0


# ---------------------------------------------------------------- the sub-layer

@pytest.mark.parametrize("kind", KINDS)
def test_attention_sublayer_steps(kind):
    """Three decoding steps of a sub-layer: boundary and QKV projection,
    rotation and append, attention, output projection; the oracle keeps a cache
    of its own and takes every step's QKV rows from the library's, so that each
    part is held to its own error.  The last output feeds the FFN boundary."""
    P, B, d, Hq, Hkv, D, page, eps = 2, 4, 256, 4, 1, 64, 16, 1e-6
    dtype = "fp32" if kind == "fp32" else "bf16"
    cfg = synth.AttnConfig("step", B, d, P * (Hq + 2 * Hkv) * D, P * Hq * D, P, 2, dtype)
    inp = synth.attn_inputs(cfg)
    T = {n: dev_tensor(a, dtype) for n, a in inp.items()}
    turns = st.sptp_rope_turns(D)
    cache = st.paged_kv_cache(P, 20, Hkv, page, D, TD[dtype], e4m3=kind == "e4m3")
    rng = np.random.default_rng(3)
    table = rng.permutation(20)[: B * 3].reshape(B, 3)
    start = np.array([0, 14, 15, 30])
    # the cache's past: rows appended as one prompt
    past = [(b, j) for b in range(B) for j in range(start[b])]
    rows = synth._cast(rng.standard_normal((P, len(past), (Hq + 2 * Hkv) * D)), dtype)
    st.sptp_rope_append_kv(dev_tensor(rows, dtype), ints([j for _, j in past]), ints([b for b, _ in past]), ints(table), turns, cache, Hq)
    for step in range(3):
        pos = start + step
        qkv, h = st.sptp_attn_qkv_forward(T["x"], T["partials"], T["gamma"], T["Wqkv"], P, 2, eps)
        ws = nan_workspace(st.sptp_paged_attn_workspace_size(P, B, Hq, Hkv, D))
        q = st.sptp_rope_append_kv(qkv, ints(pos), ints(range(B)), ints(table), turns, cache, Hq, workspace=ws)
        assert st.sptp_read_device_status(ws) == 0
        attn, lse = st.sptp_paged_attn_decode(q, cache, ints(table), ints(pos + 1), workspace=ws)
        assert st.sptp_read_device_status(ws) == 0
        # the cache's new rows are the rotated keys and the values
        x64 = host_f64(qkv).reshape(P, B, Hq + 2 * Hkv, D)
        ref = ao.rope(x64, ao.angles_from_turns(pos, turns.cpu().tolist()), Hq + Hkv)
        wide = [ao.dequantised(t.cpu().numpy(), s.cpu().numpy()) if kind == "e4m3" else host_f64(t) for t, s in zip(cache[:2], cache[2:])]
        for b in range(B):
            pg, off = table[b, pos[b] // page], pos[b] % page
            rel = 2.0 ** -4 + 2.0 ** -7 if kind == "e4m3" else 2 * HALF[dtype]
            for p in range(P):
                for i, w in enumerate(wide):
                    want = ref[p, b, Hq + i * Hkv: Hq + (i + 1) * Hkv]
                    assert np.abs(w[p, pg, :, off] - want).max() <= rel * np.abs(want).max() + 1e-5
        c = dict(P=P, B=B, Hq=Hq, Hkv=Hkv, D=D, lens=pos + 1, table=table, kind=kind, dtype=dtype, window=0, scale=D ** -0.5,
                 q64=host_f64(q), k64=wide[0], v64=wide[1])
        check(c, attn, lse)
        partials = st.sptp_down_proj(attn, T["Wo"], P)
        want = oracle.rowparallel_projection(host_f64(attn), to_f64(inp["Wo"], dtype), P)
        assert max(rel_err(host_f64(partials[p]), want[p]) for p in range(P)) <= TOL[dtype]
        T["x"], T["partials"] = h, partials
    F = 128
    W = [dev_tensor(synth.draw(s, 0.06, 0.0, dtype, 1, i), dtype) for i, s in enumerate(((F, d), (F, d), (d, F)))]
    out, h2 = st.sptp_ffn_forward(h, partials, T["gamma"], *W, P, 2, eps)
    assert not torch.isnan(out.float()).any() and not torch.isnan(h2.float()).any()
