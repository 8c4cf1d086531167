"""GPU parity of prompts' attention over a paged key-value cache, against the float64
oracle (bounds: batch_cases.check)."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

from batch_cases import arguments, call, check, ints, make, workspace
from helpers import host_f64

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp32", "e4m3"]
SHAPE, TIMEOUT = st.STATUS["shape"], st.STATUS["timeout"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


def run(c, status=0):
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == status
    check(c, out, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,lens", [
    ((1,), (1,)), ((1,), (129,)), ((5,), (5,)), ((3, 1, 0, 7), (3, 64, 40, 200)), ((130,), (130,)), ((64,), (64,)), ((65, 2), (193, 128)),
    ((2, 2), (127, 128))])
def test_lengths(kind, rows, lens):
    run(make(2, rows, lens, 4, 2, 64, 16, kind, first=1, pad=2))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 144, 256])
def test_head_sizes(kind, D):
    run(make(1, (37, 4), (150, 70), 2, 1, D, 16, kind))


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [8, 24, 40, 72, 88, 136, 200, 248])
def test_head_sizes_of_odd_eights(kind, D):
    run(make(1, (37, 4), (150, 70), 2, 1, D, 32, kind, cap=10.0))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (7, 1), (10, 2), (16, 1), (33, 1), (64, 1), (65, 1), (130, 1), (8, 8)])
def test_groups(kind, Hq, Hkv):
    run(make(1, (11, 2), (20, 140), Hq, Hkv, 32, 16, kind, pad=1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 48, 64, 80, 128, 256])
def test_pages(kind, page):
    run(make(2, (40, 9), (300, 257), 2, 1, 64, page, kind))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 2, 15, 100, 128, 300, 2 ** 31 - 1])
def test_windows(kind, window):
    run(make(1, (70, 5), (260, 131), 2, 1, 64, 16, kind, window=window))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("prefix", [(0, 0), (130, 1), (260, 131), (200, 60)])
def test_prefixes(kind, window, prefix):
    run(make(1, (140, 5), (260, 131), 2, 1, 64, 16, kind, window=window, prefix=prefix))


def test_prefixes_outside_are_cut():
    c = make(1, (40, 5), (60, 31), 2, 1, 64, 16, "bf16", prefix=(60, 0))
    args, kw = arguments(c)
    want = st.sptp_paged_attn_prompt(*args, **kw)
    got = st.sptp_paged_attn_prompt(*args, **{**kw, "prefix_lens": ints([1 << 30, -5])})
    assert all(torch.equal(a, b) for a, b in zip(got, want))


SLOPES = {"usual": lambda n: 2.0 ** (-8.0 * np.arange(1, n + 1) / n), "steep": lambda n: np.full(n, 3.0),
          "mixed": lambda n: np.linspace(-0.05, 0.2, n)}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cap", [0.0, 1.0, 15.0, 127.0, 300.0])
@pytest.mark.parametrize("slopes", [None, "usual", "steep", "mixed"])
@pytest.mark.parametrize("prefix", [False, True])
def test_caps_and_biases(kind, cap, slopes, prefix):
    P, Hq = 2, 4
    run(make(P, (60, 3), (200, 90), Hq, 2, 64, 16, kind, q_std=4.0, cap=cap, slopes=None if slopes is None else SLOPES[slopes](P * Hq),
             prefix=(100, 90) if prefix else None))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_scores_beyond_a_large_cap_s_half(kind, D):
    # scores of some hundreds against a cap of 200: the exact form of the tanh
    run(make(1, (40,), (300,), 2, 1, D, 16, kind, q_std=60.0, cap=200.0))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap,slopes", [(0.0, None), (50.0, None), (0.0, "mixed")])
def test_large_scores_of_rising_and_falling_size(kind, D, cap, slopes):
    # maxima that move by far more than 2^8 from tile to tile
    run(make(1, (20, 1), (700, 400), 4, 2, D, 16, kind, q_std=12.0, spread=1.0, cap=cap,
             slopes=None if slopes is None else SLOPES[slopes](4)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_scales(kind, scale, cap):
    run(make(1, (33,), (150,), 2, 1, 64, 16, kind, scale=scale, cap=cap))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_few_rows_of_a_long_sequence(kind, D):
    # keys split over all CTAs, parts joined
    run(make(2, (3, 1), (9000, 5000), 4, 2, D, 64, kind, cap=30.0))
    run(make(1, (1,), (20001,), 2, 1, D, 16, kind))


@pytest.mark.parametrize("kind", KINDS)
def test_many_short_sequences(kind):
    rng = np.random.default_rng(4)
    rows = rng.integers(0, 4, 150)
    run(make(1, rows, rows + rng.integers(0, 30, 150), 2, 1, 64, 16, kind, first=3, pad=5))


@pytest.mark.parametrize("kind", KINDS)
def test_more_rows_than_keys(kind):
    # rows before position 0 see nothing, and the call says so
    run(make(2, (6, 3), (4, 0), 2, 1, 64, 16, kind), SHAPE)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_bad_pages_count_as_zeros(kind, bad):
    c = make(2, (30, 4), (100, 200), 4, 2, 64, 16, kind)
    page = c["table"][1][3]
    c["table"] = c["table"].copy()
    c["table"][1][3] = bad
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == SHAPE
    # the oracle: a page of zeros
    c["table"][1][3] = page
    c["k64"][:, page] = c["v64"][:, page] = 0.0
    check(c, out, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("starts", [(0, 30, 20), (-3, 10, 34), (0, 10, 60), (34, 0, 34), (2 ** 31 - 1, -2 ** 31, 5)])
def test_bad_row_numbers_are_reported(kind, starts):
    c = make(1, (30, 4), (100, 200), 4, 2, 64, 16, kind)
    c["starts"] = np.array(starts)
    ws = workspace(c)
    args, kw = arguments(c)
    st.sptp_paged_attn_prompt(*args, **kw, workspace=ws)
    assert st.sptp_read_device_status(ws) == SHAPE
    # the next call is not affected
    run(make(1, (30, 4), (100, 200), 4, 2, 64, 16, kind))


@pytest.mark.parametrize("kind", KINDS)
def test_bad_lengths_are_cut_and_reported(kind):
    c = make(1, (5, 4), (64, 32), 2, 1, 64, 16, kind)
    span = c["table"].shape[1] * 16
    args, kw = arguments(c)
    for lens in ((span + 1, 32), (64, -1)):
        ws = workspace(c)
        st.sptp_paged_attn_prompt(*args[:3], ints(lens), args[4], **kw, workspace=ws)
        assert st.sptp_read_device_status(ws) == SHAPE


@pytest.mark.parametrize("kind", KINDS)
def test_equal_inputs_give_equal_bits_and_outputs_are_optional(kind):
    c = make(2, (70, 9), (700, 50), 4, 2, 128, 32, kind, cap=20.0)
    out, lse, _ = call(c)
    again, lse2, _ = call(c)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    args, kw = arguments(c)
    o, l = st.sptp_paged_attn_prompt(*args, **kw)
    assert torch.equal(o, out) and torch.equal(l, lse)
    o, l = st.sptp_paged_attn_prompt(*args, **kw, write_lse=False)
    assert torch.equal(o, out) and l is None


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cap,slopes", [(10.0, None), (0.0, "usual"), (10.0, "usual")])
def test_what_lies_outside_does_not_change_a_bit(kind, cap, slopes):
    """Shared memory that other calls have left, in place of keys that no row sees."""
    c = make(1, (60, 5), (400, 90), 4, 2, 64, 16, kind, cap=cap, slopes=None if slopes is None else SLOPES[slopes](4))
    loud = make(1, (200, 70), (1500, 900), 4, 2, 64, 16, kind, q_std=1e4, spread=3.0)
    out, lse, _ = call(c)
    for _ in range(3):
        call(loud)
        again, lse2, _ = call(c)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", KINDS)
def test_without_rows_nothing_is_written(kind):
    c = make(1, (0, 0), (5, 9), 2, 1, 64, 16, kind, pad=3)
    run(c)
    q = c["q"][:, :0].contiguous()
    args, kw = arguments(c)
    out, lse = st.sptp_paged_attn_prompt(q, *args[1:], **kw)
    assert out.shape == (1, 0, 128) and lse.shape == (1, 0, 2)


def test_infinite_and_nan_queries_stay_in_their_rows():
    c = make(1, (40,), (90,), 4, 2, 64, 16, "bf16")
    args, kw = arguments(c)
    want, wl = st.sptp_paged_attn_prompt(*args, **kw)
    q = c["q"].clone()
    q[0, 3, 1] = float("nan")
    q[0, 20, 2] = float("inf")
    got, gl = st.sptp_paged_attn_prompt(q, *args[1:], **kw)
    same = torch.ones(40, 4, dtype=torch.bool, device="cuda")
    same[3, 1] = same[20, 2] = False
    assert torch.equal(got[0].view(40, 4, 64)[same], want[0].view(40, 4, 64)[same]) and torch.equal(gl[0][same], wl[0][same])
    assert torch.isnan(gl[0, 3, 1]) and torch.isnan(got[0].view(40, 4, 64)[3, 1]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("withhold", [0, 1, 3])
def test_a_tile_that_never_comes_is_reported(kind, withhold):
    c = make(1, (300,), (1500,), 4, 1, 128, 16, kind)
    ws = workspace(c)
    args, _ = arguments(c)
    out = torch.empty(1, 300, 4 * 128, dtype=torch.bfloat16, device="cuda")
    st.sptp_paged_attn_prompt_wait_selftest(*args, out, ws, withhold)
    assert st.sptp_read_device_status(ws) == TIMEOUT
    run(c)  # the GPU is fine


def test_a_tile_beyond_the_share_is_not_missed():
    c = make(1, (30,), (150,), 4, 1, 128, 16, "bf16")
    ws = workspace(c)
    args, _ = arguments(c)
    out = torch.empty(1, 30, 4 * 128, dtype=torch.bfloat16, device="cuda")
    st.sptp_paged_attn_prompt_wait_selftest(*args, out, ws, 1000)
    assert st.sptp_read_device_status(ws) == 0
    assert torch.equal(out, st.sptp_paged_attn_prompt(*args)[0])


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 72, 128, 256])
@pytest.mark.parametrize("rows,lens,window,prefix", [
    ((300,), (300,), 0, None),            # every tile on the diagonal
    ((40, 1, 33), (1500, 9, 9000), 0, None),  # masked tiles at the end only, parts to join
    ((150, 20), (700, 64), 200, None),    # a window's lower edge too
    ((90,), (400,), 16, None),            # windows smaller than a tile
    ((120, 60), (500, 60), 0, (450, 30)),  # a prefix that reaches beyond some rows
    ((50,), (20,), 0, None),              # rows that see nothing
])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(kind, D, rows, lens, window, prefix):
    """Infinities and NaN at keys that some rows of a sequence see and others do not: a
    row's other elements, and other rows, keep their bits."""
    P, Hq, Hkv, page = 2, 4, 2, 16
    c = make(P, rows, lens, Hq, Hkv, D, page, kind, window=window, prefix=prefix)
    out, lse, ws = call(c)
    status = SHAPE if any(r > n for r, n in zip(rows, lens)) else 0
    assert st.sptp_read_device_status(ws) == status
    rng = np.random.default_rng(1)
    want = host_f64(out).reshape(P, c["M"], Hq, D).copy()
    v = c["cache"][1]
    for b, n in enumerate(lens):
        near = np.arange(max(0, n - rows[b]), n)  # keys of the new rows, of which some are not seen by all
        keys = np.unique(np.concatenate([rng.choice(near, min(6, near.size), replace=False), [n - 1], rng.integers(0, n, 2)]))
        for i, key in enumerate(keys):
            for p in range(P):
                h, d = int(rng.integers(Hkv)), int(rng.integers(D))
                x = (np.inf, -np.inf, np.nan)[i % 3]
                v[p, int(c["table"][b][key // page]), h, key % page, d] = x
                for r in range(rows[b]):
                    pos = n - rows[b] + r
                    hi = 0 if pos < 0 else max(pos + 1, 0 if prefix is None else min(prefix[b], n))
                    lo = max(0, pos + 1 - window) if window else 0
                    if lo <= key < hi:
                        with np.errstate(invalid="ignore"):
                            want[p, int(c["starts"][b]) + r, h * 2: h * 2 + 2, d] += x
    again, lse2, ws = call(c)
    assert st.sptp_read_device_status(ws) == status
    got = host_f64(again).reshape(want.shape)
    assert np.array_equal(got, want, equal_nan=True), np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))[:5]
    assert torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,lens,window", [((300,), (300,), 0), ((40, 33), (1500, 9000), 0), ((150, 20), (700, 64), 200)])
def test_scales_that_are_not_finite_stay_with_the_rows_that_see_them(D, rows, lens, window):
    """The same for the scales of an E4M3 cache's values, and of its keys beyond a row's position."""
    P, Hq, Hkv, page = 2, 4, 2, 16
    c = make(P, rows, lens, Hq, Hkv, D, page, "e4m3", window=window)
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    rng = np.random.default_rng(2)
    want = host_f64(out).reshape(P, c["M"], Hq, D).copy()
    for b, n in enumerate(lens):
        keys = np.unique(np.concatenate([rng.integers(n - rows[b], n, 3), [n - 1], rng.integers(0, n, 1)]))
        for i, key in enumerate(keys):
            h, at = int(rng.integers(Hkv)), (int(c["table"][b][key // page]), int(key % page))
            bad = (np.inf, np.nan)[i % 2]
            c["cache"][3][1, at[0], h, at[1]] = bad
            for r in range(rows[b]):
                pos = n - rows[b] + r
                if max(0, pos + 1 - window if window else 0) <= key <= pos:
                    with np.errstate(invalid="ignore"):
                        want[1, int(c["starts"][b]) + r, h * 2: h * 2 + 2] += c["v64"][1, at[0], h, at[1]] * bad
    again, lse2, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    got = host_f64(again).reshape(want.shape)
    assert np.array_equal(got, want, equal_nan=True), np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))[:5]
    assert torch.equal(lse, lse2)
