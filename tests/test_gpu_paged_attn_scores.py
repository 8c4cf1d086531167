"""GPU parity of the one-token attention with a cap on the scores and a bias by
distance, against the float64 oracle (bounds: batch_cases.check; E4M3 weights are fp16
there, finer than the bf16 that the bounds allow for)."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

from batch_cases import TD, check, ints, make
from helpers import nan_workspace

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp32", "e4m3"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


def slopes_of(kind, n):
    return {None: None, "usual": 2.0 ** (-8.0 * np.arange(1, n + 1) / n), "mixed": np.linspace(-0.02, 0.3, n)}[kind]


def run(lens, Hq, Hkv, D, kind, P=2, page=16, **kw):
    # a row per sequence; empty ones have none in the oracle's case and zeros here
    lens = np.asarray(lens)
    c = make(P, (lens > 0).astype(int), lens, Hq, Hkv, D, page, kind, **kw)
    have = np.flatnonzero(lens > 0)
    q = torch.full((P, len(lens), Hq, D), 3.0, dtype=TD[c["dtype"]], device="cuda")
    q[:, torch.from_numpy(have).cuda()] = c["q"]
    ws = nan_workspace(st.sptp_paged_attn_workspace_size(P, len(lens), Hq, Hkv, D))
    slopes = None if c["slopes"] is None else torch.from_numpy(c["slopes"]).cuda()
    out, lse = st.sptp_paged_attn_decode(q, c["cache"], ints(c["table"]), ints(lens), c["scale"], c["window"], workspace=ws,
                                         cap=c["cap"], slopes=slopes)
    assert st.sptp_read_device_status(ws) == 0
    pick = torch.from_numpy(have).cuda()
    check(c, out[:, pick], lse[:, pick])
    none = torch.from_numpy(np.flatnonzero(lens == 0)).cuda()
    assert not out[:, none].any() and torch.isneginf(lse[:, none]).all()
    return c, q, out, lse, slopes


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cap", [0.0, 2.0, 30.0, 300.0])
@pytest.mark.parametrize("slopes", [None, "usual", "mixed"])
@pytest.mark.parametrize("D", [64, 128])
def test_caps_and_biases(kind, cap, slopes, D):
    run((1, 0, 40, 700, 129), 4, 2, D, kind, q_std=4.0, cap=cap, slopes=slopes_of(slopes, 8))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (9, 1), (20, 1), (40, 1), (8, 4)])
@pytest.mark.parametrize("D", [48, 128, 256])
def test_groups_and_heads(kind, Hq, Hkv, D):
    run((300, 17), Hq, Hkv, D, kind, P=1, cap=10.0, slopes=slopes_of("usual", Hq))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 100, 4096])
def test_windows(kind, window):
    run((1, 600, 130, 0), 4, 2, 64, kind, window=window, cap=10.0, slopes=slopes_of("usual", 8), page=48)


@pytest.mark.parametrize("kind", KINDS)
def test_a_long_row(kind):
    run((30000, 9), 4, 1, 128, kind, P=1, page=64, cap=20.0, slopes=slopes_of("mixed", 4) / 100)


@pytest.mark.parametrize("kind", KINDS)
def test_neither_is_the_call_without_them(kind):
    c, q, out, lse, _ = run((1, 300, 70), 4, 2, 64, kind)
    zero = st.sptp_paged_attn_decode(q, c["cache"], ints(c["table"]), ints(c["lens"]), c["scale"], slopes=torch.zeros(2, 4, device="cuda"))
    assert torch.equal(zero[0], out) and torch.equal(zero[1], lse)


@pytest.mark.parametrize("kind", KINDS)
def test_the_last_row_of_a_prompt(kind):
    """One token each, by both entry points: the same definition."""
    c, q, out, lse, slopes = run((33, 300, 70), 4, 2, 64, kind, cap=15.0, slopes=slopes_of("usual", 8))
    o, l = st.sptp_paged_attn_prompt(q, c["cache"], ints(c["table"]), ints(c["lens"]), ints(c["starts"]), c["scale"], cap=15.0,
                                     slopes=slopes)
    check(c, o, l)
