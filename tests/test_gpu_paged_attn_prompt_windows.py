"""Prompts' attention of rows that see long runs of keys between a window's lower edge and
their own position: many tiles of keys that every row of an item sees between two that some do not,
and several items in a CTA's share."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

from batch_cases import call, make
from helpers import host_f64
from prompt_reference import compare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


def run(c):
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    compare(c, out, lse)
    for _ in range(4):
        again, lse2, ws = call(c)
        assert st.sptp_read_device_status(ws) == 0
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1000, 2048, 4096])
def test_windows_of_many_tiles(kind, D, window):
    # some 16 to 40 tiles a share
    run(make(2, (4096,), (6000,), 8, 8, D, 64, kind, window=window, first=1, pad=2))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap,slope", [(0.0, 0.0), (20.0, 0.0), (0.0, 0.01), (20.0, 0.01)])
def test_windows_over_several_sequences(D, cap, slope):
    run(make(2, (1500, 2000, 3, 700), (1500, 4000, 3001, 2500), 6, 3, D, 16, "bf16", window=1333, cap=cap,
             slopes=np.full(12, slope) if slope else None))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_items_without_a_window(D):
    # the last tiles of an item still on their way when the next one's first are due
    run(make(4, (300, 1200), (1300, 1200), 16, 16, D, 32, "bf16"))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1000, 2048])
def test_values_that_are_not_finite_at_both_edges(D, window):
    P, rows, n, page = 2, 3000, 5000, 16
    c = make(P, (rows,), (n,), 8, 8, D, page, "bf16", window=window)
    out, lse, _ = call(c)
    want = host_f64(out).reshape(P, rows, 8, D).copy()
    rng = np.random.default_rng(3)
    pos = n - rows + np.arange(rows)
    v = c["cache"][1]
    for i, key in enumerate(np.unique(rng.integers(n - rows - window + 1, n, 40))):
        p, h, d, x = int(rng.integers(P)), int(rng.integers(8)), int(rng.integers(D)), (np.inf, -np.inf, np.nan)[i % 3]
        v[p, int(c["table"][0][key // page]), h, key % page, d] = x
        with np.errstate(invalid="ignore"):
            want[p, (pos >= key) & (pos < key + window), h, d] += x
    for _ in range(3):
        again, lse2, ws = call(c)
        assert st.sptp_read_device_status(ws) == 0
        assert np.array_equal(host_f64(again).reshape(want.shape), want, equal_nan=True)
        assert torch.equal(lse, lse2)
