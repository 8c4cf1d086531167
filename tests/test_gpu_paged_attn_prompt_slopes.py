"""Steep biases by distance, of prompts' attention: a key's bias is off by 2^-23 of itself, so
that the keys next to a row, whose biases are small, keep their scores."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

from batch_cases import call, make, score_error
from helpers import host_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("slope", [0.7, 5.0, 1000.0, 1e6, 1e37])
@pytest.mark.parametrize("cap,prefix", [(0.0, None), (20.0, None), (0.0, (90, 20)), (20.0, (0, 0))])
def test_steep_biases(kind, D, slope, cap, prefix):
    """lse to the mean, by weight, of its keys' errors: score_error without a bias, and 2^-22 of
    the key's own (2^-23 and its sum with the score), 2^-17 with slopes up to 1; the sum
    over n keys by n 2^-24 of it.  One row and head at a time, in 64 bits."""
    P, Hq, Hkv = 1, 4, 2
    slopes = slope * np.array([1.0, 0.7, 1.3, 0.01])
    c = make(P, (70, 5), (200, 30), Hq, Hkv, D, 16, kind, cap=cap, slopes=slopes, prefix=prefix)
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    out, lse = host_f64(out).reshape(c["M"], Hq, D), host_f64(lse)[0]
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    for b, (n, length) in enumerate(zip(c["rows"], c["lens"])):
        for r in range(n):
            m, pos = c["starts"][b] + r, length - n + r
            at = np.arange(max(pos + 1, 0 if prefix is None else prefix[b]))
            pages, off = c["table"][b][at // 16], at % 16
            for h in range(Hq):
                K, q = c["k64"][0, pages, h // 2, off], c["q64"][0, m, h]
                z = K @ q * c["scale"]
                z = cap * np.tanh(z / cap) if cap else z
                bias = float(c["slopes"][0, h]) * np.abs(pos - at)
                w = np.exp(z - bias - (z - bias).max())
                want = (z - bias).max() + np.log(w.sum())
                w /= w.sum()
                dots = np.abs(K) @ np.abs(q) * c["scale"]
                tol = w @ (score_error(D, dots, bias * (w > 0), cap)) * 1.01 + at.size * 2.0 ** -24 + 2.0 ** -22 * abs(want)
                tol += 2.0 ** -17 if c["slopes"].max() <= 1 else 0.0
                assert abs(lse[m, h] - want) <= tol, (m, h, lse[m, h], want, tol)
