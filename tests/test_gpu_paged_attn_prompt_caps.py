"""Caps far from the scores, of prompts' attention: below an eighth of the cap a score is
off by 2^-22 of itself, however large the cap is."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

from batch_cases import call, make
from prompt_reference import compare

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp32", "e4m3"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


def run(c):
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    # scores below an eighth of the cap: 2^-22 of a score, which is at most `dots`
    compare(c, out, lse, cap_error=lambda dots: 2.0 ** -22 * dots)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("slope", [0.0, 0.25])
@pytest.mark.parametrize("cap", [1e3, 1e4, 1e5, 1e6, 1e7, 1e9, 1e20, 1e30])
def test_caps_far_above_the_scores(kind, D, slope, cap):
    # scores of deviation 3
    run(make(2, (150, 3), (400, 90), 4, 2, D, 16, kind, q_std=3.0, cap=cap, slopes=np.full(8, slope) if slope else None))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_std,scale,cap", [(1e19, 1e-20, 1e30), (1e19, 1e-20, 100.0), (1e10, 1e-11, 1e9)])
def test_small_scales(kind, q_std, scale, cap):
    # scale / cap below the normal numbers of 32 bits, the scores not
    run(make(1, (70, 5), (300, 90), 4, 2, 64, 16, kind, q_std=q_std, scale=scale, cap=cap))


@pytest.mark.parametrize("kind", KINDS)
def test_a_cap_far_below_the_scale(kind):
    """scale / cap beyond the numbers of 32 bits: every score is within 1e-30 of 0, that of a
    query of zeros 0, so that all keys weigh the same."""
    c = make(1, (70, 5), (300, 90), 4, 2, 64, 16, kind, scale=1e10, cap=1e-30)
    c["q64"][:, ::3], c["q"][:, ::3] = 0.0, 0.0
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    compare({**c, "scale": 0.0, "cap": 0.0}, out, lse)
