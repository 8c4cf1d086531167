"""Infinities in low-rank adapters and their rows: what the formula gives, with few rows and
with many."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st
from helpers import dev_tensor, host_f64
from sequence_tensor_transformer_gb300 import synth

from test_gpu_lora import BOTH, TYPES, arguments, make

pytestmark = pytest.mark.gpu

ROWS = pytest.mark.parametrize("M", [30, 300])
RANKS = pytest.mark.parametrize("R", [8, 16, 32, 64, 128])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


def shape_of(a):
    """0: finite, 1 and -1: an infinity, 2: NaN."""
    return np.where(np.isnan(a), 2, np.where(np.isinf(a), np.sign(np.nan_to_num(a, posinf=1, neginf=-1)), 0))


def formula(c, x, A, B):
    out = c["base64"].copy()
    P, n = c["P"], c["base64"].shape[2]
    with np.errstate(invalid="ignore"):
        for m, a in enumerate(c["ids"]):
            if a < 0:
                continue
            for p in range(P):
                if c["rowwise"]:
                    f = c["K"] // P
                    t, up = A[a][:, p * f:(p + 1) * f] @ x[p, m], B[a]
                else:
                    t, up = A[a] @ x[m], B[a][p * n:(p + 1) * n]
                out[p, m] += float(c["gains"][a]) * (up @ t)
    return out


@BOTH
@TYPES
@RANKS
@ROWS
@pytest.mark.parametrize("where", ["x", "A", "B", "base"])
def test_infinities_are_those_of_the_formula(where, M, R, dtype, rowwise):
    c = make(2, M, 64, 80, R, 3, dtype, rowwise)
    v64 = {k: c[k + "64"].copy() for k in ("x", "A", "B", "base")}
    at = {"x": (..., 4, 7), "A": (1, 3, 5), "B": (1, slice(None, None, 3), R - 1), "base": (1, 9, 11)}[where]
    for sign in (1, -1):
        for k in v64:
            v64[k] = c[k + "64"].copy()
        v64[where][at] = sign * np.inf
        t = c[where].clone()
        t[at] = sign * float("inf")
        args, kw = arguments({**c, where: t})
        ref = formula({**c, "base64": v64["base"]}, v64["x"], v64["A"], v64["B"])
        got = host_f64(st.sptp_lora(*args, **kw))
        assert np.array_equal(shape_of(got), shape_of(ref))


@BOTH
@ROWS
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_products_between_the_largest_numbers_of_bf16_and_fp32(dtype, M, rowwise):
    """A row times A gives 3.3995e38, above bf16's largest and below fp32's; times B it is 3.2e32."""
    R, K, N, big = 16, 32, 48, 255 / 128 * 2.0 ** 127
    A, B = np.zeros((1, R, K), np.float32), np.full((1, N, R), 2.0 ** -20, np.float32)
    A[0, 0, :2] = big, 1e36
    x = np.ones((1, M, K) if rowwise else (M, K), np.float32)
    A, B, x, base = (dev_tensor(synth._cast(a, dtype), dtype) for a in (A, B, x, np.zeros((1, M, N), np.float32)))
    got = host_f64(st.sptp_lora(x, A, B, torch.zeros(M, dtype=torch.int32, device="cuda"), base))
    want = (big + float(A[0, 0, 1])) * 2.0 ** -20
    assert want * 2.0 ** 20 < np.finfo(np.float32).max
    assert np.all(np.abs(got - want) <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22) * want)
