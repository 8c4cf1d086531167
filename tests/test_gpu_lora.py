"""GPU parity of low-rank adapters per row, against the float64 oracle.

Bounds, with S the sum of the terms' sizes: A_a x is a sum of K products in fp32, B_a
times it one of R: (K + R + 8) 2^-24 S; in bf16 the former is held to 2^-16 of itself,
2^-16 S more; the result is rounded once, half a step of it."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st
from oracle import attn_oracle as ao
from sequence_tensor_transformer_gb300 import synth

from batch_cases import HALF, TD
from helpers import dev_tensor, host_f64, nan_tensor, nan_workspace, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


def make(P, M, K, N, R, n, dtype, rowwise, ids=None, gains=True, seed=0):
    rng = np.random.default_rng(seed + M + K)
    cast = lambda a: synth._cast(a, dtype)  # noqa: E731
    c = dict(P=P, M=M, K=K, N=N, R=R, n=n, dtype=dtype, rowwise=rowwise)
    raw = dict(x=cast(rng.standard_normal((P, M, K // P) if rowwise else (M, K))), A=cast(rng.standard_normal((n, R, K)) * K ** -0.5),
               B=cast(rng.standard_normal((n, N, R)) * R ** -0.5),
               base=cast(rng.standard_normal((P, M, N if rowwise else N // P))))
    c["ids"] = rng.integers(-1, n, M) if ids is None else np.asarray(ids)
    c["gains"] = rng.uniform(0.2, 2.0, n).astype(np.float32) if gains else None
    for k, v in raw.items():
        c[k], c[k + "64"] = dev_tensor(v, dtype), to_f64(v, dtype)
    return c


def arguments(c):
    return (c["x"], c["A"], c["B"], torch.from_numpy(c["ids"].astype(np.int32)).cuda(), c["base"]), dict(
        gains=None if c["gains"] is None else torch.from_numpy(c["gains"]).cuda())


def check(c, out):
    ids = np.where(c["ids"] < c["n"], c["ids"], -1)
    ref, size = ao.lora(c["x64"], c["A64"], c["B64"], ids, c["base64"], c["gains"])
    got = host_f64(out)
    assert not np.isnan(got).any()
    tol = ((c["K"] + c["R"] + 8) * 2.0 ** -24 + (2.0 ** -16 if c["dtype"] == "bf16" else 0.0)) * size
    tol += HALF[c["dtype"]] * np.abs(ref) * (1 + 2.0 ** -7)
    none = ids < 0
    assert np.array_equal(got[:, none], c["base64"][:, none])
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], (np.abs(got - ref) / tol).max())


def run(*a, status=0, **kw):
    c = make(*a, **kw)
    args, kws = arguments(c)
    ws = nan_workspace(st.sptp_lora_workspace_size(c["P"], c["M"], c["K"], c["N"], c["R"], c["rowwise"]))
    out = nan_tensor(c["base"].shape, TD[c["dtype"]])
    got = st.sptp_lora(*args, **kws, out=out, workspace=ws)
    assert got is out and st.sptp_read_device_status(ws) == status
    check(c, out)
    # in place: the same bits
    base = c["base"].clone()
    assert st.sptp_lora(*args[:4], base, **kws, out=base) is base and torch.equal(base, out)
    return c, out


BOTH = pytest.mark.parametrize("rowwise", [False, True])
TYPES = pytest.mark.parametrize("dtype", ["bf16", "fp32"])


@BOTH
@TYPES
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 100, 159, 160, 161, 300])
def test_rows(M, dtype, rowwise):
    run(2, M, 128, 96, 16, 5, dtype, rowwise)


@BOTH
@TYPES
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 120, 128])
@pytest.mark.parametrize("M", [20, 200])
def test_ranks(M, R, dtype, rowwise):
    run(1, M, 256, 136, R, 3, dtype, rowwise)


@BOTH
@TYPES
@pytest.mark.parametrize("P,K,N", [(1, 8, 8), (1, 40, 24), (3, 120, 72), (8, 192, 64), (4, 1000 * 4, 8 * 4), (2, 16, 2064)])
@pytest.mark.parametrize("M", [33, 170])
def test_sizes(M, P, K, N, dtype, rowwise):
    run(P, M, K, N, 16, 4, dtype, rowwise)


@BOTH
@TYPES
def test_many_rows(dtype, rowwise):
    # runs of rows with one adapter, and one tile of 16 with all of them
    ids = np.repeat(np.arange(9) % 4, 260)[:2100]
    ids[512:528] = np.arange(16) % 5 - 1
    run(2, 2100, 64, 80, 32, 4, dtype, rowwise, ids=ids)


@BOTH
@TYPES
def test_every_row_its_own_adapter_in_any_order(dtype, rowwise):
    run(2, 180, 64, 80, 16, 180, dtype, rowwise, ids=np.random.default_rng(1).permutation(180))


@BOTH
@TYPES
def test_long_rows_are_split(dtype, rowwise):
    run(1, 20, 8192 + 24, 64, 16, 3, dtype, rowwise)
    run(1, 3, 70000, 16, 8, 2, dtype, rowwise)


@TYPES
def test_without_adapters_and_without_gains(dtype):
    run(2, 40, 64, 80, 16, 3, dtype, False, gains=False)
    run(2, 40, 64, 80, 16, 3, dtype, False, ids=np.full(40, -1))
    run(2, 200, 64, 80, 16, 3, dtype, True, ids=np.full(200, -7))
    run(2, 20, 64, 80, 16, 0, dtype, False, ids=np.full(20, -1))


@BOTH
@TYPES
@pytest.mark.parametrize("M", [30, 300])
def test_adapters_out_of_range_are_reported(M, dtype, rowwise):
    ids = np.arange(M) % 3
    ids[[7, M - 1]] = 3, 2 ** 31 - 1
    run(2, M, 64, 80, 16, 3, dtype, rowwise, ids=ids, status=st.STATUS["shape"])


@BOTH
@TYPES
@pytest.mark.parametrize("M", [30, 300])
def test_another_adapters_infinities_do_not_reach_a_row(M, dtype, rowwise):
    c = make(2, M, 64, 80, 16, 3, dtype, rowwise)
    args, kw = arguments(c)
    want = st.sptp_lora(*args, **kw)
    A, B = c["A"].clone(), c["B"].clone()
    A[1, 3, 5], B[1, ::2] = float("nan"), float("inf")
    got = st.sptp_lora(args[0], A, B, *args[3:], **kw)
    others = torch.from_numpy(c["ids"] != 1).cuda()
    assert torch.equal(got[:, others], want[:, others]) and not torch.isfinite(got[:, ~others]).all()
    # nor another row's
    x = c["x"].clone()
    x[..., 4, :] = float("nan")
    got = st.sptp_lora(x, *args[1:], **kw)
    rest = torch.arange(M, device="cuda") != 4
    assert torch.equal(got[:, rest], want[:, rest])


@TYPES
@pytest.mark.parametrize("M", [30, 300])
def test_a_row_does_not_depend_on_its_neighbours(M, dtype):
    c = make(1, M, 512, 80, 16, 4, dtype, False, ids=np.full(M, 2))
    args, kw = arguments(c)
    want = st.sptp_lora(*args, **kw)
    ids = args[3].clone()
    ids[1::2] = torch.arange(M // 2, device="cuda", dtype=torch.int32) % 5 - 1
    got = st.sptp_lora(*args[:3], ids, args[4], **kw)
    if dtype == "bf16":  # (how the sums along K are split depends on how many adapters 16 rows name)
        check({**c, "ids": ids.cpu().numpy()}, got)
    else:
        assert torch.equal(got[:, ::2], want[:, ::2])
    assert torch.equal(got, st.sptp_lora(*args[:3], ids, args[4], **kw))
