"""Adapters as an argument of the projections: refused before anything is enqueued, and their
status where the caller looks for it."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

from helpers import nan_workspace

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SHAPE, TIMEOUT = st.STATUS["shape"], st.STATUS["timeout"]
P, M, d, N, R, n = 2, 64, 128, 256, 16, 3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)
    torch.manual_seed(0)


def randn(*s):
    return torch.randn(*s, device="cuda").to(BF)


def adapters(K, N, **kw):
    a = dict(A=randn(n, R, K), B=randn(n, N, R), ids=torch.arange(M, device="cuda", dtype=torch.int32) % n,
             gains=torch.ones(n, device="cuda"))
    a.update({k: v for k, v in kw.items() if k in a})
    return tuple(a.values())


def down(adapters, ws=None, **kw):
    out = kw.pop("out", None)
    return st.sptp_down_proj(kw.pop("s"), kw.pop("W2"), P, out=out, workspace=ws, adapters=adapters, **kw)


def qkv(adapters, ws=None, **kw):
    out = kw.pop("out", None)
    return st.sptp_attn_qkv_forward(kw.pop("s"), torch.zeros(P, M, d, dtype=BF, device="cuda"), torch.ones(d, dtype=BF, device="cuda"),
                                    kw.pop("W2"), P, 2, 1e-6, qkv_out=out, workspace=ws, adapters=adapters, **kw)[0]


def setup(which):
    """(call, its tensors, shape of out, the adapters' K and N, workspace bytes)"""
    if which == "down":
        return down, dict(s=randn(P, M, N // P), W2=randn(d, N)), (P, M, d), (N, d), 4096
    return qkv, dict(s=randn(M, d), W2=randn(N, d)), (P, M, N // P), (d, N), st.sptp_attn_qkv_workspace_size(M, d, N, P, 2)


BOTH = pytest.mark.parametrize("which", ["down", "qkv"])


@BOTH
@pytest.mark.parametrize("wrong", ["A", "B", "ids", "gains", "type", "rank", "workspace", "overlap"])
def test_adapters_that_are_refused_leave_the_output_as_it_was(which, wrong):
    call, tensors, shape, (K, n_out), size = setup(which)
    out, kw = torch.full(shape, 7.0, dtype=BF, device="cuda"), {}
    right = dict(zip(("A", "B", "ids", "gains"), adapters(K, n_out)))
    if wrong == "type":
        right["A"] = right["A"].float()
    elif wrong == "rank":
        right["A"], right["B"] = right["A"][:, :12].contiguous(), right["B"][:, :, :12].contiguous()
    elif wrong == "workspace":
        kw["adapter_workspace"] = nan_workspace(256)
    elif wrong == "overlap":
        right["A"] = out.view(-1)[: R * K].view(1, R, K)
        right["B"], right["gains"] = right["B"][:1], right["gains"][:1]
    else:
        right[wrong] = right[wrong][:-1]
    ws = nan_workspace(size)
    with pytest.raises((ValueError, TypeError, st.SptpError)):
        call(tuple(right.values()), ws, **tensors, out=out, **kw)
    torch.cuda.synchronize()
    assert (out == 7.0).all() and (ws == 0xFF).all()


@BOTH
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("bad", [None, n, 2 ** 31 - 1])
def test_the_status_is_where_it_is_looked_for(which, own, bad):
    call, tensors, shape, (K, n_out), size = setup(which)
    a = adapters(K, n_out)
    if bad is not None:
        a[2][5] = bad
    ws, aws = nan_workspace(size), nan_workspace(st.sptp_lora_workspace_size(P, M, K, n_out, R, which == "down"))
    kw = dict(adapter_workspace=aws) if own else {}
    out = call(a, ws, **tensors, **kw)
    status = 0 if bad is None else SHAPE
    assert st.sptp_read_device_status(ws) == (0 if own else status)
    assert st.sptp_read_device_status(aws) == (status if own else -1)  # (not used: as it was)
    if status and not own:
        assert ws.view(torch.int32)[3].item() == 5  # the row
    # the row is treated as one without adapter, and the other form gives the same bits
    plain = call(None, nan_workspace(size), **tensors)
    want = call(a, nan_workspace(size), **tensors, **({} if own else dict(adapter_workspace=aws)))
    assert torch.equal(out, want) and (bad is None or torch.equal(out[:, 5], plain[:, 5]))
    assert not torch.equal(out[:, 6], plain[:, 6])
    # what a call before recorded is gone
    assert st.sptp_read_device_status(ws) == (0 if own else status)
    a[2][5] = 0
    call(a, ws, **tensors, **kw)
    assert st.sptp_read_device_status(ws) == 0


def test_another_call_s_error_is_kept():
    A, B, ids, gains = adapters(d, N)
    ids[3] = n
    x, out = randn(M, d), randn(P, M, N // P)
    ws, status = nan_workspace(st.sptp_lora_workspace_size(P, M, d, N, R)), torch.zeros(4096, dtype=torch.uint8, device="cuda")
    args = (x.data_ptr(), A.data_ptr(), B.data_ptr(), ids.data_ptr(), gains.data_ptr(), P, M, d, N, R, n, 0, 0, out.data_ptr(),
            out.data_ptr(), ws.data_ptr(), ws.nbytes, torch.cuda.current_stream().cuda_stream, status.data_ptr())
    for code in (0, TIMEOUT):
        status.view(torch.int32)[0] = code
        assert st.lib().sptp_lora_ex(*args, 0) == 0
        assert st.sptp_read_device_status(status) == (code or SHAPE)


def test_a_workspace_of_another_type():
    call, tensors, shape, (K, n_out), size = setup("qkv")
    a = adapters(K, n_out)
    want = call(a, nan_workspace(size), **tensors)
    ws = torch.zeros(2, size // 8 + 1, device="cuda")  # fp32
    assert torch.equal(call(a, ws, **tensors), want)


@BOTH
def test_without_rows(which):
    A, B, _, gains = adapters(N if which == "down" else d, d if which == "down" else N)
    ids = torch.zeros(0, dtype=torch.int32, device="cuda")
    if which == "down":
        assert st.sptp_down_proj(randn(P, 0, N // P), randn(d, N), P, adapters=(A, B, ids, gains)).shape == (P, 0, d)
    else:
        out = st.sptp_attn_qkv_forward(randn(0, d), randn(P, 0, d), randn(d), randn(N, d), P, 2, 1e-6, adapters=(A, B, ids, gains))[0]
        assert out.shape == (P, 0, N // P)
