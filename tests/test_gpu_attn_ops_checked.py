"""The rotation, the append and the one-token attention through the
bounds-checked build (build(checked=True)): every cache row and TMA box that
the kernels compute is checked against its buffer, a failure would be
reported as SPTP_ERR_BOUNDS in the status words; parity as in the tests of the
ordinary build."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

import test_gpu_paged_attn as ta
import test_gpu_rope_cache as tr
from helpers import dev_tensor, nan_tensor, nan_workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def checked_library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sequence_tensor_transformer_gb300 import build
    path = build.build(checked=True)
    normal = st.load_library()
    torch.cuda.set_device(0)
    st.load_library(path, replace=True)
    yield
    st.set_library(normal)


@pytest.mark.parametrize("kind", ta.KINDS)
@pytest.mark.parametrize("P,lens,Hq,Hkv,D,page,window", [
    (4, [333, 0, 17], 7, 1, 128, 16, 0), (1, [5000, 1, 300], 24, 2, 64, 48, 0), (2, [700, 90], 34, 1, 80, 32, 100), (1, [260, 513], 20, 1, 256, 256, 0)])
def test_decode_checked(P, lens, Hq, Hkv, D, page, window, kind):
    c = ta.make(P, lens, Hq, Hkv, D, page, kind, window=window)
    out, lse, ws = ta.call(c)
    assert st.sptp_read_device_status(ws) == 0
    ta.check(c, out, lse)


def test_decode_bad_page_checked():
    """A page outside the pool is the caller's error, not a bounds failure of
    the kernel: it is caught before any box is asked for."""
    c = ta.make(1, [100, 60], 4, 2, 64, 16, "e4m3")
    table = c["table"].copy()
    table[1, 1] = 1 << 30
    out, lse, ws = ta.call(c, page_table=ta.ints(table))
    assert st.sptp_read_device_status(ws) == st.STATUS["shape"]


@pytest.mark.parametrize("dtype,e4m3", [("bf16", False), ("fp32", False), ("bf16", True)])
@pytest.mark.parametrize("P,M,Hq,Hkv,D,rot,B,page", [(4, 33, 7, 1, 128, 128, 3, 16), (2, 2500, 2, 1, 16, 16, 30, 48), (1, 40, 4, 4, 80, 32, 2, 64)])
def test_append_checked(P, M, Hq, Hkv, D, rot, B, page, dtype, e4m3):
    c = tr.append_case(P, M, Hq, Hkv, D, rot, B, page, dtype, e4m3, False)
    turns = st.sptp_rope_turns(rot)
    ws, q = nan_workspace(st.SPTP_WS_HEADER_BYTES), nan_tensor((P, M, Hq, D), tr.TD[dtype])
    args = (dev_tensor(c["qkv"], dtype), tr.ints(c["pos"]), tr.ints(c["seq"]), tr.ints(c["table"]), turns, c["cache"], Hq)
    st.sptp_rope_append_kv(*args, q_out=q, workspace=ws)
    assert st.sptp_read_device_status(ws) == 0
    tr.check_append(c, turns, q)
    seq = c["seq"].copy()
    seq[M // 2] = B
    st.sptp_rope_append_kv(args[0], args[1], tr.ints(seq), *args[3:], workspace=ws)
    assert st.sptp_read_device_status(ws) == st.STATUS["shape"]


def test_rope_checked():
    x = torch.randn(2, 50, 6, 80, device="cuda")
    turns = st.sptp_rope_turns(48)
    pos = tr.ints(np.arange(50) * 1000)
    y = st.sptp_rope(x, pos, turns, 4, True)
    assert torch.allclose(st.sptp_rope(y, pos, turns, 4, True, transpose=True), x, atol=1e-5)
