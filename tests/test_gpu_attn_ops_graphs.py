"""Captured calls of the rotation, the append and the one-token attention beside
other work: behind copies, fills and joined streams, which are no kernels whose
end a launch could overlap, and the append that clears its status words first."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

import test_gpu_paged_attn as ta
import test_gpu_rope_cache as tr
from helpers import dev_tensor, nan_tensor, nan_workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("M", [2048, 2049, 5000])
def test_append_of_many_small_rows_captured(M, e4m3):
    """Rows of 96 bytes: up to 2048 of them a block checks their indexes, above
    the words are cleared first.  Every replay's status is its own."""
    c = tr.append_case(1, M, 1, 1, 16, 16, M // 100 + 1, 16, "bf16", e4m3, False, pad=3)
    turns = st.sptp_rope_turns(16)
    ws = nan_workspace(4096)
    qkv, pos, seq, table = dev_tensor(c["qkv"], "bf16"), tr.ints(c["pos"]), tr.ints(c["seq"]), tr.ints(c["table"])
    q = nan_tensor((1, M, 1, 16))
    st.sptp_rope_append_kv(qkv, pos, seq, table, turns, c["cache"], 1, q_out=q, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.sptp_rope_append_kv(qkv, pos, seq, table, turns, c["cache"], 1, q_out=q, workspace=ws)
    for bad in (M - 1, None, 0, 1500, None):
        s = c["seq"].copy()
        if bad is not None:
            s[bad] = c["table"].shape[0] + 3
        seq.copy_(tr.ints(s))
        for t in (q, *c["cache"]):
            if t is not None:
                t.fill_(0xFF if t.dtype == torch.uint8 else float("nan"))
        g.replay()
        assert st.sptp_read_device_status(ws) == (0 if bad is None else st.STATUS["shape"])
        if bad is None:
            tr.check_append(c, turns, q)
        else:
            assert ws[:20].view(torch.int32).tolist()[3] == bad


def test_captured_behind_copies_fills_and_joined_streams():
    """Inputs that the same graph makes: copied, filled, and made on a second
    stream that is joined right before the call; each replay on new values."""
    P, B, Hq, Hkv, D, page = 2, 3, 4, 2, 64, 16
    a, b = (ta.make(P, [50, 20, 33], Hq, Hkv, D, page, "bf16", seed=s) for s in (1, 2))
    src = [t.clone() for t in (a["q"], *a["cache"][:2])]
    q, k, v = (nan_tensor(t.shape) for t in src)
    table, lens, lens_src = ta.ints(a["table"]), ta.ints([0, 0, 0]), ta.ints(a["lens"])
    ws = nan_workspace(st.sptp_paged_attn_workspace_size(P, B, Hq, Hkv, D))
    out, lse = nan_tensor((P, B, Hq * D)), nan_tensor((P, B, Hq), torch.float32)
    x, turns, pos = torch.randn(P, B, Hq, D, device="cuda"), st.sptp_rope_turns(D), ta.ints([3, 9, 70])
    y = torch.empty_like(x)
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            k.copy_(src[1])
            torch.mul(src[2], 1, out=v)
        q.copy_(src[0])
        lens.copy_(lens_src)
        main.wait_stream(side)
        st.sptp_paged_attn_decode(q, (k, v, None, None), table, lens, a["scale"], out=out, lse=lse, workspace=ws)
        # and a call on the second stream behind the first one's
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.mul(x, 2, out=y)
            st.sptp_rope(y, pos, turns, out=y)
        main.wait_stream(side)
        st.sptp_rope(y, pos, turns, transpose=True, out=y)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for c in (b, a, b):
        for t, new in zip(src, (c["q"], *c["cache"][:2])):
            t.copy_(new)
        table.copy_(ta.ints(c["table"]))
        x.normal_()
        for t in (q, k, v, out, lse, y):
            t.fill_(float("nan"))
        ws.fill_(0xFF)
        g.replay()
        assert st.sptp_read_device_status(ws) == 0
        ta.check(c, out, lse)
        # rotated and back: the sum of squares of a pair is kept to a few roundings
        assert torch.allclose(y, 2 * x, atol=2e-5)


def test_eager_behind_joined_streams():
    """The same order of streams without a graph, while both are busy."""
    c = ta.make(2, [400, 31, 0, 200], 4, 2, 64, 16, "bf16")
    table, lens = ta.ints(c["table"]), ta.ints(c["lens"])
    torch.cuda.synchronize()
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    big = torch.randn(2048, 2048, device="cuda")
    ref, ref_lse = st.sptp_paged_attn_decode(c["q"], c["cache"], table, lens)
    for _ in range(5):
        q = nan_tensor(c["q"].shape)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(3):
                big = big @ big * 1e-2
            q.copy_(c["q"])
        main.wait_stream(side)
        out, lse = st.sptp_paged_attn_decode(q, c["cache"], table, lens)
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
