"""Calls of the rotation, the append and the one-token attention that a user's
program makes and that no parity test covers: shared pages, many sequences,
non-finite values of others, streams and graphs that share a workspace,
refusals of strided tensors, prompts with bad indexes."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st
from sequence_tensor_transformer_gb300 import synth

import test_gpu_paged_attn as ta
import test_gpu_rope_cache as tr
from helpers import dev_tensor, nan_tensor, nan_workspace, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ta.KINDS)
def test_sequences_share_pages(kind):
    """Sequences with one prefix, and a page twice in one sequence."""
    c = ta.make(2, [200, 200, 130], 4, 2, 64, 16, kind)
    t = c["table"]
    t[1, :8] = t[0, :8]
    t[2, 3] = t[2, 1]
    out, lse, ws = ta.call(c)
    assert st.sptp_read_device_status(ws) == 0
    ta.check(c, out, lse)
    assert torch.equal(out[:, 0], ta.call(dict(c, table=np.concatenate([t[:1], t[:1], t[2:]])))[0][:, 0])


@pytest.mark.parametrize("kind", ta.KINDS)
def test_thousands_of_sequences(kind):
    """Every thread of a CTA adds up a run of lengths."""
    lens = np.random.default_rng(0).integers(0, 40, 3000)
    lens[[0, 1499, 2999]] = 0, 37, 0
    c = ta.make(1, lens, 2, 2, 16, 16, kind)
    out, lse, ws = ta.call(c)
    assert st.sptp_read_device_status(ws) == 0
    ta.check(c, out, lse)


def test_one_sequence_of_a_wide_table():
    """A table far longer than the sequence: the grid is the table's, the work the length's."""
    c = ta.make(1, [40], 4, 1, 128, 16, "bf16")
    wide = np.full((1, 60000), -1)
    wide[:, : c["table"].shape[1]] = c["table"]
    out, lse, ws = ta.call(c, page_table=ta.ints(wide))
    assert st.sptp_read_device_status(ws) == 0
    ta.check(c, out, lse)


@pytest.mark.parametrize("kind", ta.KINDS)
def test_non_finite_values_stay_where_they_are(kind):
    """A NaN query, or NaN keys and values of a sequence, reach that head's, that
    sequence's rows alone."""
    c = ta.make(1, [100, 70, 300], 8, 2, 64, 16, kind)
    ref, ref_lse, _ = ta.call(c)
    q = c["q"].clone()
    q[0, 1, 2] = float("nan")
    out, lse, ws = ta.call(dict(c, q=q))
    keep = torch.ones(1, 3, 8, dtype=torch.bool, device="cuda")
    if kind == "e4m3":  # non-finite queries are outside an E4M3 cache's contract for their own row alone
        keep[0, 1, 2] = False
    else:
        assert torch.isnan(out.view(1, 3, 8, 64)[0, 1, 2]).all() and torch.isnan(lse[0, 1, 2])
        keep[0, 1, 2] = False
    assert torch.equal(out.view(1, 3, 8, 64)[keep], ref.view(1, 3, 8, 64)[keep]) and torch.equal(lse[keep], ref_lse[keep])
    if kind == "e4m3":
        return
    k, v = c["cache"][0].clone(), c["cache"][1].clone()
    page = int(c["table"][2, 0])
    k[0, page, 1] = float("nan")
    v[0, page, 1] = float("inf")
    out, lse, ws = ta.call(dict(c, cache=(k, v, None, None)))
    keep[:] = True
    keep[0, 2, 4:] = False
    assert torch.equal(out.view(1, 3, 8, 64)[keep], ref.view(1, 3, 8, 64)[keep])


def test_large_groups_and_teams_of_uneven_heads():
    for kind in ta.KINDS:
        for Hq, D in ((9, 64), (17, 128), (31, 64), (33, 128), (11, 256), (96, 64)):
            c = ta.make(1, [70, 200], Hq, 1, D, 16, kind, seed=Hq)
            out, lse, ws = ta.call(c)
            assert st.sptp_read_device_status(ws) == 0
            ta.check(c, out, lse)


def test_outputs_left_out_on_a_stream_of_its_own():
    """stream= with outputs and workspaces left out, while the current stream
    is busy: they are the call's stream's."""
    c = ta.make(2, [300, 40], 8, 2, 64, 16, "bf16")
    table, lens = ta.ints(c["table"]), ta.ints(c["lens"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    got = []
    for _ in range(4):
        for _ in range(4):
            busy = busy @ busy * 1e-3
        got.append(st.sptp_paged_attn_decode(c["q"], c["cache"], table, lens, c["scale"], stream=side))
    side.synchronize()
    for out, lse in got:
        ta.check(c, out, lse)
    x = torch.randn(2, 9, 4, 64, device="cuda")
    turns = st.sptp_rope_turns(64)
    torch.cuda.synchronize()
    y = st.sptp_rope(x, tr.ints(range(9)), turns, stream=side)
    side.synchronize()
    assert torch.equal(y, st.sptp_rope(x, tr.ints(range(9)), turns))


def test_two_graphs_share_a_workspace():
    """An append and an attention, each captured with the same workspace, and
    the attention of another batch captured with it too, replayed in turn."""
    rng = np.random.default_rng(2)
    P, B, Hq, Hkv, D, page = 2, 3, 4, 2, 64, 16
    c = ta.make(P, [50, 20, 33], Hq, Hkv, D, page, "bf16")
    other = ta.make(1, [400, 900], 6, 3, 64, 16, "bf16", seed=5)
    n = max(st.sptp_paged_attn_workspace_size(P, B, Hq, Hkv, D), st.sptp_paged_attn_workspace_size(1, 2, 6, 3, 64))
    ws = nan_workspace(n)
    qkv = torch.zeros(P, B, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda")
    cache = tuple(t.clone() for t in c["cache"][:2]) + (None, None)
    table, pos, lens = ta.ints(c["table"]), ta.ints([49, 19, 32]), ta.ints([50, 20, 33])
    seq, turns = ta.ints(range(B)), st.sptp_rope_turns(D)
    q, out, lse = (nan_tensor(s, t) for s, t in (((P, B, Hq, D), torch.bfloat16), ((P, B, Hq * D), torch.bfloat16), ((P, B, Hq), torch.float32)))
    out2, lse2 = nan_tensor((1, 2, 6 * 64)), nan_tensor((1, 2, 6), torch.float32)
    t2, l2 = ta.ints(other["table"]), ta.ints(other["lens"])
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        st.sptp_rope_append_kv(qkv, pos, seq, table, turns, cache, Hq, q_out=q, workspace=ws)
        st.sptp_paged_attn_decode(q, cache, table, lens, out=out, lse=lse, workspace=ws)
    with torch.cuda.graph(g2):
        st.sptp_paged_attn_decode(other["q"], other["cache"], t2, l2, out=out2, lse=lse2, workspace=ws)
    for _ in range(3):
        x = synth._cast(rng.standard_normal(tuple(qkv.shape)), "bf16")
        qkv.copy_(dev_tensor(x, "bf16"))
        ws.fill_(0xFF)
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert st.sptp_read_device_status(ws) == 0
        ta.check(other, out2, lse2)
        now = dict(c, q64=to_f64(q.view(torch.int16).cpu().numpy().view(np.uint16), "bf16"),
                   k64=cache[0].float().cpu().double().numpy(), v64=cache[1].float().cpu().double().numpy())
        ta.check(now, out, lse)
        want = tr.ao.rope(to_f64(x, "bf16").reshape(P, B, -1, D), tr.angles([49, 19, 32], turns), Hq + Hkv)
        tr.close(q.float().cpu().double().numpy(), want[:, :, :Hq],
                 tr.ao.rope_pair_sizes(to_f64(x, "bf16").reshape(P, B, -1, D), D // 2, Hq)[:, :, :Hq], "bf16")


def test_strided_tensors_are_refused():
    c = ta.make(1, [30], 4, 2, 64, 16, "bf16")
    table, lens = ta.ints(c["table"]), ta.ints(c["lens"])
    wide = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16, device="cuda")[..., :64]
    with pytest.raises(ValueError, match="contiguous"):
        st.sptp_paged_attn_decode(wide, c["cache"], table, lens)
    k = c["cache"][0].transpose(2, 3).contiguous().transpose(2, 3)
    with pytest.raises(ValueError, match="contiguous"):
        st.sptp_paged_attn_decode(c["q"], (k, c["cache"][1], None, None), table, lens)
    x = torch.zeros(1, 5, 4, 64, device="cuda").transpose(1, 2)
    with pytest.raises(ValueError, match="contiguous"):
        st.sptp_rope(x, ta.ints(range(4)), st.sptp_rope_turns(64))
    # a slice of a larger table or list that is itself dense is fine
    lens2 = ta.ints([0, 30])[1:]
    out, _ = st.sptp_paged_attn_decode(c["q"], c["cache"], table, lens2)
    assert torch.equal(out, st.sptp_paged_attn_decode(c["q"], c["cache"], table, lens)[0])


@pytest.mark.parametrize("P,M,Hq,Hkv,D", [(1, 2049, 1, 1, 16), (1, 5000, 1, 1, 16), (4, 2100, 14, 2, 128)])
def test_long_prompts_with_a_bad_row(P, M, Hq, Hkv, D):
    """Both ways in which an append of many rows reports a bad index, whichever row it is."""
    c = tr.append_case(P, M, Hq, Hkv, D, 16, M // 100 + 1, 16, "bf16", False, False, pad=0)
    turns = st.sptp_rope_turns(16)
    ws = nan_workspace(4096)
    qkv, pos, table = dev_tensor(c["qkv"], "bf16"), tr.ints(c["pos"]), tr.ints(c["table"])
    for row in (0, 1024, M - 1):
        seq = c["seq"].copy()
        seq[row] = c["table"].shape[0] + 3
        q = nan_tensor((P, M, Hq, D))
        for t in c["cache"][:2]:
            t.fill_(float("nan"))
        st.sptp_rope_append_kv(qkv, pos, tr.ints(seq), table, turns, c["cache"], Hq, q_out=q, workspace=ws)
        assert st.sptp_read_device_status(ws) == st.STATUS["shape"]
        assert ws[:20].view(torch.int32).tolist()[3] == row
    st.sptp_rope_append_kv(qkv, pos, tr.ints(c["seq"]), table, turns, c["cache"], Hq, q_out=q, workspace=ws)
    assert st.sptp_read_device_status(ws) == 0
    tr.check_append(c, turns, q)


def test_append_then_attend_prefix_then_grow():
    """A sequence grown token by token equals one appended at once: the cache's
    bits, and the attention's."""
    P, Hq, Hkv, D, page, n = 1, 4, 2, 128, 16, 37
    x = torch.randn(P, n, (Hq + 2 * Hkv) * D, device="cuda").bfloat16()
    turns = st.sptp_rope_turns(D)
    table = ta.ints([[3, 0, 2]])
    for e4m3 in (False, True):
        a, b = (st.paged_kv_cache(P, 4, Hkv, page, D, e4m3=e4m3) for _ in range(2))
        qa = st.sptp_rope_append_kv(x, ta.ints(range(n)), ta.ints([0] * n), table, turns, a, Hq)
        for j in range(n):
            qb = st.sptp_rope_append_kv(x[:, j: j + 1].contiguous(), ta.ints([j]), ta.ints([0]), table, turns, b, Hq)
        for s, t in zip(a, b):
            assert s is None or torch.equal(s, t)
        assert torch.equal(qa[:, -1:], qb)
        oa, la = st.sptp_paged_attn_decode(qa[:, -1:].contiguous(), a, table, ta.ints([n]))
        ob, lb = st.sptp_paged_attn_decode(qb, b, table, ta.ints([n]))
        assert torch.equal(oa, ob) and torch.equal(la, lb)
