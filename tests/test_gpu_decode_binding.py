"""The extension module of a decoding step's calls on the GPU: the results, the
outputs it makes and the errors are those of the functions without it."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def loaded():
    st.load_library()
    assert st._fast is not None, "the extension module is not built"


def both_ways(call):
    """The results with the module and without it."""
    results = [call()]
    fast, st._fast = st._fast, None
    try:
        results.append(call())
    finally:
        st._fast = fast
    torch.cuda.synchronize()
    return results


def taken(name, *args):
    """Calls the module alone: it took the call."""
    done = getattr(st._fast, name)(*args)
    assert done is not NotImplemented
    return done


def same(a, b):
    assert (a is None) == (b is None)
    if a is not None:
        assert a.shape == b.shape and a.dtype == b.dtype and a.device == b.device
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def inputs(kind, P=2, M=5, Hq=4, Hkv=2, D=64, B=3, page=16, pages=4):
    g = torch.Generator(device="cuda").manual_seed(7)
    dt = torch.float32 if kind == "fp32" else torch.bfloat16
    qkv = torch.randn(P, M, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(dt)
    pos = torch.arange(M, dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, 0, 1, 2, -1], dtype=torch.int32, device="cuda")
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    turns = st.sptp_rope_turns(D, device="cuda")
    cache = st.paged_kv_cache(P, B * pages, Hkv, page, D, dt, kind == "e4m3")
    ws = torch.empty(st.sptp_paged_attn_workspace_size(P, B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    return qkv, pos, seq, table, turns, cache, ws


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("interleaved,transpose,Hr", [(False, False, None), (True, True, 3), (False, True, 1)])
def test_rope(kind, given, interleaved, transpose, Hr):
    dt = torch.float32 if kind == "fp32" else torch.bfloat16
    x = torch.randn(2, 5, 4, 64, device="cuda").to(dt)
    pos, turns = torch.arange(5, dtype=torch.int32, device="cuda"), st.sptp_rope_turns(64, device="cuda")
    out = torch.empty_like(x) if given else None
    if given:
        assert taken("rope", x, pos, turns, Hr, interleaved, transpose, 1.5, out) is out
    else:
        taken("rope", x, pos, turns, Hr, interleaved, transpose, 1.5, None)
    a, b = both_ways(lambda: st.sptp_rope(x, pos, turns, Hr, interleaved, transpose, 1.5, out).clone())
    same(a, b)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("given", [False, True])
def test_append_then_decode(kind, given):
    qkv, pos, seq, table, turns, cache, ws = inputs(kind)
    q_out = torch.empty(2, 5, 4, 64, dtype=qkv.dtype, device="cuda") if given else None

    def append():
        for t in cache:
            if t is not None:
                t.zero_()
        if q_out is not None:
            q_out.zero_()
        q = st.sptp_rope_append_kv(qkv, pos, seq, table, turns, cache, 4, q_out=q_out, workspace=ws)
        return [q[:, :4].clone()] + [None if t is None else t.clone() for t in cache]

    taken("append", qkv, pos, seq, table, turns, cache, 4, False, 1.0, q_out, ws)
    for a, b in zip(*both_ways(append)):
        same(a, b)
    assert st.sptp_read_device_status(ws) == 0

    q = torch.randn(2, 3, 4, 64, device="cuda").to(qkv.dtype)
    lens = torch.tensor([2, 3, 4], dtype=torch.int32, device="cuda")
    out = torch.empty(2, 3, 256, dtype=q.dtype, device="cuda") if given else None
    lse = torch.empty(2, 3, 4, device="cuda") if given else None
    for write_lse in (True, False):
        for scale in (None, 0.25):
            taken("decode", q, cache, table, lens, scale, 1, out, lse, ws, write_lse)

            def decode():
                o, l = st.sptp_paged_attn_decode(q, cache, table, lens, scale, 1, out, lse, ws, write_lse=write_lse)
                assert (l is None) == (not given and not write_lse)
                return o.clone(), None if l is None else l.clone()

            for a, b in zip(*both_ways(decode)):
                same(a, b)
    assert st.sptp_read_device_status(ws) == 0


def test_left_to_the_functions():
    """A stream of the caller's, a workspace left out, a list, numpy integers:
    calls that the functions take and the module does not."""
    qkv, pos, seq, table, turns, cache, ws = inputs("bf16")
    want = st.sptp_rope_append_kv(qkv, pos, seq, table, turns, cache, 4, workspace=ws)[:, :4].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in ({"workspace": ws, "stream": side}, {}):
        got = st.sptp_rope_append_kv(qkv, pos, seq, table, turns, list(cache), np.int64(4), **kw)
        torch.cuda.synchronize()
        same(want, got[:, :4].contiguous())


def test_the_current_stream_and_capture():
    """The module launches on the current stream, also while it is captured."""
    qkv, pos, seq, table, turns, cache, ws = inputs("bf16")
    q = torch.randn(2, 3, 4, 64, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([2, 3, 4], dtype=torch.int32, device="cuda")
    st.sptp_rope_append_kv(qkv, pos, seq, table, turns, cache, 4, workspace=ws)
    want, want_lse = (t.clone() for t in st.sptp_paged_attn_decode(q, cache, table, lens, workspace=ws))
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    for t in cache[:2]:
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        taken("append", qkv, pos, seq, table, turns, cache, 4, False, 1.0, None, ws)
        taken("decode", q, cache, table, lens, None, 0, out, lse, ws, True)
    torch.cuda.synchronize()
    assert not out.any() and not cache[0].any()  # captured, not run
    graph.replay()
    torch.cuda.synchronize()
    same(want, out)
    same(want_lse, lse)


def test_errors_are_the_same():
    qkv, pos, seq, table, turns, cache, ws = inputs("bf16")
    q, lens = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    x = qkv.view(2, 5, 8, 64)
    out = torch.empty_like(x)
    calls = [
        lambda: st.sptp_rope(x, pos.long(), turns),
        lambda: st.sptp_rope(x, pos[:4], turns),
        lambda: st.sptp_rope(x, pos, turns, out=out.float()),
        lambda: st.sptp_rope(x, pos, turns, out=out[:, :, :4]),
        lambda: st.sptp_rope(x.transpose(1, 2), torch.zeros(8, dtype=torch.int32, device="cuda"), turns),
        lambda: st.sptp_rope(x, pos.cpu(), turns),
        lambda: st.sptp_rope(x, pos, turns, Hr=9),
        lambda: st.sptp_rope(x, pos, turns, Hr=0),
        lambda: st.sptp_rope(x, pos, turns, gain=float("nan")),
        lambda: st.sptp_rope(x.half(), pos, turns),
        lambda: st.sptp_rope_append_kv(qkv, pos, seq, table, turns, cache, 5, workspace=ws),
        lambda: st.sptp_rope_append_kv(qkv, pos, seq, table, turns, cache, 4, workspace=ws[:100]),
        lambda: st.sptp_rope_append_kv(qkv, pos, seq, table, turns, cache, 4, q_out=qkv[:, :, :256].view(2, 5, 4, 64), workspace=ws),
        lambda: st.sptp_rope_append_kv(qkv.float(), pos, seq, table, turns, cache, 4, workspace=ws),
        lambda: st.sptp_paged_attn_decode(q, cache, table[:2], lens, workspace=ws),
        lambda: st.sptp_paged_attn_decode(q, cache, table, lens, float("inf"), workspace=ws),
        lambda: st.sptp_paged_attn_decode(q, cache, table, lens, window=-1, workspace=ws),
        lambda: st.sptp_paged_attn_decode(q, cache, table, lens, workspace=ws[256:]),
        lambda: st.sptp_paged_attn_decode(q, cache, table, lens, out=q.view(2, 3, 256), workspace=ws),
        lambda: st.sptp_paged_attn_decode(q, (cache[0], cache[1], lens, None), table, lens, workspace=ws),
        lambda: st.sptp_paged_attn_decode(q[:, :, :3], cache, table, lens, workspace=ws),
    ]

    def error_of(call):
        with pytest.raises(Exception) as e:
            call()
        return type(e.value), str(e.value)

    for call in calls:
        with_module, without = both_ways(lambda: error_of(call))
        assert with_module == without
