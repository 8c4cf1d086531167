"""Prompts' attention, the one-token attention's cap and slopes and the low-rank
adapters as a program that serves many requests uses them: together, on streams of
its own, in graphs, on the largest pool."""
import numpy as np
import pytest
import torch

import oracle
import sequence_tensor_transformer_gb300 as st
from oracle import attn_oracle as ao
from sequence_tensor_transformer_gb300 import synth

import batch_cases as bc
from helpers import dev_tensor, host_f64, nan_workspace, to_f64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


def adapters_of(rng, n, R, K, N, dtype="bf16"):
    A, B = (synth._cast(rng.standard_normal(s) * s[-1] ** -0.5, dtype) for s in ((n, R, K), (n, N, R)))
    gains = rng.uniform(0.3, 1.5, n).astype(np.float32)
    return (A, B, gains), (dev_tensor(A, dtype), dev_tensor(B, dtype), torch.from_numpy(gains).cuda())


def close(got, ref, size, rounded, dtype="bf16"):
    """Within `rounded` of the terms' size, and one rounding of the result."""
    tol = rounded * size + bc.HALF[dtype] * np.abs(ref) * (1 + 2.0 ** -7)
    bad = np.abs(host_f64(got) - ref) > tol
    assert not bad.any(), (np.abs(host_f64(got) - ref) / tol).max()


@pytest.mark.parametrize("variant", ["pair", "fused"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_batch_of_requests(variant, kind):
    """Two prompts in pieces, then tokens one at a time, an adapter per request on both
    projections: each stage against its oracle on the stage's own inputs, and the
    answers of a whole prompt against those of its pieces."""
    rng = np.random.default_rng(2)
    P, d, Hq, Hkv, D, R, page, chunks = 2, 256, 4, 2, 64, 16, 16, 2
    N, cap, B = P * (Hq + 2 * Hkv) * D, 12.0, 3
    slopes = torch.from_numpy((2.0 ** -np.arange(1, P * Hq + 1)).astype(np.float32).reshape(P, Hq)).cuda()
    Wqkv, Wo = (synth._cast(rng.standard_normal(s) * s[1] ** -0.5, "bf16") for s in ((N, d), (d, P * Hq * D)))
    gamma = synth._cast(1 + 0.1 * rng.standard_normal(d), "bf16")
    (A1, B1, g1), (dA1, dB1, dg1) = adapters_of(rng, 2, R, d, N)
    (A2, B2, g2), (dA2, dB2, dg2) = adapters_of(rng, 2, R, P * Hq * D, d)
    adapter = np.array([1, 0, -1])  # of the requests
    prompts = [50, 23, 9]
    cache = st.paged_kv_cache(P, 40, Hkv, page, D, e4m3=kind == "e4m3")
    table = bc.ints(rng.permutation(39)[: B * 8].reshape(B, 8))
    turns = st.sptp_rope_turns(D)
    hidden = [synth._cast(rng.standard_normal((n + 4, d)), "bf16") for n in prompts]  # rows in, of all steps
    zeros = lambda M: torch.zeros(P, M, d, dtype=BF, device="cuda")  # noqa: E731
    done = np.zeros(B, int)
    answers = [[] for _ in range(B)]

    def step(rows):
        """rows: new rows of each request."""
        M, starts = int(sum(rows)), np.concatenate([[0], np.cumsum(rows)])
        M2 = M + M % chunks  # padded
        seq = np.concatenate([np.repeat(np.arange(B), rows), np.full(M2 - M, -1)])
        pos = np.concatenate([np.arange(done[b], done[b] + rows[b]) for b in range(B)] + [np.zeros(M2 - M)]).astype(int)
        x = np.concatenate([hidden[b][done[b]: done[b] + rows[b]] for b in range(B)] + [np.zeros((M2 - M, d), hidden[0].dtype)])
        ids = np.where(seq >= 0, adapter[seq], -1)
        dx, dids = dev_tensor(x, "bf16"), bc.ints(ids)
        ws = nan_workspace(st.sptp_attn_qkv_workspace_size(M2, d, N, P, chunks))
        base, _ = st.sptp_attn_qkv_forward(dx, zeros(M2), dev_tensor(gamma, "bf16"), dev_tensor(Wqkv, "bf16"), P, chunks, 1e-6,
                                           workspace=ws, variant=variant)
        y = ws[4096: 4096 + M2 * d * 2].view(BF).view(M2, d).clone()
        qkv, _ = st.sptp_attn_qkv_forward(dx, zeros(M2), dev_tensor(gamma, "bf16"), dev_tensor(Wqkv, "bf16"), P, chunks, 1e-6,
                                          workspace=ws, variant=variant, adapters=(dA1, dB1, dids, dg1))
        ref, size = ao.lora(host_f64(y), to_f64(A1, "bf16"), to_f64(B1, "bf16"), ids, host_f64(base), g1)
        close(qkv, ref, size, (d + R + 8) * 2.0 ** -24 + 2.0 ** -16)
        q = torch.zeros(P, M2, Hq, D, dtype=BF, device="cuda")
        aws = nan_workspace(4096)
        st.sptp_rope_append_kv(qkv, bc.ints(pos), bc.ints(seq), table, turns, cache, Hq, q_out=q, workspace=aws)
        assert st.sptp_read_device_status(aws) == 0
        done[:] += rows
        lens = done.copy()
        wide = [ao.dequantised(t.cpu().numpy(), s.cpu().numpy()) if kind == "e4m3" else host_f64(t)
                for t, s in zip(cache[:2], cache[2:])]
        c = dict(P=P, M=M2, B=B, Hq=Hq, Hkv=Hkv, D=D, kind=kind, dtype="bf16", window=0, cap=cap, slopes=slopes.cpu().numpy(),
                 prefix=None, scale=D ** -0.5, q64=host_f64(q), k64=wide[0], v64=wide[1], table=table.cpu().numpy(), lens=lens,
                 starts=starts)
        if (np.asarray(rows) == 1).all():
            pws = nan_workspace(st.sptp_paged_attn_workspace_size(P, B, Hq, Hkv, D))
            attn = torch.full((P, M2, Hq * D), 7.0, dtype=BF, device="cuda")
            lse = torch.full((P, M2, Hq), 7.0, device="cuda")
            attn[:, :B], lse[:, :B] = st.sptp_paged_attn_decode(q[:, :B].contiguous(), cache, table, bc.ints(lens), workspace=pws,
                                                                cap=cap, slopes=slopes)
        else:
            pws = nan_workspace(st.sptp_paged_attn_prompt_workspace_size(P, M2, B, Hq, Hkv, D))
            attn, lse = (torch.full(s, 7.0, dtype=t, device="cuda") for s, t in (((P, M2, Hq * D), BF), ((P, M2, Hq), torch.float32)))
            st.sptp_paged_attn_prompt(q, cache, table, bc.ints(lens), bc.ints(starts), cap=cap, slopes=slopes, out=attn, lse=lse,
                                      workspace=pws)
        assert st.sptp_read_device_status(pws) == 0
        bc.check(c, attn, lse)
        parts = st.sptp_down_proj(attn, dev_tensor(Wo, "bf16"), P)
        out = st.sptp_down_proj(attn, dev_tensor(Wo, "bf16"), P, adapters=(dA2, dB2, dids, dg2))
        ref, size = ao.lora(host_f64(attn), to_f64(A2, "bf16"), to_f64(B2, "bf16"), ids, host_f64(parts), g2)
        close(out, ref, size, (P * Hq * D + R + 8) * 2.0 ** -24 + 2.0 ** -16)
        for b in range(B):
            answers[b].append(host_f64(attn)[:, starts[b]: starts[b + 1]])

    step([30, 23, 0])
    step([20, 0, 9])
    for _ in range(3):
        step([1, 1, 1])
    pieces = [np.concatenate(a, 1) for a in answers]
    # all rows at once into a fresh cache
    for t in cache:
        if t is not None:
            t.zero_()
    done[:] = 0
    answers = [[] for _ in range(B)]
    step([53, 26, 12])
    for b in range(B):
        # the same rows by other splits: bf16 q, k, v and weights, each rounded the same
        assert oracle.rel_max_error(answers[b][0], pieces[b]) <= 2e-2


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
def test_calls_on_two_streams_at_once(kind):
    cases = [bc.make(1, (60, 5), (400 + 50 * i, 90), 4, 2, 64, 16, kind, seed=i, cap=10.0) for i in range(2)]
    want = [bc.call(c)[:2] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    prepared = [(bc.arguments(c), bc.workspace(c)) for c in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, ((args, kw), ws) in zip(streams, prepared):
            got.append(st.sptp_paged_attn_prompt(*args, **kw, workspace=ws, stream=s))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        n = cases[i % 2]["starts"][-1]
        assert torch.equal(o[:, :n], want[i % 2][0][:, :n]) and torch.equal(l[:, :n], want[i % 2][1][:, :n])


def test_calls_under_a_stream_of_the_callers():
    c = bc.make(1, (60, 5), (400, 90), 4, 2, 64, 16, "bf16")
    out, lse, _ = bc.call(c)
    with torch.cuda.stream(torch.cuda.Stream()):
        args, kw = bc.arguments(c)
        got = st.sptp_paged_attn_prompt(*args, **kw)
        torch.cuda.current_stream().synchronize()
        assert torch.equal(got[0], out)
        x, A, B = torch.randn(20, 64, device="cuda"), torch.randn(2, 8, 64, device="cuda"), torch.randn(2, 32, 8, device="cuda")
        base, ids = torch.randn(1, 20, 32, device="cuda"), torch.arange(20, device="cuda", dtype=torch.int32) % 3 - 1
        y = st.sptp_lora(x, A, B, ids, base)
        torch.cuda.current_stream().synchronize()
    assert torch.equal(y, st.sptp_lora(x, A, B, ids, base, stream=torch.cuda.current_stream()))


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
def test_two_graphs_on_one_workspace(kind):
    """Captured calls replayed on other lengths, rows, prefixes and values, one graph after
    the other on one workspace."""
    a, b = (bc.make(2, (40, 0, 9), (300, 20, 77), 4, 2, 64, 16, kind, seed=s, prefix=(10, 20, 0), cap=9.0, pad=20, holes=False)
            for s in (1, 2))
    ws = nan_workspace(bc.workspace(a).numel())
    graphs = []
    for c in (a, b):
        args, kw = bc.arguments(c)
        out = torch.full((c["P"], c["M"], c["Hq"] * c["D"]), 7.0, dtype=bc.TD[c["dtype"]], device="cuda")
        lse = torch.full((c["P"], c["M"], c["Hq"]), 7.0, device="cuda")
        st.sptp_paged_attn_prompt(*args, **kw, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st.sptp_paged_attn_prompt(*args, **kw, out=out, lse=lse, workspace=ws)
        graphs.append((g, c, args, kw, out, lse))
    for rows, lens, prefix in (((40, 0, 9), (300, 20, 77), (10, 20, 0)), ((20, 8, 30), (260, 19, 30), (0, 0, 30)), ((1, 1, 1), (1, 2, 70), (1, 1, 1))):
        for g, c, args, kw, out, lse in graphs:
            starts = np.concatenate([[0], np.cumsum(rows)])
            for t, v in ((args[3], lens), (args[4], starts), (kw["prefix_lens"], prefix)):
                t.copy_(bc.ints(v))
            out.fill_(7.0)
            lse.fill_(7.0)
            g.replay()
            assert st.sptp_read_device_status(ws) == 0
            bc.check(dict(c, rows=np.array(rows), lens=np.array(lens), starts=starts, prefix=prefix), out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M", [40, 400])
def test_adapters_in_a_graph(M, dtype):
    rng = np.random.default_rng(3)
    (A, B, g), (dA, dB, dg) = adapters_of(rng, 4, 16, 128, 96, dtype)
    x, base = (synth._cast(rng.standard_normal(s), dtype) for s in ((M, 128), (2, M, 48)))
    dx, db, ids = dev_tensor(x, dtype), dev_tensor(base, dtype), bc.ints(np.arange(M) % 4)
    ws, out = nan_workspace(st.sptp_lora_workspace_size(2, M, 128, 96, 16)), torch.empty(2, M, 48, dtype=bc.TD[dtype], device="cuda")
    st.sptp_lora(dx, dA, dB, ids, db, dg, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.sptp_lora(dx, dA, dB, ids, db, dg, out=out, workspace=ws)
    for shift in range(4):
        now = np.where(np.arange(M) % 7 == 0, -1, (np.arange(M) // 3 + shift) % 4)
        if shift == 2:
            now[5] = 4
        ids.copy_(bc.ints(now))
        graph.replay()
        assert st.sptp_read_device_status(ws) == (st.STATUS["shape"] if shift == 2 else 0)
        now[now == 4] = -1
        ref, size = ao.lora(to_f64(x, dtype), to_f64(A, dtype), to_f64(B, dtype), now, to_f64(base, dtype), g)
        close(out, ref, size, (128 + 16 + 8) * 2.0 ** -24 + (2.0 ** -16 if dtype == "bf16" else 0), dtype)


def test_strided_tensors_are_refused():
    c = bc.make(1, (17, 3), (40, 5), 4, 2, 64, 16, "bf16")
    args, kw = bc.arguments(c)
    wide = torch.zeros(1, 20, 8, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        st.sptp_paged_attn_prompt(wide[:, :, :4], *args[1:], **kw)
    with pytest.raises(ValueError, match="contiguous"):
        st.sptp_paged_attn_prompt(*args[:3], torch.zeros(4, dtype=torch.int32, device="cuda")[::2], args[4], **kw)
    x = torch.zeros(20, 128, dtype=BF, device="cuda")
    A, B = torch.zeros(2, 8, 64, dtype=BF, device="cuda"), torch.zeros(2, 32, 8, dtype=BF, device="cuda")
    ids, base = torch.zeros(20, dtype=torch.int32, device="cuda"), torch.zeros(1, 20, 32, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        st.sptp_lora(x[:, :64], A, B, ids, base)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
def test_pages_beyond_four_gigabytes(kind):
    """The same sequence at the end of a pool of more than 2^32 bytes."""
    c = bc.make(1, (70,), (300,), 4, 1, 128, 128, kind, cap=20.0)
    out, lse, _ = bc.call(c)
    es = {"bf16": 2, "fp32": 4, "e4m3": 1}[kind]
    pages = (1 << 32) // (128 * 128 * es) + 64
    n = c["cache"][0].shape[1]
    big = []
    for t in c["cache"]:
        if t is None:
            big.append(None)
            continue
        b = torch.empty(1, pages, *t.shape[2:], dtype=t.dtype, device="cuda")
        b[:, pages - n:] = t
        big.append(b)
    got, gl, _ = bc.call(dict(c, cache=tuple(big), table=c["table"] + pages - n))
    assert torch.equal(got, out) and torch.equal(gl, lse)


def test_shared_pages():
    """A prefix that two sequences share, and one page twice in a sequence."""
    c = bc.make(2, (30, 20), (200, 200), 4, 2, 64, 16, "bf16")
    t = c["table"]
    t[1, :8] = t[0, :8]
    t[0, 9] = t[0, 2]
    out, lse, ws = bc.call(c)
    assert st.sptp_read_device_status(ws) == 0
    bc.check(c, out, lse)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
def test_another_sequences_nan_stays_there(kind):
    c = bc.make(1, (30, 20), (100, 90), 4, 2, 64, 16, kind)
    want, wl, _ = bc.call(c)
    for t in c["cache"][:2]:
        t[:, torch.from_numpy(c["table"][1]).cuda()] = 0xFF if kind == "e4m3" else float("nan")
    got, gl, _ = bc.call(c)
    assert torch.equal(got[:, :30], want[:, :30]) and torch.equal(gl[:, :30], wl[:, :30])


# ---------------------------------------------------------------- the extension module

def ways(name, call):
    """The results of a call through the extension module, which has to take it, and without it."""
    fast, results = st._fast, []
    took = []

    class Watch:
        def __getattr__(self, n):
            def made(*args):
                done = getattr(fast, n)(*args)
                took.append((n, done is not NotImplemented))
                return done
            return made

    for module in (Watch(), None):
        st._fast = module
        try:
            results.append([None if t is None else t.clone() for t in call()])
        finally:
            st._fast = fast
    torch.cuda.synchronize()
    assert took == [(name, True)]
    for a, b in zip(*results):
        assert (a is None) == (b is None)
        assert a is None or (a.shape == b.shape and a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8)))


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("given", [False, True])
def test_the_extension_module_makes_the_same_calls(kind, given):
    assert st._fast is not None
    g = torch.Generator(device="cuda").manual_seed(3)
    P, B, Hq, Hkv, D, page = 2, 3, 4, 2, 64, 16
    dt = torch.float32 if kind == "fp32" else torch.bfloat16
    cache = st.paged_kv_cache(P, 12, Hkv, page, D, dt, kind == "e4m3")
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(dt)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for t in cache[:2]:
        t.copy_(torch.randint(0, 100, t.shape, generator=g, device="cuda") if kind == "e4m3" else randn(*t.shape))
    for t in cache[2:]:
        if t is not None:
            t.fill_(0.125)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(B, 4)
    lens, starts, prefixes = ints(40, 5, 64), ints(0, 7, 9, 10), ints(0, 5, 12)
    slopes = torch.rand(P, Hq, generator=g, device="cuda")
    q1, q = randn(P, B, Hq, D), randn(P, 10, Hq, D)
    ws = torch.empty(max(st.sptp_paged_attn_workspace_size(P, B, Hq, Hkv, D),
                         st.sptp_paged_attn_prompt_workspace_size(P, 10, B, Hq, Hkv, D)), dtype=torch.uint8, device="cuda")
    new = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device="cuda") if given else None
    out1, lse1 = new(P, B, Hq * D), new(P, B, Hq, dtype=torch.float32)
    out, lse = new(P, 10, Hq * D), new(P, 10, Hq, dtype=torch.float32)
    for cap, bias, prefix in ((0.0, None, None), (20.0, None, prefixes), (0, slopes, prefixes), (20.0, slopes, None)):
        for write in (True, False):
            how = dict(scale=None if given else 0.2, window=0 if prefix is None else 17, cap=cap, slopes=bias, workspace=ws, write_lse=write)
            ways("decode" if not cap and bias is None else "decode_ex",
                 lambda: st.sptp_paged_attn_decode(q1, cache, table, lens, out=out1, lse=lse1, **how))
            ways("prompt", lambda: st.sptp_paged_attn_prompt(q, cache, table, lens, starts, prefix_lens=prefix, out=out, lse=lse, **how))
            assert st.sptp_read_device_status(ws) == 0
    if kind == "e4m3":
        return
    a, b, ids, gains = randn(3, 8, 64), randn(3, 32, 8), ints(0, 2, -1, 1, 1, 2, 0, 0, 1, 2), torch.rand(3, generator=g, device="cuda")
    for x, base in ((randn(10, 64), randn(P, 10, 16)), (randn(P, 10, 32), randn(P, 10, 32))):
        lws = torch.empty(st.sptp_lora_workspace_size(P, 10, 64, 32, 8, x.dim() == 3), dtype=torch.uint8, device="cuda")
        for gain in (None, gains):
            ways("lora", lambda: [st.sptp_lora(x, a, b, ids, base, gain, torch.empty_like(base) if given else None, lws)])


def test_the_extension_module_leaves_what_is_wrong():
    P, M, Hq, D = 1, 4, 2, 64
    cache = st.paged_kv_cache(P, 2, 1, 16, D, torch.bfloat16)
    q = torch.zeros(P, M, Hq, D, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.full((1,), 4, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    ws = torch.empty(st.sptp_paged_attn_prompt_workspace_size(P, M, 1, Hq, 1, D), dtype=torch.uint8, device="cuda")
    prompt = lambda *a, **kw: st.sptp_paged_attn_prompt(*a, **{"workspace": ws, **kw})
    x, base = torch.zeros(M, 64, device="cuda"), torch.zeros(1, M, 16, device="cuda")
    a, b, ids = torch.zeros(1, 8, 64, device="cuda"), torch.zeros(1, 16, 8, device="cuda"), torch.zeros(M, dtype=torch.int32, device="cuda")
    lws = torch.empty(st.sptp_lora_workspace_size(1, M, 64, 16, 8), dtype=torch.uint8, device="cuda")
    calls = [
        lambda: prompt(q, cache, table, lens, starts[:1]),
        lambda: prompt(q, cache, table, lens.long(), starts),
        lambda: prompt(q, cache, table, lens, starts, cap=-1.0),
        lambda: prompt(q, cache, table, lens, starts, cap=float("nan")),
        lambda: prompt(q, cache, table, lens, starts, window=-1),
        lambda: prompt(q, cache, table, lens, starts, slopes=torch.zeros(2, 1, device="cuda")),
        lambda: prompt(q, cache, table, lens, starts, prefix_lens=lens.cpu()),
        lambda: prompt(q, cache, table, lens, starts, out=q.view(P, M, Hq * D)),
        lambda: prompt(q, cache, table, lens, starts, workspace=ws[:4096]),
        lambda: prompt(q.transpose(1, 2), cache, table, lens, starts),
        lambda: st.sptp_paged_attn_decode(q[:, :1].contiguous(), cache, table, lens, cap=-1.0, workspace=ws),
        lambda: st.sptp_lora(x, a, b.bfloat16(), ids, base, workspace=lws),
        lambda: st.sptp_lora(x, a, b, ids.long(), base, workspace=lws),
        lambda: st.sptp_lora(x, a, b, ids, base, workspace=lws[:100]),
        lambda: st.sptp_lora(x[:, :32], a, b, ids, base, workspace=lws),
        lambda: st.sptp_lora(x, a, b, ids, base, out=base[:, :, :8], workspace=lws),
    ]
    for call in calls:
        errors = []
        fast = st._fast
        for module in (fast, None):
            st._fast = module
            try:
                with pytest.raises(Exception) as e:
                    call()
                errors.append((type(e.value), str(e.value)))
            finally:
                st._fast = fast
        assert errors[0] == errors[1]
