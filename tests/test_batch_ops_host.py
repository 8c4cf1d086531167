"""CPU tests of prompts' attention, the one-token attention's cap and slopes, and the
low-rank adapters: every refusal of the C ABI and of the binding, and the workspace
sizes (nothing here reaches a GPU)."""
import ctypes

import pytest
import torch

import sequence_tensor_transformer_gb300 as st

OK, NULL, SHAPE, DTYPE, WS, ALIAS = 0, -1, -2, -3, -4, -8
BF = torch.bfloat16
A = 1 << 40  # addresses that are never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os
    if not os.path.exists(st.LIB_PATH):
        from sequence_tensor_transformer_gb300 import build
        build.build()
    st.load_library()


# ---------------------------------------------------------------- prompts' attention

def prompt(raw=None, selftest=None, **kw):
    """The call's status for a right call (with M = 0, so that nothing is launched, unless
    something is wrong with it) changed by kw."""
    a = dict(q=A, k=2 * A, v=3 * A, ks=0, vs=0, table=4 * A, lens=5 * A, starts=6 * A, prefix=0, slopes=0, out=7 * A, lse=8 * A,
             ws=9 * A, stream=0, ws_bytes=1 << 40, P=2, M=0, B=3, Hq=8, Hkv=2, D=128, max_pages=4, num_pages=16, page=16, window=0,
             dtype=0, kv=0, scale=0.1, cap=0.0)
    a.update(kw)
    block = st._PROMPT_ARGS.pack(*a.values())
    if selftest:
        return st.lib().sptp_paged_attn_prompt_wait_selftest(block, *selftest)
    return st.lib().sptp_paged_attn_prompt(block if raw is None else raw)


def test_prompt_accepts_calls_without_rows():
    assert prompt() == OK and prompt(q=0, out=0, table=0, lens=0, starts=0) == OK
    assert prompt(M=5, B=0, q=0, out=0, table=0, lens=0, starts=0) == OK
    assert prompt(dtype=1) == OK and prompt(kv=1, ks=10 * A, vs=11 * A) == OK
    assert prompt(cap=1e30, slopes=12 * A, prefix=13 * A, window=2 ** 31 - 1, scale=-1.0, lse=0) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(ws=0), NULL), (dict(kv=1), NULL), (dict(kv=1, ks=10 * A), NULL),
    (dict(M=1, q=0), NULL), (dict(M=1, table=0), NULL), (dict(M=1, lens=0), NULL), (dict(M=1, starts=0), NULL),
    (dict(M=1, out=0), NULL),
    (dict(dtype=2), DTYPE), (dict(kv=2), DTYPE), (dict(kv=1, dtype=1, ks=10 * A, vs=11 * A), DTYPE),
    (dict(P=0), SHAPE), (dict(P=9), SHAPE), (dict(M=-1), SHAPE), (dict(B=-1), SHAPE), (dict(M=1 << 30), SHAPE),
    (dict(B=1 << 30), SHAPE), (dict(Hq=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hkv=3), SHAPE), (dict(D=4), SHAPE),
    (dict(D=12), SHAPE), (dict(D=264), SHAPE), (dict(kv=1, ks=10 * A, vs=11 * A, D=24), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(num_pages=0), SHAPE), (dict(page=8), SHAPE), (dict(page=24), SHAPE), (dict(max_pages=1 << 26), SHAPE),
    (dict(num_pages=1 << 26, page=32), SHAPE), (dict(window=-1), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(cap=-1.0), SHAPE), (dict(cap=float("nan")), SHAPE), (dict(cap=float("inf")), SHAPE),
    (dict(cap=1e-31), SHAPE), (dict(cap=2e30), SHAPE), (dict(q=A + 8), SHAPE), (dict(lens=A + 2), SHAPE),
    (dict(starts=A + 1), SHAPE), (dict(prefix=A + 2), SHAPE), (dict(slopes=A + 2), SHAPE), (dict(ws=9 * A + 128), SHAPE),
    (dict(out=7 * A + 4), SHAPE), (dict(lse=8 * A + 4), SHAPE), (dict(ws_bytes=4096), WS),
    (dict(M=4, out=A), ALIAS), (dict(M=4, out=2 * A + 16), ALIAS), (dict(M=4, lse=7 * A), ALIAS), (dict(M=4, lse=6 * A), ALIAS),
    (dict(M=4, ws=3 * A), ALIAS), (dict(M=4, ws=12 * A, slopes=12 * A), ALIAS)])
def test_prompt_refusals(kw, code):
    assert prompt(**kw) == code


def test_prompt_takes_a_block():
    assert st.lib().sptp_paged_attn_prompt(None) == NULL
    assert st.lib().sptp_paged_attn_prompt_wait_selftest(None, 0, 1) == NULL


@pytest.mark.parametrize("kw,args,code", [
    ({}, (-1, 1000), SHAPE), ({}, (0, 0), SHAPE), ({}, (0, 10 ** 11), SHAPE), (dict(dtype=1), (0, 1000), DTYPE),
    (dict(D=64), (0, 1000), SHAPE), (dict(D=136), (0, 1000), SHAPE), (dict(cap=1.0), (0, 1000), SHAPE),
    (dict(slopes=12 * A), (0, 1000), SHAPE), (dict(scale=0.0), (0, 1000), SHAPE), ({}, (0, 1000), OK)])
def test_prompt_selftest_refusals(kw, args, code):
    assert prompt(selftest=args, **kw) == code


def test_prompt_workspace():
    size = st.sptp_paged_attn_prompt_workspace_size
    assert size(2, 0, 3, 8, 2, 128) >= st.SPTP_WS_HEADER_BYTES and size(9, 1, 1, 8, 2, 128) == 0 and size(1, -1, 1, 8, 2, 128) == 0
    assert size(1, 1, 1, 8, 3, 128) == 0 and size(1, 1 << 30, 1, 8, 2, 128) == 0
    # parts of up to 256 rows for 160 CTAs, or of 64 for 320
    assert size(1, 10 ** 6, 1, 8, 2, 128) >= 160 * 2 * 256 * (128 + 2) * 4
    assert size(1, 1, 1, 2, 2, 128) >= 320 * 2 * 1 * (128 + 2) * 4
    assert size(1, 10 ** 6, 64, 8, 2, 256) >= 160 * 2 * 128 * (256 + 2) * 4
    # needs no more for more rows than an item can have
    assert size(1, 10 ** 6, 1, 8, 2, 128) == size(4, 300, 64, 8, 2, 128)


def cpu_call(**kw):
    P, M, Hq, D, B = 2, 6, 4, 64, 2
    cache = (torch.zeros(P, 4, 2, 16, D, dtype=BF), torch.zeros(P, 4, 2, 16, D, dtype=BF), None, None)
    a = dict(q=torch.zeros(P, M, Hq, D, dtype=BF), cache=cache, page_table=torch.zeros(B, 2, dtype=torch.int32),
             seq_lens=torch.zeros(B, dtype=torch.int32), row_starts=torch.zeros(B + 1, dtype=torch.int32))
    a.update(kw)
    return st.sptp_paged_attn_prompt(**a)


@pytest.mark.parametrize("kw,error,text", [
    ({}, ValueError, "device tensors only"),
    (dict(row_starts=torch.zeros(2, dtype=torch.int32)), ValueError, "row_starts"),
    (dict(row_starts=torch.zeros(3)), TypeError, "row_starts"),
    (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), ValueError, "seq_lens"),
    (dict(prefix_lens=torch.zeros(3, dtype=torch.int32)), ValueError, "prefix_lens"),
    (dict(prefix_lens=torch.zeros(2, dtype=torch.int64)), TypeError, "prefix_lens"),
    (dict(slopes=torch.zeros(4)), ValueError, "slopes"),
    (dict(slopes=torch.zeros(2, 4, dtype=BF)), TypeError, "slopes"),
    (dict(out=torch.zeros(2, 6, 4, 64, dtype=BF)), ValueError, "out"),
    (dict(lse=torch.zeros(2, 6, 4, dtype=BF)), TypeError, "lse"),
    (dict(q=torch.zeros(2, 6, 4, 64, dtype=torch.float16)), TypeError, "dtype")])
def test_prompt_binding_names_what_is_wrong(kw, error, text):
    with pytest.raises(error, match=text):
        cpu_call(**kw)


# ---------------------------------------------------------------- one token, with a cap and slopes

def decode(cap=0.0, slopes=0, **kw):
    a = dict(q=A, k=2 * A, v=3 * A, ks=0, vs=0, table=4 * A, lens=5 * A, out=7 * A, lse=8 * A, ws=9 * A, stream=0,
             ws_bytes=1 << 40, P=2, B=0, Hq=8, Hkv=2, D=128, max_pages=4, num_pages=16, page=16, window=0, dtype=0, kv=0, scale=0.1)
    a.update(kw)
    return st.lib().sptp_paged_attn_decode_ex(st._DECODE_ARGS.pack(*a.values()), ctypes.c_float(cap), slopes or None)


def test_decode_ex_refusals():
    assert decode() == OK and decode(50.0, 12 * A) == OK and decode(0.0, 12 * A) == OK
    for cap in (-1.0, float("nan"), float("inf"), 1e-31, 2e30):
        assert decode(cap) == SHAPE
    assert decode(1.0, 12 * A + 2) == SHAPE and decode(1.0, 7 * A, B=1) == ALIAS and decode(1.0, 9 * A + 8, B=1) == ALIAS
    assert st.lib().sptp_paged_attn_decode_ex(None, ctypes.c_float(0), None) == NULL


def test_decode_binding_names_slopes():
    P, B, Hq, D = 2, 3, 4, 64
    cache = (torch.zeros(P, 4, 2, 16, D, dtype=BF), torch.zeros(P, 4, 2, 16, D, dtype=BF), None, None)
    args = (torch.zeros(P, B, Hq, D, dtype=BF), cache, torch.zeros(B, 2, dtype=torch.int32), torch.zeros(B, dtype=torch.int32))
    with pytest.raises(ValueError, match="slopes"):
        st.sptp_paged_attn_decode(*args, slopes=torch.zeros(4))
    with pytest.raises(TypeError, match="slopes"):
        st.sptp_paged_attn_decode(*args, cap=3.0, slopes=torch.zeros(2, 4, dtype=BF))


# ---------------------------------------------------------------- low-rank adapters

def lora(**kw):
    a = dict(x=A, A=2 * A, B=3 * A, ids=4 * A, gains=5 * A, P=2, M=0, K=64, N=96, R=16, n=3, rowwise=0, dtype=0, base=6 * A,
             out=7 * A, ws=8 * A, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return st.lib().sptp_lora(*a.values())


def test_lora_accepts_calls_without_rows():
    assert lora() == OK and lora(gains=None, x=None, ids=None, base=None, out=None, A=None, B=None) == OK
    assert lora(rowwise=1) == OK and lora(dtype=1) == OK and lora(out=6 * A) == OK and lora(n=0, A=None, B=None) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(ws=None), NULL), (dict(M=1, x=None), NULL), (dict(M=1, A=None), NULL), (dict(M=1, B=None), NULL),
    (dict(M=1, ids=None), NULL), (dict(M=1, base=None), NULL), (dict(M=1, out=None), NULL), (dict(dtype=2), DTYPE),
    (dict(P=0), SHAPE), (dict(P=9), SHAPE), (dict(M=-1), SHAPE), (dict(R=0), SHAPE), (dict(R=12), SHAPE), (dict(R=136), SHAPE),
    (dict(K=60), SHAPE), (dict(N=104), SHAPE), (dict(K=72, rowwise=1), SHAPE), (dict(N=100, rowwise=1), SHAPE), (dict(K=0), SHAPE),
    (dict(n=-1), SHAPE), (dict(n=1 << 24), SHAPE), (dict(K=(1 << 20) + 8), SHAPE), (dict(M=1 << 30), SHAPE),
    (dict(M=1 << 29, N=1 << 20, P=8), SHAPE), (dict(x=A + 8), SHAPE), (dict(ids=A + 2), SHAPE), (dict(gains=A + 2), SHAPE),
    (dict(ws=8 * A + 128), SHAPE), (dict(out=7 * A + 8), SHAPE), (dict(ws_bytes=0), WS), (dict(M=1, out=A), ALIAS),
    (dict(M=1, out=2 * A), ALIAS), (dict(M=4, out=6 * A + 16), ALIAS), (dict(M=1, ws=3 * A), ALIAS), (dict(M=1, out=8 * A), ALIAS)])
def test_lora_refusals(kw, code):
    assert lora(**kw) == code


def test_lora_workspace():
    size = st.sptp_lora_workspace_size
    assert size(2, 0, 64, 96, 16) >= st.SPTP_WS_HEADER_BYTES and size(9, 1, 64, 96, 16) == 0 and size(2, 1, 64, 100, 16) == 0
    for M, K, R, P, rowwise in ((1, 64, 8, 1, 0), (64, 3584, 16, 4, 0), (5000, 4096, 128, 2, 1), (100, 1000, 24, 1, 0)):
        assert size(P, M, K, 64 * P, R, rowwise) >= st.SPTP_WS_HEADER_BYTES + M * R * 4 * (P if rowwise else 1)


@pytest.mark.parametrize("kw,error,text", [
    ({}, ValueError, "device tensors only"),
    (dict(x=torch.zeros(5, 56, dtype=BF)), ValueError, "x"),
    (dict(x=torch.zeros(5, 64)), TypeError, "A"),
    (dict(ids=torch.zeros(5, dtype=torch.int64)), TypeError, "ids"),
    (dict(ids=torch.zeros(4, dtype=torch.int32)), ValueError, "ids"),
    (dict(gains=torch.zeros(2)), ValueError, "gains"),
    (dict(gains=torch.zeros(3, dtype=BF)), TypeError, "gains"),
    (dict(base=torch.zeros(5, 5, 96 // 5, dtype=BF)), ValueError, "multiple"),
    (dict(base=torch.zeros(2, 5, 96, dtype=BF)), ValueError, "base"),
    (dict(B=torch.zeros(3, 96, 8, dtype=BF)), ValueError, "B"),
    (dict(out=torch.zeros(2, 5, 48)), TypeError, "out")])
def test_lora_binding_names_what_is_wrong(kw, error, text):
    a = dict(x=torch.zeros(5, 64, dtype=BF), A=torch.zeros(3, 16, 64, dtype=BF), B=torch.zeros(3, 96, 16, dtype=BF),
             ids=torch.zeros(5, dtype=torch.int32), base=torch.zeros(2, 5, 48, dtype=BF))
    a.update(kw)
    with pytest.raises(error, match=text):
        st.sptp_lora(**a)


# ---------------------------------------------------------------- the extension module

def test_the_extension_module_leaves_the_calls():
    """Tensors on the host, wrong numbers of arguments, and addresses that are none."""
    fast = st._fast
    assert fast is not None
    P, B, Hq, D = 2, 3, 4, 64
    cache = (torch.zeros(P, 4, 2, 16, D, dtype=BF), torch.zeros(P, 4, 2, 16, D, dtype=BF), None, None)
    q, ws = torch.zeros(P, B, Hq, D, dtype=BF), torch.zeros(4096, dtype=torch.uint8)
    table, lens, starts = torch.zeros(B, 2, dtype=torch.int32), torch.zeros(B, dtype=torch.int32), torch.zeros(B + 1, dtype=torch.int32)
    x, base = torch.zeros(5, 32), torch.zeros(2, 5, 8)
    a, b, ids = torch.zeros(3, 8, 32), torch.zeros(3, 16, 8), torch.zeros(5, dtype=torch.int32)
    assert fast.decode_ex(q, cache, table, lens, None, 0, None, None, ws, True, 1.0, None) is NotImplemented
    assert fast.prompt(q, cache, table, lens, starts, None, 0, 0.0, None, None, None, None, ws, True) is NotImplemented
    assert fast.lora(x, a, b, ids, base, None, None, ws) is NotImplemented
    for call in (fast.decode_ex, fast.prompt, fast.lora):
        for n in (0, 1, 8, 12, 14, 15):
            assert call(*[None] * n) is NotImplemented
    for addresses in ((), (1, 2), (0, 1, 2), ("a", 1, 2)):
        with pytest.raises((TypeError, ValueError)):
            fast.use_batch(*addresses)
    st.set_library(st.lib())
