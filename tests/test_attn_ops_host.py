"""CPU tests of the rotary-position, paged-cache and one-token-attention entry
points: the frequency table against exact arithmetic, the oracle's pins, and
every refusal of the C ABI and of the binding (nothing here reaches a GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st
from oracle import attn_oracle as ao

OK, NULL, SHAPE, DTYPE, WS, UNIMPL, ALIAS = 0, -1, -2, -3, -4, -7, -8
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os
    if not os.path.exists(st.LIB_PATH):
        from sequence_tensor_transformer_gb300 import build
        build.build()
    st.load_library()


# ---------------------------------------------------------------- frequency table

@pytest.mark.parametrize("rot,theta,scaling,factor,orig,alpha,beta", [
    (16, 10000.0, "none", 1.0, 0, 1, 32), (128, 1e6, "none", 7.0, 0, 1, 32), (256, 10000.0, "linear", 8.0, 0, 1, 32),
    (64, 500000.0, "ntk", 4.0, 0, 1, 32), (128, 10000.0, "parts", 32.0, 4096, 1, 32),
    (128, 500000.0, "parts", 8.0, 8192, 1, 4), (48, 10000.0, "parts", 1.0, 100, -1, 0.5)])
def test_turns_against_many_digits(rot, theta, scaling, factor, orig, alpha, beta):
    mp = pytest.importorskip("mpmath")
    got = st.sptp_rope_turns(rot, theta, scaling, factor, orig, alpha, beta, device="cpu").tolist()
    assert len(got) == rot // 2
    with mp.workdps(60):
        th = mp.mpf(theta) * (mp.mpf(factor) ** (mp.mpf(rot) / (rot - 2)) if scaling == "ntk" else 1)
        for i in range(rot // 2):
            f = th ** (mp.mpf(-2 * i) / rot)
            if scaling == "linear":
                f /= factor
            if scaling == "parts":
                c = min(mp.mpf(1), max(mp.mpf(0), (orig * f / (2 * mp.pi) - alpha) / (mp.mpf(beta) - alpha)))
                f = c * f + (1 - c) * f / factor
            want = f / (2 * mp.pi) * 2 ** 64
            # double arithmetic: pow (1 ulp of a double, and of its rounded
            # exponent: |2i/rot ln theta| <= 14 half-ulps), a few products
            assert abs(got[i] - want) <= want * 2.0 ** -53 * 32 + 1, i
            assert 0 <= got[i] < 1 << 62


def test_turns_agree_with_the_oracle_frequencies():
    for kw in (dict(), dict(scaling="linear", factor=3.0), dict(scaling="ntk", factor=3.0),
               dict(scaling="parts", factor=16.0, orig_len=2048)):
        u = st.sptp_rope_turns(96, 10000.0, device="cpu", **kw).numpy().astype(np.float64)
        # the table's grid of 2^-64 of a turn: off by half a step, and by double arithmetic
        np.testing.assert_allclose(u / 2.0 ** 64 * 2 * math.pi, ao.rope_frequencies(96, 10000.0, **kw), rtol=1e-14,
                                   atol=2 * math.pi * 2.0 ** -65)


def test_turns_refusals():
    lib = st.lib()
    buf = (ctypes.c_ulonglong * 128)()
    call = lambda rot=64, theta=1e4, sc=0, f=1.0, o=4096.0, a=1.0, b=32.0, t=buf: lib.sptp_rope_turns(
        rot, theta, sc, f, o, a, b, t)
    assert call() == OK
    assert call(t=None) == NULL
    for rot in (0, 8, 24, 272, -16):
        assert call(rot=rot) == SHAPE
    for theta in (1.0, 0.5, -3.0, math.nan, math.inf):
        assert call(theta=theta) == SHAPE
    assert call(sc=4) == UNIMPL and call(sc=-1) == UNIMPL
    assert call(f=0.0) == OK  # ignored without scaling
    for f in (0.5, 0.0, math.nan, math.inf):
        assert call(sc=1, f=f) == SHAPE
    assert call(sc=2, theta=1e300, f=1e300) == SHAPE
    assert call(sc=3, o=0.0) == SHAPE and call(sc=3, a=32.0) == SHAPE and call(sc=3, b=math.nan) == SHAPE
    assert call(sc=1, o=0.0) == OK
    with pytest.raises(ValueError, match="scaling"):
        st.sptp_rope_turns(64, scaling="other", device="cpu")
    with pytest.raises(st.SptpError) as e:
        st.sptp_rope_turns(20, device="cpu")
    assert e.value.code == SHAPE


# ---------------------------------------------------------------- oracle pins

def test_oracle_rotation_closed_forms():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 5, 3, 32))
    f = ao.rope_frequencies(16, 100.0)
    pos = np.array([0, 1, 7, 100, 3])
    for inter in (False, True):
        a = np.outer(pos, f)
        y = ao.rope(x, a, 2, inter)
        assert np.array_equal(y[:, 0], x[:, 0]) and np.array_equal(y[:, :, 2], x[:, :, 2])
        assert np.array_equal(y[..., 16:], x[..., 16:])
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
        np.testing.assert_allclose(ao.rope(y, a, 2, inter, transpose=True), x, atol=1e-12)
        np.testing.assert_allclose(ao.rope(y, a, 2, inter), ao.rope(x, 2 * a, 2, inter), atol=1e-12)
        # a key's product with a query depends on the difference of positions alone
        q, k = ao.rope(x, a + 5 * f, 3, inter), ao.rope(x, a, 3, inter)
        q0 = ao.rope(x, np.tile(5 * f, (5, 1)), 3, inter)
        np.testing.assert_allclose((q * k).sum(-1), (q0 * x).sum(-1), atol=1e-11)
    e = np.zeros((1, 1, 1, 16))
    e[..., 0] = 1.0
    y = ao.rope(e, np.full((1, 8), math.pi / 2), 1)
    assert abs(y[0, 0, 0, 8] - 1) < 1e-15  # half layout: element 0 turns into element 8
    y = ao.rope(e, np.full((1, 8), math.pi / 2), 1, interleaved=True)
    assert abs(y[0, 0, 0, 1] - 1) < 1e-15
    u = [1 << 63, 1 << 62, 3]
    assert np.allclose(ao.angles_from_turns([1, 2, -1], u) / math.pi, [[-1, 0.5, 0], [0, -1, 0], [-1, -0.5, 0]])


def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 1, 6, 2, 16, 8))
    table = np.array([[4, 0, 2], [1, 5, 3]])
    q = np.zeros((1, 2, 4, 8))
    out, lse, mean, _ = ao.paged_attn_decode(q, k, v, table, [0, 37], 1.0)
    assert not out[:, 0].any() and np.all(lse[:, 0] == -np.inf)
    rows = np.concatenate([v[0, 1, 0], v[0, 5, 0], v[0, 3, 0, :5]])
    np.testing.assert_allclose(out[0, 1, 0], rows.mean(0), rtol=1e-12)  # equal scores: the mean
    np.testing.assert_allclose(lse[0, 1], math.log(37))
    q[0, 1, 2] = 100 * k[0, 5, 1, 3]  # one key's direction: its value alone
    k[0, 5, 1, 3] *= 20
    out, _, _, _ = ao.paged_attn_decode(q, k, v, table, [0, 37], 1.0)
    np.testing.assert_allclose(out[0, 1, 2], v[0, 5, 1, 3], rtol=1e-9)
    # the window: the last keys alone
    o, l, _, _ = ao.paged_attn_decode(q * 0, k, v, table, [0, 37], 1.0, window=5)
    np.testing.assert_allclose(o[0, 1, 0], v[0, 3, 0, :5].mean(0), rtol=1e-12)


def test_oracle_dequantisation_matches_the_quantiser():
    rng = np.random.default_rng(2)
    from oracle import fp8_oracle as f8
    a = f8.round_bf16(rng.standard_normal((7, 32)) * np.exp(rng.uniform(-9, 9, (7, 1))))
    a[3] = 0
    codes, scale = ao.quantise_rows(a)
    q, e = f8.quantize_rows_e4m3(a)
    assert np.array_equal(ao.dequantised(codes, scale), q * np.ldexp(1.0, e)[:, None])


# ---------------------------------------------------------------- C ABI refusals

A = 1 << 32  # an aligned address that nothing dereferences; buffers lie 64 GiB apart
at = lambda i: A * 16 * (i + 1)


def rope(**k):
    a = dict(x=at(0), pos=at(1), turns=at(2), P=2, M=8, H=6, Hr=4, D=64, rot=64, inter=0, tr=0, gain=1.0, dt=0, out=at(3))
    a.update(k)
    return st.lib().sptp_rope(*a.values(), None)


def test_rope_refusals():
    for name in ("x", "pos", "turns", "out"):
        assert rope(**{name: None}) == NULL
    assert rope(dt=2) == DTYPE
    for bad in (dict(P=0), dict(P=9), dict(M=-1), dict(H=0), dict(Hr=0), dict(Hr=7), dict(D=60), dict(D=264), dict(D=0),
                dict(rot=0), dict(rot=8), dict(rot=72), dict(rot=80), dict(gain=math.nan), dict(gain=math.inf),
                dict(H=1 << 23, Hr=1), dict(x=at(0) + 8), dict(out=at(3) + 2), dict(pos=at(1) + 2), dict(turns=at(2) + 4)):
        assert rope(**bad) == SHAPE, bad
    nbytes = 2 * 8 * 6 * 64 * 2
    assert rope(out=at(0) + 16) == ALIAS and rope(out=at(0) + nbytes - 16) == ALIAS
    assert rope(out=at(1) - 16) == ALIAS and rope(out=at(2)) == ALIAS
    assert rope(M=0, x=None, pos=None, out=None) == OK


def append(**k):
    a = dict(qkv=at(0), pos=at(1), seq=at(2), table=at(3), turns=at(4), P=2, M=8, Hq=8, Hkv=2, D=64, rot=32, inter=0,
             gain=1.0, B=4, max_pages=8, num_pages=50, page=16, dt=0, kv=0, q=at(5), k=at(6), v=at(7), ks=None, vs=None,
             ws=at(8), wsb=1 << 20)
    a.update(k)
    return st.lib().sptp_rope_append_kv(*a.values(), None)


def test_append_refusals():
    for name in ("qkv", "pos", "seq", "table", "turns", "q", "k", "v", "ws"):
        assert append(**{name: None}) == NULL, name
    assert append(kv=1) == NULL and append(kv=1, ks=at(9)) == NULL
    assert append(dt=5) == DTYPE and append(kv=2) == DTYPE and append(kv=1, ks=at(9), vs=at(10), dt=1) == DTYPE
    for bad in (dict(P=0), dict(P=9), dict(M=-1), dict(Hq=7), dict(Hkv=0), dict(Hq=0), dict(D=36), dict(D=512), dict(rot=-16),
                dict(rot=24), dict(rot=80), dict(gain=math.nan), dict(B=-1), dict(max_pages=0), dict(num_pages=0),
                dict(page=0), dict(page=8), dict(page=24), dict(page=-16), dict(max_pages=1 << 27), dict(num_pages=1 << 27),
                dict(num_pages=1 << 25), dict(kv=1, ks=at(9), vs=at(10), D=72, rot=0), dict(qkv=at(0) + 4), dict(seq=at(2) + 1),
                dict(table=at(3) + 2), dict(k=at(6) + 8), dict(ws=at(8) + 16), dict(kv=1, ks=at(9) + 4, vs=at(10))):
        assert append(**bad) == SHAPE, bad
    assert append(wsb=4095) == WS
    for bad in (dict(q=at(0)), dict(k=at(0) + 64), dict(v=at(6) + 32), dict(q=at(7)), dict(ws=at(6)), dict(v=at(3)),
                dict(kv=1, ks=at(9), vs=at(9)), dict(kv=1, ks=at(5), vs=at(9)), dict(ws=at(4))):
        assert append(**bad) == ALIAS, bad
    assert append(M=0, qkv=None, pos=None, seq=None, table=None, q=None) == OK


def decode(**k):
    a = dict(q=at(0), k=at(1), v=at(2), ks=None, vs=None, table=at(3), lens=at(4), P=2, B=4, Hq=8, Hkv=2, D=64, max_pages=8,
             num_pages=50, page=16, window=0, scale=0.125, dt=0, kv=0, out=at(5), lse=at(6), ws=at(7), wsb=1 << 40)
    a.update(k)
    return st.lib().sptp_paged_attn_decode(*a.values(), None)


def test_decode_refusals():
    for name in ("q", "k", "v", "table", "lens", "out", "ws"):
        assert decode(**{name: None}) == NULL, name
    assert decode(kv=1) == NULL
    assert decode(dt=-1) == DTYPE and decode(kv=-1) == DTYPE and decode(kv=1, ks=at(9), vs=at(10), dt=1) == DTYPE
    for bad in (dict(P=0), dict(P=9), dict(B=-1), dict(Hq=9), dict(Hkv=0), dict(D=4), dict(D=260), dict(max_pages=0),
                dict(page=17), dict(window=-1), dict(scale=math.nan), dict(scale=math.inf), dict(num_pages=1 << 26),
                dict(kv=1, ks=at(9), vs=at(10), D=40), dict(q=at(0) + 2), dict(lens=at(4) + 2), dict(lse=at(6) + 4),
                dict(ws=at(7) + 128)):
        assert decode(**bad) == SHAPE, bad
    need = st.sptp_paged_attn_workspace_size(2, 4, 8, 2, 64)
    assert need >= st.SPTP_WS_HEADER_BYTES and decode(wsb=need - 1) == WS
    for bad in (dict(out=at(0)), dict(lse=at(1)), dict(out=at(6)), dict(ws=at(2)), dict(out=at(4)), dict(lse=at(3))):
        assert decode(**bad) == ALIAS, bad
    assert decode(B=0, q=None, table=None, lens=None, out=None, lse=None) == OK
    for bad in ((0, 4, 8, 2, 64), (2, -1, 8, 2, 64), (2, 4, 9, 2, 64), (2, 4, 8, 2, 63)):
        assert st.sptp_paged_attn_workspace_size(*bad) == 0


# ---------------------------------------------------------------- binding refusals

def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


I32 = torch.int32


def test_binding_checks_rope():
    args = dict(x=z(2, 4, 3, 32), positions=z(4, dtype=I32), turns=z(8, dtype=torch.int64))
    with pytest.raises(ValueError, match="device tensors only"):
        st.sptp_rope(**args)
    for k, v, err in (("positions", z(5, dtype=I32), ValueError), ("positions", z(4, dtype=torch.int64), TypeError),
                      ("turns", z(8, dtype=torch.float32), TypeError), ("out", z(2, 4, 3, 16), ValueError),
                      ("out", z(2, 4, 3, 32, dtype=torch.float32), TypeError), ("x", z(2, 4, 3, 32, dtype=torch.float16), TypeError)):
        with pytest.raises(err):
            st.sptp_rope(**dict(args, **{k: v}))


def test_binding_checks_append_and_decode():
    cache = st.paged_kv_cache(2, 5, 2, 16, 32, device="cpu")
    assert [tuple(t.shape) for t in cache[:2]] == [(2, 5, 2, 16, 32)] * 2 and cache[2] is None
    codes = st.paged_kv_cache(2, 5, 2, 16, 32, e4m3=True, device="cpu")
    assert codes[0].dtype == torch.uint8 and tuple(codes[3].shape) == (2, 5, 2, 16)
    args = dict(qkv=z(2, 4, 8 * 32), positions=z(4, dtype=I32), seq_ids=z(4, dtype=I32), page_table=z(3, 2, dtype=I32),
                turns=z(16, dtype=torch.int64), cache=cache, Hq=4)
    for c in (cache, codes):
        with pytest.raises(ValueError, match="device tensors only"):
            st.sptp_rope_append_kv(**dict(args, cache=c))
    for k, v, err in (("qkv", z(2, 4, 7 * 32), ValueError), ("seq_ids", z(3, dtype=I32), ValueError),
                      ("page_table", z(3, 2, dtype=torch.int64), TypeError), ("Hq", 5, ValueError),
                      ("q_out", z(2, 4, 128), ValueError), ("cache", (cache[0], cache[1][:, :4], None, None), ValueError),
                      ("cache", (codes[0], codes[1], None, None), ValueError), ("cache", (cache[0], cache[1], codes[2], None), ValueError),
                      ("cache", (cache[0][0], cache[1][0], None, None), ValueError),
                      ("cache", (cache[0], cache[1].float(), None, None), TypeError)):
        with pytest.raises(err):
            st.sptp_rope_append_kv(**dict(args, **{k: v}))
    with pytest.raises(TypeError, match="E4M3"):
        st.sptp_rope_append_kv(**dict(args, qkv=z(2, 4, 256, dtype=torch.float32), cache=codes))
    dec = dict(q=z(2, 3, 4, 32), cache=cache, page_table=z(3, 2, dtype=I32), seq_lens=z(3, dtype=I32))
    with pytest.raises(ValueError, match="device tensors only"):
        st.sptp_paged_attn_decode(**dec)
    for k, v, err in (("page_table", z(2, 2, dtype=I32), ValueError), ("seq_lens", z(3, dtype=torch.int64), TypeError),
                      ("out", z(2, 3, 4, 32), ValueError), ("lse", z(2, 3, 4), TypeError), ("q", z(2, 3, 4, 16), ValueError)):
        with pytest.raises(err):
            st.sptp_paged_attn_decode(**dict(dec, **{k: v}))


def test_packed_calls_are_the_calls():
    """The argument blocks have the C structs' layout: every field, set to a
    value that only it may have, reaches the check that it belongs to."""
    lib = st.lib()
    assert lib.sptp_rope_packed(None) == NULL and lib.sptp_rope_append_kv_packed(None) == NULL
    assert lib.sptp_paged_attn_decode_packed(None) == NULL

    def rope_p(**k):
        a = dict(x=at(0), pos=at(1), turns=at(2), out=at(3), stream=0, P=2, M=0, H=6, Hr=4, D=64, rot=64, inter=0, tr=0, dt=0,
                 gain=1.0)
        a.update(k)
        return lib.sptp_rope_packed(st._ROPE_ARGS.pack(*a.values()))

    assert rope_p() == OK
    for bad, code in ((dict(turns=0), NULL), (dict(x=0, M=1), NULL), (dict(pos=0, M=1), NULL), (dict(out=0, M=1), NULL),
                      (dict(dt=9), DTYPE), (dict(P=9), SHAPE), (dict(M=-1), SHAPE), (dict(H=0), SHAPE), (dict(Hr=7), SHAPE),
                      (dict(D=12), SHAPE), (dict(rot=24), SHAPE), (dict(gain=math.nan), SHAPE), (dict(out=at(2), M=1), ALIAS)):
        assert rope_p(**bad) == code, bad

    def append_p(**k):
        a = dict(qkv=at(0), pos=at(1), seq=at(2), table=at(3), turns=at(4), q=at(5), k=at(6), v=at(7), ks=0, vs=0, ws=at(8),
                 stream=0, wsb=1 << 20, P=2, M=0, Hq=8, Hkv=2, D=64, rot=32, inter=0, B=4, max_pages=8, num_pages=50, page=16,
                 dt=0, kv=0, gain=1.0)
        a.update(k)
        return lib.sptp_rope_append_kv_packed(st._APPEND_ARGS.pack(*a.values()))

    assert append_p() == OK
    for bad, code in ((dict(qkv=0, M=1), NULL), (dict(pos=0, M=1), NULL), (dict(seq=0, M=1), NULL), (dict(table=0, M=1), NULL),
                      (dict(turns=0), NULL), (dict(q=0, M=1), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(ws=0), NULL),
                      (dict(kv=1, ks=0, vs=at(9)), NULL), (dict(kv=1, ks=at(9), vs=0), NULL), (dict(dt=4), DTYPE),
                      (dict(kv=2), DTYPE), (dict(wsb=9), WS), (dict(P=0), SHAPE), (dict(M=-1), SHAPE), (dict(Hq=7), SHAPE),
                      (dict(Hkv=3), SHAPE), (dict(D=36), SHAPE), (dict(rot=24), SHAPE), (dict(B=-1), SHAPE),
                      (dict(max_pages=0), SHAPE), (dict(num_pages=0), SHAPE), (dict(page=8), SHAPE), (dict(gain=math.inf), SHAPE)):
        assert append_p(**bad) == code, bad

    def decode_p(**k):
        a = dict(q=at(0), k=at(1), v=at(2), ks=0, vs=0, table=at(3), lens=at(4), out=at(5), lse=at(6), ws=at(7), stream=0,
                 wsb=1 << 40, P=2, B=0, Hq=8, Hkv=2, D=64, max_pages=8, num_pages=50, page=16, window=0, dt=0, kv=0, scale=0.125)
        a.update(k)
        return lib.sptp_paged_attn_decode_packed(st._DECODE_ARGS.pack(*a.values()))

    assert decode_p() == OK
    for bad, code in ((dict(q=0, B=1), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(kv=1, ks=0, vs=at(9)), NULL),
                      (dict(kv=1, ks=at(9)), NULL), (dict(table=0, B=1), NULL), (dict(lens=0, B=1), NULL), (dict(out=0, B=1), NULL),
                      (dict(ws=0), NULL), (dict(lse=at(1), B=1), ALIAS), (dict(wsb=5), WS), (dict(dt=4), DTYPE), (dict(kv=3), DTYPE),
                      (dict(P=9), SHAPE), (dict(B=-1), SHAPE), (dict(Hq=9), SHAPE), (dict(Hkv=3), SHAPE), (dict(D=4), SHAPE),
                      (dict(max_pages=0), SHAPE), (dict(num_pages=0), SHAPE), (dict(page=24), SHAPE), (dict(window=-1), SHAPE),
                      (dict(scale=math.nan), SHAPE)):
        assert decode_p(**bad) == code, bad
