"""GPU parity of the rotary positions and of their append to a paged
key-value cache, against the float64 oracle.

Bounds, per element.  An angle is off by at most 2^-25 of a turn (1.9e-7 rad),
its sine and cosine by 2 ulp (1.2e-7) more, the gain's product, the two
products and the sum by 2^-24 each of at most |a| + |b|: together under
1e-6 gain (|a| + |b|).  The result is rounded once: half a step, 2^-8 (bf16)
or 2^-24 (fp32) of the value.  What is copied is equal bit for bit."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st
from oracle import attn_oracle as ao
from oracle import fp8_oracle as f8
from sequence_tensor_transformer_gb300 import synth

from helpers import dev_tensor, host_f64, nan_tensor, nan_workspace, to_f64

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
TD = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


def draw(rng, shape, dtype):
    return synth._cast(rng.standard_normal(shape), dtype)


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def close(got, ref, pair, dtype, gain=1.0):
    tol = HALF[dtype] * np.abs(ref) + 1e-6 * abs(gain) * pair
    assert not np.isnan(got).any(), "an element was never written"
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])


def angles(pos, turns):
    return ao.angles_from_turns(pos, turns.cpu().tolist())


# ---------------------------------------------------------------- rotation

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("P,M,H,Hr,D,rot", [(1, 1, 1, 1, 16, 16), (4, 1, 9, 8, 128, 128), (2, 33, 5, 3, 80, 32), (1, 700, 3, 3, 64, 48),
                                            (3, 7, 24, 20, 256, 256), (8, 5, 2, 1, 24, 16), (2, 3001, 4, 4, 96, 96), (1, 2, 65, 64, 40, 32),
                                            (1, 5, 7, 7, 136, 64)])
def test_rope(P, M, H, Hr, D, rot, inter, dtype):
    rng = np.random.default_rng(P * M + D)
    x = draw(rng, (P, M, H, D), dtype)
    pos = rng.integers(0, 1 << 20, M)
    pos[0] = 0
    turns = st.sptp_rope_turns(rot, 10000.0, "parts", 8.0, 4096)
    gain = 1.2079441541679836
    for transpose in (False, True):
        out = nan_tensor((P, M, H, D), TD[dtype])
        r = st.sptp_rope(dev_tensor(x, dtype), ints(pos), turns, Hr, inter, transpose, gain, out=out)
        assert r is out
        x64 = to_f64(x, dtype)
        ref = ao.rope(x64, angles(pos, turns), Hr, inter, transpose, gain)
        got = host_f64(out)
        close(got, ref, ao.rope_pair_sizes(x64, rot // 2, Hr, inter), dtype, gain)
        assert np.array_equal(got[..., rot:], x64[..., rot:]) and np.array_equal(got[:, :, Hr:], x64[:, :, Hr:])
        # in place: the same bits
        t = dev_tensor(x, dtype)
        assert st.sptp_rope(t, ints(pos), turns, Hr, inter, transpose, gain, out=t) is t
        assert torch.equal(t, out)


def test_rope_every_int32_position():
    """Angles stay exact at the ends of int32, negative positions among them."""
    pos = np.array([-2 ** 31, -2 ** 31 + 1, -1, 0, 1, 2 ** 24 + 1, 2 ** 31 - 2, 2 ** 31 - 1])
    rng = np.random.default_rng(5)
    x = draw(rng, (1, len(pos), 2, 128), "fp32")
    turns = st.sptp_rope_turns(128, 500000.0)
    got = host_f64(st.sptp_rope(dev_tensor(x, "fp32"), ints(pos), turns))
    ref = ao.rope(to_f64(x, "fp32"), angles(pos, turns), 2)
    close(got, ref, ao.rope_pair_sizes(to_f64(x, "fp32"), 64, 2), "fp32")


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient_against_differences(inter):
    """The rotation is linear: its gradient for a weight w on the outputs is
    the difference quotient of sum(w y) along every unit vector."""
    rng = np.random.default_rng(6)
    M, D, rot, gain = 3, 32, 16, 1.5
    turns = st.sptp_rope_turns(rot, 100.0)
    pos = ints([0, 3, 77])
    w = torch.randn(1, M, 1, D, device="cuda")
    g = st.sptp_rope(w, pos, turns, 1, inter, True, gain)
    x = dev_tensor(draw(rng, (1, M, 1, D), "fp32"), "fp32")
    base = st.sptp_rope(x, pos, turns, 1, inter, False, gain)
    for d in range(D):
        step = x.clone()
        step[..., d] += 1.0
        q = ((st.sptp_rope(step, pos, turns, 1, inter, False, gain) - base).double() * w.double()).sum(-1)
        # x + 1, two roundings of values below 12, sums of two terms
        assert torch.allclose(q, g[..., d].double(), atol=1e-5)


def test_rope_no_rows():
    x = torch.empty((2, 0, 3, 32), dtype=torch.bfloat16, device="cuda")
    assert st.sptp_rope(x, ints([]), st.sptp_rope_turns(32)).shape == x.shape


# ---------------------------------------------------------------- append

def append_case(P, M, Hq, Hkv, D, rot, B, page, dtype, e4m3, inter, seed=0, pad=2):
    """Random rows of B sequences at distinct slots, in random order."""
    rng = np.random.default_rng(seed + M + D)
    max_pages = 7
    num_pages = B * max_pages + 2
    table = rng.permutation(num_pages)[: B * max_pages].reshape(B, max_pages)
    slots = rng.choice(B * max_pages * page, M, replace=False)
    seq, pos = slots // (max_pages * page), slots % (max_pages * page)
    for i in rng.choice(M, min(pad, M - 1), replace=False):
        seq[i] = -1 - i
    qkv = draw(rng, (P, M, (Hq + 2 * Hkv) * D), dtype)
    kind = torch.uint8 if e4m3 else TD[dtype]
    shape = (P, num_pages, Hkv, page, D)
    cache = [nan_tensor(shape, kind), nan_tensor(shape, kind), None, None]
    if e4m3:
        cache[2:] = nan_tensor(shape[:-1], torch.float32), nan_tensor(shape[:-1], torch.float32)
    return dict(qkv=qkv, seq=seq, pos=pos, table=table, cache=tuple(cache), rot=rot, Hq=Hq, dtype=dtype, e4m3=e4m3, inter=inter)


def check_append(c, turns, q_out):
    P, M, N = c["qkv"].shape
    k, v, ks, vs = c["cache"]
    _, num_pages, Hkv, page, D = k.shape
    Hq, dtype, rot = c["Hq"], c["dtype"], c["rot"]
    x = to_f64(c["qkv"], dtype).reshape(P, M, Hq + 2 * Hkv, D)
    ref = ao.rope(x, angles(c["pos"], turns), Hq + Hkv, c["inter"]) if rot else x
    pair = ao.rope_pair_sizes(x, rot // 2, Hq + Hkv, c["inter"])
    live = c["seq"] >= 0
    got = host_f64(q_out)
    assert np.isnan(got[:, ~live]).all(), "a padding row was written"
    close(got[:, live], ref[:, live, :Hq], pair[:, live, :Hq], dtype)
    pages, off = c["table"][c["seq"][live], c["pos"][live] // page], c["pos"][live] % page
    written = np.zeros((num_pages, page), bool)
    written[pages, off] = True
    for pool, scale, first, rotated in ((k, ks, Hq, True), (v, vs, Hq + Hkv, False)):
        want, size = ref[:, live, first: first + Hkv], pair[:, live, first: first + Hkv]
        if not c["e4m3"]:
            all_ = host_f64(pool)
            have = all_[:, pages, :, off].transpose(1, 0, 2, 3)  # [P, rows, Hkv, D]
            close(have, want, size, dtype)
            assert np.isnan(all_.transpose(1, 3, 0, 2, 4)[~written]).all(), "a slot of another token was written"
            continue
        codes, sc = pool.cpu().numpy(), scale.cpu().numpy()
        assert (codes.transpose(1, 3, 0, 2, 4)[~written] == 0xFF).all()
        assert np.isnan(sc.transpose(1, 3, 0, 2)[~written]).all()
        have_c, have_s = codes[:, pages, :, off].transpose(1, 0, 2, 3), sc[:, pages, :, off].transpose(1, 0, 2)
        if not rotated or not rot:
            cw, sw = ao.quantise_rows(want)
            assert np.array_equal(have_c, cw) and np.array_equal(have_s, sw)
            continue
        # the value rounded to bf16 (2^-8), then to E4M3: half a step, 2^-4 of
        # the value or 2^-10 of the scale below the smallest normal code
        val = ao.dequantised(have_c, have_s)
        one = 2.0 ** -8 * np.abs(want) + 1e-6 * size
        tol = one + np.maximum(2.0 ** -4 * (np.abs(want) + one), 2.0 ** -10 * have_s[..., None])
        assert (np.abs(val - want) <= tol).all()
        # and the scale is the least that holds the row: its largest code is above 224 (the next scale's 448)
        top = np.abs(val).max(-1) / have_s
        assert ((top > 216) | (have_s == 2.0 ** -126)).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,e4m3", [("bf16", False), ("fp32", False), ("bf16", True)])
@pytest.mark.parametrize("P,M,Hq,Hkv,D,rot,B,page", [
    (4, 1, 7, 1, 128, 128, 1, 16), (2, 64, 8, 4, 64, 64, 5, 16), (1, 300, 3, 3, 80, 32, 3, 48), (2, 37, 16, 2, 256, 256, 4, 32),
    (3, 130, 10, 2, 96, 96, 2, 64), (8, 9, 1, 1, 16, 16, 9, 128), (1, 50, 4, 4, 128, 0, 2, 16), (2, 2500, 14, 2, 64, 32, 8, 112)])
def test_append(P, M, Hq, Hkv, D, rot, B, page, dtype, e4m3, inter):
    c = append_case(P, M, Hq, Hkv, D, rot, B, page, dtype, e4m3, inter)
    turns = st.sptp_rope_turns(rot) if rot else None
    ws, q = nan_workspace(st.SPTP_WS_HEADER_BYTES), nan_tensor((P, M, Hq, D), TD[dtype])
    r = st.sptp_rope_append_kv(dev_tensor(c["qkv"], dtype), ints(c["pos"]), ints(c["seq"]), ints(c["table"]), turns,
                               c["cache"], Hq, inter, q_out=q, workspace=ws)
    assert r is q and st.sptp_read_device_status(ws) == 0
    check_append(c, turns, q)


def test_append_zero_and_tiny_rows_e4m3():
    """Zero rows take the least scale; rows far below one keep their codes."""
    c = append_case(1, 6, 2, 1, 32, 16, 1, 16, "bf16", True, False, pad=0)
    x = to_f64(c["qkv"], "bf16")
    x[:, 0] = 0
    x[:, 1] *= 2.0 ** -100
    x[:, 2] *= 2.0 ** 60
    c["qkv"] = synth._cast(x, "bf16")
    turns = st.sptp_rope_turns(16)
    q = nan_tensor((1, 6, 2, 32))
    st.sptp_rope_append_kv(dev_tensor(c["qkv"], "bf16"), ints(c["pos"]), ints(c["seq"]), ints(c["table"]), turns, c["cache"], 2,
                           q_out=q)
    check_append(c, turns, q)


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_bad_indexes_are_recorded_and_skipped(e4m3):
    """A sequence, position or page outside its range: status, no store, the
    other rows as ever; the next call's status is its own."""
    c = append_case(2, 40, 4, 2, 64, 64, 3, 16, "bf16", e4m3, False, pad=0)
    turns = st.sptp_rope_turns(64)
    ws = nan_workspace(st.SPTP_WS_HEADER_BYTES)
    span = 7 * 16
    good_seq, good_pos, good_table = c["seq"].copy(), c["pos"].copy(), c["table"].copy()
    for name in ("seq", "pos+", "pos-", "page+", "page-"):
        seq, pos, table = good_seq.copy(), good_pos.copy(), good_table.copy()
        bad = np.zeros(40, bool)
        if name == "seq":
            seq[[5, 17]] = [3, 2 ** 31 - 1]
            bad[[5, 17]] = True
        elif name.startswith("pos"):
            pos[11] = span if name == "pos+" else -1
            bad[11] = True
        else:
            s, j = good_seq[7], good_pos[7] // 16
            table[s, j] = c["cache"][0].shape[1] if name == "page+" else -1
            bad = (good_seq == s) & (good_pos // 16 == j)
        for t in c["cache"]:
            if t is not None:
                t.fill_(0xFF if t.dtype == torch.uint8 else float("nan"))
        q = nan_tensor((2, 40, 4, 64))
        st.sptp_rope_append_kv(dev_tensor(c["qkv"], "bf16"), ints(pos), ints(seq), ints(table), turns, c["cache"], 4, q_out=q,
                               workspace=ws)
        assert st.sptp_read_device_status(ws) == st.STATUS["shape"]
        assert ws[:20].view(torch.int32).tolist()[3] == np.flatnonzero(bad)[0]  # the first such row
        assert not torch.isnan(q).any()  # q is rotated all the same
        q[:, torch.from_numpy(bad).cuda()] = float("nan")
        check_append(dict(c, seq=np.where(bad, -1, seq), pos=pos, table=np.where((table < 0) | (table >= c["cache"][0].shape[1]), 0, table)),
                     turns, q)
    st.sptp_rope_append_kv(dev_tensor(c["qkv"], "bf16"), ints(good_pos), ints(good_seq), ints(good_table), turns, c["cache"], 4,
                           workspace=ws)
    assert st.sptp_read_device_status(ws) == 0


def test_append_all_padding():
    c = append_case(1, 9, 2, 1, 32, 16, 1, 16, "bf16", False, False)
    q = nan_tensor((1, 9, 2, 32))
    ws = nan_workspace(4096)
    st.sptp_rope_append_kv(dev_tensor(c["qkv"], "bf16"), ints(c["pos"]), ints([-1] * 9), ints(c["table"]), st.sptp_rope_turns(16),
                           c["cache"], 2, q_out=q, workspace=ws)
    assert st.sptp_read_device_status(ws) == 0 and torch.isnan(q).all() and torch.isnan(c["cache"][0]).all()


def test_append_past_2_31_elements():
    """Slots whose element offsets pass 32 bits (a pool of 4.3 GB a side)."""
    P, Hkv, page, D = 1, 8, 64, 256
    num_pages = (1 << 31) // (Hkv * page * D) + 40
    cache = tuple(torch.zeros((P, num_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)) + (None, None)
    rng = np.random.default_rng(9)
    x = draw(rng, (P, 3, 24 * D), "bf16")
    table = np.array([[num_pages - 1, 0, num_pages - 17]])
    pos = np.array([63, 64, 140])
    turns = st.sptp_rope_turns(256)
    st.sptp_rope_append_kv(dev_tensor(x, "bf16"), ints(pos), ints([0, 0, 0]), ints(table), turns, cache, 8)
    x64 = to_f64(x, "bf16").reshape(1, 3, 24, D)
    ref = ao.rope(x64, angles(pos, turns), 16)
    pair = ao.rope_pair_sizes(x64, 128, 16)
    for i, (pg, off) in enumerate(((num_pages - 1, 63), (0, 0), (num_pages - 17, 12))):
        close(host_f64(cache[0][0, pg, :, off]), ref[0, i, 8:16], pair[0, i, 8:16], "bf16")
        close(host_f64(cache[1][0, pg, :, off]), ref[0, i, 16:], 0, "bf16")
    assert int((cache[0] != 0).any(-1).sum()) == 24 and int((cache[1] != 0).any(-1).sum()) == 24
