"""Pins of the oracles of prompts' attention and of low-rank adapters (CPU)."""
import numpy as np

from oracle import attn_oracle as ao


def case(P=2, lens=(9, 4, 0), rows=(3, 4, 0), Hq=4, Hkv=2, D=8, page=16):
    rng = np.random.default_rng(3)
    table = rng.permutation(8)[: len(lens) * 2].reshape(len(lens), 2)
    starts = np.concatenate([[0], np.cumsum(rows)])
    q = rng.standard_normal((P, int(starts[-1]), Hq, D))
    k, v = (rng.standard_normal((P, 8, Hkv, page, D)) for _ in range(2))
    return q, k, v, table, np.array(lens), starts


def test_last_rows_are_the_one_token_attention():
    q, k, v, table, lens, starts = case()
    out, lse, _, _ = ao.paged_attn_prompt(q, k, v, table, lens, starts, 0.3, window=5)
    for b in range(2):
        last = q[:, starts[b + 1] - 1: starts[b + 1]]
        o, l, _, _ = ao.paged_attn_decode(last, k, v, table[b: b + 1], lens[b: b + 1], 0.3, 5)
        assert np.allclose(out[:, starts[b + 1] - 1], o[:, 0]) and np.allclose(lse[:, starts[b + 1] - 1], l[:, 0])


def test_a_whole_prefix_is_uncaused_attention():
    q, k, v, table, lens, starts = case(lens=(6,), rows=(6,))
    out, lse, _, _ = ao.paged_attn_prompt(q, k, v, table, lens, starts, 0.3, prefix_lens=[6])
    K, V = k[:, table[0][0], :, :6], v[:, table[0][0], :, :6]  # [P, Hkv, 6, D]
    z = np.einsum("pmhd,phjd->pmhj", q, np.repeat(K, 2, 1)) * 0.3
    w = np.exp(z)
    assert np.allclose(out, np.einsum("pmhj,phjd->pmhd", w / w.sum(-1, keepdims=True), np.repeat(V, 2, 1)))
    assert np.allclose(lse, np.log(w.sum(-1)))


def test_caps_and_biases():
    z = np.linspace(-50, 50, 101)
    assert np.allclose(ao.modified_scores(z, 1e9, 0.0, 0), z) and np.abs(ao.modified_scores(z, 3.0, 0.0, 0)).max() < 3
    assert np.allclose(ao.modified_scores(z, 0, 0.5, np.arange(101)), z - 0.5 * np.arange(101))
    # a steep slope leaves the nearest key alone
    q, k, v, table, lens, starts = case(lens=(5,), rows=(5,))
    out, _, _, _ = ao.paged_attn_prompt(q, k, v, table, lens, starts, 0.3, slopes=np.full((2, 4), 200.0))
    for m in range(5):
        assert np.allclose(out[:, m], np.repeat(v[:, table[0][0], :, m], 2, 1))


def test_rows_without_keys_and_rows_of_no_sequence():
    q, k, v, table, lens, starts = case(lens=(2,), rows=(3,))
    q = np.concatenate([q, q[:, :1]], 1)
    out, lse, _, _ = ao.paged_attn_prompt(q, k, v, table, lens, starts, 1.0)
    assert not out[:, 0].any() and np.isneginf(lse[:, 0]).all() and np.isnan(out[:, 3]).all()


def test_adapters_are_a_change_of_the_weights():
    rng = np.random.default_rng(5)
    P, M, K, N, R = 2, 5, 16, 32, 8
    A, B, x = rng.standard_normal((3, R, K)), rng.standard_normal((3, N, R)), rng.standard_normal((M, K))
    ids, gains = np.array([2, -1, 0, 0, 1]), np.array([0.5, 2.0, -1.0])
    W = rng.standard_normal((N, K))
    base = (x @ W.T).reshape(M, P, N // P).transpose(1, 0, 2)
    got, _ = ao.lora(x, A, B, ids, base, gains)
    for m in range(M):
        Wm = W if ids[m] < 0 else W + gains[ids[m]] * B[ids[m]] @ A[ids[m]]
        assert np.allclose(got[:, m].ravel(), Wm @ x[m])
    # split over the shards' inputs: the partials sum to the same
    xs = x.reshape(M, P, K // P).transpose(1, 0, 2)
    parts = np.stack([xs[p] @ W[:, p * K // P:(p + 1) * K // P].T for p in range(P)])
    rows, _ = ao.lora(xs, A, B, ids, parts, gains)
    assert np.allclose(rows.sum(0), got.transpose(1, 0, 2).reshape(M, N))
