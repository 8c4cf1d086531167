"""Refusals of the attention's wait self-test (nothing here reaches a GPU)."""
import os

import pytest
import torch

import sequence_tensor_transformer_gb300 as st


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(st.LIB_PATH):
        from sequence_tensor_transformer_gb300 import build
        build.build()
    st.load_library()


def args(D=128, base=1 << 20, **k):
    """A call that is right as far as the host can tell, on addresses that are never read."""
    p = [base * (i + 1) for i in range(11)]
    v = dict(q=p[0], k=p[1], v=p[2], ks=0, vs=0, table=p[5], lens=p[6], out=p[7], lse=0, ws=p[9], stream=0, ws_bytes=1 << 40,
             P=1, B=1, Hq=2, Hkv=1, D=D, max_pages=2, num_pages=2, page_size=16, window=0, dtype=0, kv_type=0, scale=1.0)
    v.update(k)
    return st._DECODE_ARGS.pack(*v.values())


def test_refusals():
    f = st.lib().sptp_paged_attn_wait_selftest
    NULL, SHAPE, WS = -1, -2, -4
    assert f(None, 0, -1, 1000) == NULL
    assert f(args(q=0), 0, -1, 1000) == NULL
    assert f(args(), 0, -1, 0) == SHAPE                # no limit
    assert f(args(), 0, -1, 10_000_000_001) == SHAPE   # more than ten seconds
    assert f(args(), -1, -1, 1000) == SHAPE            # nothing withheld
    assert f(args(), 0, 0, 1000) == SHAPE              # both
    assert f(args(D=136), 0, -1, 1000) == SHAPE
    assert f(args(page_size=24), 0, -1, 1000) == SHAPE
    assert f(args(ws_bytes=4096), 0, -1, 1000) == WS
    assert f(args(B=0), 0, -1, 1000) == 0


def test_binding():
    q = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    cache = st.paged_kv_cache(1, 2, 1, 16, 64, device="cpu")
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    out, ws = torch.zeros(1, 2, 128, dtype=torch.bfloat16), torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="seq_lens"):
        st.sptp_paged_attn_wait_selftest(q, cache, table, lens[:1], out, ws, 0)
    with pytest.raises(ValueError, match="device"):
        st.sptp_paged_attn_wait_selftest(q, cache, table, lens, out, ws, 0)
