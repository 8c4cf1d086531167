"""The extension module of a decoding step's calls, without a GPU: it takes only
calls that are right as they stand, and leaves the others to the functions of
the package, which say what is wrong."""
import os

import pytest
import torch

import sequence_tensor_transformer_gb300 as st
from sequence_tensor_transformer_gb300 import build as build_mod


@pytest.fixture(scope="module")
def fast():
    if not os.path.exists(st.BINDING_PATH):
        build_mod.build()
    st.load_library()
    st.set_library(st.lib())
    assert st._fast is not None
    return st._fast


def test_the_module_calls_the_library_in_use(fast):
    handle = st.lib()
    st.set_library(None)
    assert st._fast is None
    st.set_library(handle)
    assert st._fast is fast


@pytest.mark.parametrize("addresses", [(), (1, 2), (1, 2, 3, 4), (0, 1, 2), ("a", 1, 2), (1.5, 1, 2)])
def test_addresses_are_checked(fast, addresses):
    with pytest.raises((TypeError, ValueError)):
        fast.use(*addresses)
    st.set_library(st.lib())


ROPE = dict(x=torch.zeros(2, 3, 4, 64), positions=torch.zeros(3, dtype=torch.int32), turns=torch.zeros(32, dtype=torch.int64),
            Hr=None, interleaved=False, transpose=False, gain=1.0, out=None)


@pytest.mark.parametrize("change", [{}, {"x": None}, {"x": 3}, {"x": torch.zeros(3)}, {"positions": [0, 1, 2]}, {"turns": None},
                                    {"Hr": 1.5}, {"Hr": 1 << 40}, {"gain": "1"}, {"gain": 1e300}, {"gain": 10 ** 400},
                                    {"interleaved": None}, {"out": 1}, {"x": torch.zeros(2, 3, 4, 64, device="meta")},
                                    {"x": torch.zeros(2, 3, 4, 64).to_sparse()}])
def test_rope_leaves_the_call(fast, change):
    assert fast.rope(*{**ROPE, **change}.values()) is NotImplemented


def test_wrong_numbers_of_arguments(fast):
    for call in (fast.rope, fast.append, fast.decode):
        for n in (0, 1, 7, 12):
            assert call(*[None] * n) is NotImplemented


def test_append_and_decode_leave_the_call(fast):
    cache = st.paged_kv_cache(1, 2, 1, 16, 64, device="cpu")
    table, ids = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    ws = torch.zeros(4096, dtype=torch.uint8)
    qkv, q = torch.zeros(1, 3, 4 * 64, dtype=torch.bfloat16), torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    for c in (cache, list(cache), cache[:3], None, (cache[0], None, None, None)):
        assert fast.append(qkv, ids, ids, table, None, c, 2, False, 1.0, None, ws) is NotImplemented
        assert fast.decode(q, c, table, ids[:1], None, 0, None, None, ws, True) is NotImplemented


def test_the_functions_say_what_is_wrong(fast):
    with pytest.raises(ValueError):
        st.sptp_rope(ROPE["x"], ROPE["positions"], ROPE["turns"])
    with pytest.raises(ValueError, match="positions"):
        st.sptp_rope(ROPE["x"], ROPE["positions"][:2], ROPE["turns"])
