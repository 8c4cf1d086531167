"""A cap that is no fp32 number but 0 is refused, not taken for none."""
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

from test_batch_ops_host import BF, _built, cpu_call  # noqa: F401

CAPS = pytest.mark.parametrize("cap", [1e-50, -1e-50, 5e-324, 1e-31])


def decode_arguments(device):
    P, B, Hq, D = 2, 3, 4, 64
    cache = tuple(torch.zeros(P, 4, 2, 16, D, dtype=BF, device=device) for _ in range(2)) + (None, None)
    i32 = dict(dtype=torch.int32, device=device)
    return torch.zeros(P, B, Hq, D, dtype=BF, device=device), cache, torch.zeros(B, 2, **i32), torch.zeros(B, **i32)


@CAPS
def test_caps_that_round_to_none(cap):
    with pytest.raises(st.SptpError):
        cpu_call(cap=cap)
    with pytest.raises(st.SptpError):
        st.sptp_paged_attn_decode(*decode_arguments("cpu"), cap=cap)


@pytest.mark.gpu
@CAPS
def test_caps_that_round_to_none_through_the_extension_module(cap):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    q, cache, table, lens = decode_arguments("cuda")
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    with pytest.raises(st.SptpError):
        st.sptp_paged_attn_decode(q, cache, table, lens, cap=cap, workspace=ws)
    starts = torch.arange(4, dtype=torch.int32, device="cuda")
    with pytest.raises(st.SptpError):
        st.sptp_paged_attn_prompt(q, cache, table, lens, starts, cap=cap, workspace=ws)
