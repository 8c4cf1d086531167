"""Row starts, lengths and pages outside their range, of prompts' attention: reported whichever
sequence they belong to."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

from batch_cases import arguments, call, check, ints, make, workspace

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp32", "e4m3"]
SHAPE, TIMEOUT = st.STATUS["shape"], st.STATUS["timeout"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("starts", [
    (0, 600, 100), (0, 500, 500, 10), (0, 700, 0), (0, 300, 299, 700), (650, 10, 20, 30), (0, 0, 699, 1, 1), (0, 701), (-1, 700)])
def test_row_starts_that_descend_or_leave_the_batch_are_reported(kind, starts):
    B = len(starts) - 1
    c = make(1, (700,) + (0,) * (B - 1), (900,) * B, 4, 2, 64, 16, kind, holes=False)
    c["starts"] = np.array(starts)
    ws = workspace(c)
    args, kw = arguments(c)
    st.sptp_paged_attn_prompt(*args, **kw, workspace=ws)
    assert st.sptp_read_device_status(ws) == SHAPE
    # the next call is not affected
    c = make(1, (30, 4), (100, 200), 4, 2, 64, 16, kind)
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0
    check(c, out, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("at", [0, 257, 599])
def test_a_bad_length_among_many_is_reported(kind, at):
    c = make(1, (1,) * 600, (20,) * 600, 2, 1, 64, 16, kind, holes=False)
    args, kw = arguments(c)
    beyond = c["table"].shape[1] * 16 + 1
    for bad in (-1, beyond, 0):  # 0: more rows than keys
        lens = np.array(c["lens"])
        lens[at] = bad
        ws = workspace(c)
        st.sptp_paged_attn_prompt(*args[:3], ints(lens), args[4], **kw, workspace=ws)
        assert st.sptp_read_device_status(ws) == SHAPE
        assert ws.view(torch.int32)[3].item() == at  # which sequence
    out, lse, ws = call(c)
    assert st.sptp_read_device_status(ws) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_wait_that_ran_out_is_reported_whatever_else_is_wrong(kind):
    c = make(1, (300, 0), (1500, 20), 4, 1, 128, 16, kind)
    ws = workspace(c)
    args, _ = arguments(c)
    args = (*args[:3], ints([1500, -1]), args[4])
    out = torch.empty(1, 300, 4 * 128, dtype=torch.bfloat16, device="cuda")
    st.sptp_paged_attn_prompt_wait_selftest(*args, out, ws, 1)
    assert st.sptp_read_device_status(ws) == TIMEOUT
