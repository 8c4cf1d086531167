"""The way out of the one-token attention when a bounded wait runs out: with an
arrival withheld in one CTA the kernel ends by itself, the status words say so,
and the next call on the same workspace is right."""
import time

import pytest
import torch

import sequence_tensor_transformer_gb300 as st

import test_gpu_paged_attn as ta
from helpers import nan_workspace

pytestmark = pytest.mark.gpu

LIMIT = 20_000_000  # ns
WHERE_FULL, WHERE_EMPTY = 16, 17


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)


def withheld(c, lens=None, **kw):
    """(status code, words) of a call with an arrival withheld; it ends within a
    few of its limits."""
    n = st.sptp_paged_attn_workspace_size(c["P"], c["B"], c["Hq"], c["Hkv"], c["D"])
    ws, out = nan_workspace(n), torch.empty(c["P"], c["B"], c["Hq"] * c["D"], dtype=ta.TD[c["dtype"]], device="cuda")
    torch.cuda.synchronize()
    t = time.perf_counter()
    st.sptp_paged_attn_wait_selftest(c["q"], c["cache"], ta.ints(c["table"]), ta.ints(c["lens"] if lens is None else lens), out, ws,
                                     limit_ns=LIMIT, **kw)
    code = st.sptp_read_device_status(ws)
    assert time.perf_counter() - t < 2.0
    return code, ws[:20].view(torch.int32).tolist(), ws


@pytest.mark.parametrize("kind", ta.KINDS)
@pytest.mark.parametrize("Hq", [5, 20])
@pytest.mark.parametrize("role", [dict(withhold_full=0), dict(withhold_full=1), dict(withhold_full=9), dict(withhold_empty=0), dict(withhold_empty=2)])
def test_a_wait_that_runs_out_ends_the_kernel(kind, Hq, role):
    c = ta.make(1, [1500, 2500, 700], Hq, 1, 128, 16, kind)
    code, words, ws = withheld(c, **role)
    assert code == st.STATUS["timeout"] and words[1] in (WHERE_FULL, WHERE_EMPTY) and words[2] == 0
    if "withhold_full" in role:
        assert words[1] == WHERE_FULL and words[3] == role["withhold_full"]
    # the workspace serves the next call
    out, lse = st.sptp_paged_attn_decode(c["q"], c["cache"], ta.ints(c["table"]), ta.ints(c["lens"]), c["scale"], workspace=ws)
    assert st.sptp_read_device_status(ws) == 0
    ta.check(c, out, lse)


@pytest.mark.parametrize("kind", ta.KINDS)
def test_nothing_withheld(kind):
    """A tile that the CTA does not have: the call is an ordinary one."""
    c = ta.make(1, [1500, 2500, 700], 5, 1, 128, 16, kind)
    for role in (dict(withhold_full=100000), dict(withhold_empty=100000)):
        assert withheld(c, **role)[0] == 0


@pytest.mark.parametrize("kind", ta.KINDS)
@pytest.mark.parametrize("role", [dict(withhold_full=3), dict(withhold_empty=1)])
def test_a_wait_that_ran_out_is_not_hidden_by_a_bad_index(kind, role):
    """A length outside the table (seen by every CTA) and pages outside the pool
    (in either CTA's share) leave the outputs defined, a wait that ran out does
    not: that is what is reported."""
    c = ta.make(1, [1500, 2500, 700], 5, 1, 128, 16, kind)
    for lens in ([1500, 2500, -1], [1500, 2500, 1 << 30], [-7, 2500, 1500]):
        assert withheld(c, lens=lens, **role)[0] == st.STATUS["timeout"]
    for b, j in ((0, 0), (0, 50), (1, 150), (2, 40)):
        table = c["table"].copy()
        table[b, j] = -1
        assert withheld(dict(c, table=table), **role)[0] == st.STATUS["timeout"]
        assert withheld(dict(c, table=table), withhold_full=100000)[0] == st.STATUS["shape"]
