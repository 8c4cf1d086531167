"""CPU tests of sptp_lora_ex: every refusal, and calls that are only checked (nothing here
reaches a GPU)."""
import pytest

import sequence_tensor_transformer_gb300 as st

from test_batch_ops_host import A, ALIAS, NULL, OK, SHAPE, WS, _built  # noqa: F401


def lora_ex(**kw):
    a = dict(x=A, A=2 * A, B=3 * A, ids=4 * A, gains=5 * A, P=2, M=5, K=64, N=96, R=16, n=3, rowwise=0, dtype=0, base=6 * A,
             out=7 * A, ws=8 * A, ws_bytes=1 << 40, stream=None, status=None, check=1)
    a.update(kw)
    return st.lib().sptp_lora_ex(*a.values())


def test_a_call_that_is_only_checked():
    assert lora_ex() == OK and lora_ex(status=9 * A) == OK and lora_ex(out=6 * A, status=9 * A) == OK
    assert lora_ex(M=0, check=0) == OK
    # rows of x behind a header whose words take the status
    assert lora_ex(x=9 * A + 4096, status=9 * A) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(ws=None), NULL), (dict(x=None), NULL), (dict(out=None), NULL), (dict(R=12), SHAPE), (dict(K=60), SHAPE),
    (dict(ws_bytes=4096), WS), (dict(out=2 * A), ALIAS), (dict(ws=3 * A), ALIAS), (dict(status=9 * A + 16), SHAPE),
    (dict(status=A), ALIAS), (dict(status=7 * A), ALIAS), (dict(status=8 * A), ALIAS)])
def test_refusals(kw, code):
    for check in (0, 1):
        assert lora_ex(**kw, check=check) == code
