"""Calls whose every tensor is left out reach the library's own check."""
import os

import pytest

import sequence_tensor_transformer_gb300 as st


@pytest.fixture(autouse=True)
def _built():
    if not os.path.exists(st.LIB_PATH):
        from sequence_tensor_transformer_gb300 import build
        build.build()
    st.load_library()


def test_status_of_no_workspace(monkeypatch):
    monkeypatch.setattr(st, "_stream", lambda stream: 0)
    assert st.sptp_read_device_status(None) == st.STATUS["null"]


def test_no_tensors_are_on_one_device():
    assert st._same_device() is None and st._same_device(None, None) is None
