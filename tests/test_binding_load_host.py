"""The extension module where it cannot be loaded: the library works without it."""
import os
import subprocess
import sys

import pytest

import sequence_tensor_transformer_gb300 as st

BROKEN = """
extern int sptp_no_such_symbol_anywhere(void);
void *PyInit__decode_binding(void) { return (void *)(long)sptp_no_such_symbol_anywhere(); }
"""


@pytest.fixture
def restored():
    if not (os.path.exists(st.LIB_PATH) and os.path.exists(st.BINDING_PATH)):
        from sequence_tensor_transformer_gb300 import build
        build.build()
    handle = st.load_library()
    st.set_library(handle)
    yield handle
    st.set_library(handle)
    assert st._fast is not None


@pytest.fixture
def hidden(restored):
    """The module as if it had never been imported."""
    name = st.__name__ + "._decode_binding"
    module = sys.modules.pop(name)
    attribute = st.__dict__.pop("_decode_binding")
    yield name
    sys.modules[name] = module
    st._decode_binding = attribute


def broken_module(tmp_path, kind):
    so = tmp_path / "_decode_binding.so"
    if kind == "no module":
        so.write_bytes(b"not a shared object")
    else:
        src = tmp_path / "m.c"
        src.write_text(BROKEN)
        subprocess.run(["gcc", "-shared", "-fPIC", "-Wl,-z,now", "-o", str(so), str(src)], check=True)
    return so


@pytest.mark.parametrize("kind", ["no module", "undefined symbol"])
def test_a_module_that_cannot_be_loaded(hidden, tmp_path, monkeypatch, kind):
    so = broken_module(tmp_path, kind)
    monkeypatch.setattr(st, "__path__", [str(tmp_path)])
    monkeypatch.setattr(st, "BINDING_PATH", str(so))
    monkeypatch.setattr(st, "_lib", None)
    with pytest.warns(RuntimeWarning, match="cannot be loaded"):
        assert st.sptp_status_string(0)  # the first call of any function loads the library
    assert st._fast is None
    assert st.sptp_rope_turns(16, device="cpu").shape == (8,)


def test_without_the_module(restored, tmp_path, monkeypatch):
    monkeypatch.setattr(st, "BINDING_PATH", str(tmp_path / "none.so"))
    st.set_library(restored)
    assert st._fast is None and st.sptp_rope_turns(16, device="cpu").shape == (8,)
