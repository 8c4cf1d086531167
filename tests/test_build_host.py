"""Which object the extension module is linked from, with the compiler calls
replaced: it is the one of the torch and the Python in use."""
import os
import shutil
import sysconfig

import pytest
import torch

from sequence_tensor_transformer_gb300 import build as b


@pytest.fixture
def built(tmp_path, monkeypatch):
    """build(torch version, SOABI) makes the module in a folder of its own and
    returns the compiler's and the linker's calls; module() is what it holds."""
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_decode_binding.so"))
    calls = []

    def run(cmd):
        out = cmd[cmd.index("-o") + 1]
        calls.append("compile" if "-c" in cmd else "link")
        with open(out, "w") as f:
            if "-c" in cmd:
                f.write(f"{torch.__version__} {sysconfig.get_config_var('SOABI')}")
            else:
                with open(next(a for a in cmd if a.endswith(".o"))) as g:
                    f.write(g.read())

    monkeypatch.setattr(b, "_run", run)
    config = sysconfig.get_config_var

    class Built:
        def build(self, version, abi="cpython-312"):
            monkeypatch.setattr(torch, "__version__", version)
            monkeypatch.setattr(sysconfig, "get_config_var", lambda n: abi if n == "SOABI" else config(n))
            del calls[:]
            b._build_binding()
            return list(calls)

        def module(self):
            with open(b.BINDING) as f:
                return f.read()

    return Built()


def test_linked_from_the_torch_in_use(built):
    assert built.build("2.0") == ["compile", "link"] and built.module() == "2.0 cpython-312"
    assert built.build("2.0") == []
    assert built.build("2.1") == ["compile", "link"] and built.module() == "2.1 cpython-312"
    assert built.build("2.0") == ["link"] and built.module() == "2.0 cpython-312"
    assert built.build("2.1") == ["link"] and built.module() == "2.1 cpython-312"
    assert built.build("2.1") == []


def test_linked_from_the_python_in_use(built):
    built.build("2.0")
    assert built.build("2.0", "cpython-313") == ["compile", "link"] and built.module() == "2.0 cpython-313"
    assert built.build("2.0") == ["link"] and built.module() == "2.0 cpython-312"


def test_a_module_of_unknown_origin_is_linked_anew(built, tmp_path):
    built.build("2.0")
    (tmp_path / "decode_binding.linked").unlink()
    assert built.build("2.0") == ["link"]
    os.remove(b.BINDING)
    assert built.build("2.0") == ["link"]


@pytest.mark.parametrize("missing", ["g++", "Python.h"])
def test_without_a_compiler_or_headers(built, monkeypatch, tmp_path, missing):
    """The library is built without the module; a module of another torch does not stay."""
    built.build("2.0")
    if missing == "g++":
        which = shutil.which
        monkeypatch.setattr(shutil, "which", lambda n: None if n == "g++" else which(n))
    else:
        monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert built.build("2.0") == [] and built.module() == "2.0 cpython-312"  # made earlier, still right
    with pytest.warns(RuntimeWarning, match="without the extension module"):
        assert built.build("2.1") == []
    assert not os.path.exists(b.BINDING)
