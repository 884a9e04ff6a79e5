"""The compiled torch binding is built again whenever what it was built against changes: its
sources, torch, Python's ABI, or the compile command."""
import os
import sysconfig

import pytest
import torch

from decode_attention_int8_b200 import build


@pytest.fixture
def builds(tmp_path, monkeypatch):
    """Counts the compilations of a binding in an empty folder."""
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_q8kv_torch.so"))
    made = []

    def compiler(command):
        out = command[command.index("-o") + 1]
        open(out, "w").close()
        made.append(command)

    monkeypatch.setattr(build.subprocess, "check_call", compiler)
    assert build.build_binding() == build.BINDING and len(made) == 1
    build.build_binding()
    assert len(made) == 1  # current
    return made


def test_another_torch(builds, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "2.99.0")
    build.build_binding()
    assert len(builds) == 2
    build.build_binding()
    assert len(builds) == 2


def test_another_abi_of_torch(builds, monkeypatch):
    monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    build.build_binding()
    assert len(builds) == 2


def test_another_python(builds, monkeypatch):
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var",
                        lambda n: ".cpython-399.so" if n == "EXT_SUFFIX" else real(n))
    build.build_binding()
    assert len(builds) == 2


def test_a_binding_of_unknown_origin(builds):
    """A module without a record of what it was built against."""
    for name in os.listdir(os.path.dirname(build.BINDING)):
        if os.path.join(os.path.dirname(build.BINDING), name) != build.BINDING:
            os.remove(os.path.join(os.path.dirname(build.BINDING), name))
    build.build_binding()
    assert len(builds) == 2


def test_newer_sources(builds):
    later = max(os.path.getmtime(build.BINDING_SRC), os.path.getmtime(build.BINDING)) - 1e6
    os.utime(build.BINDING, (later, later))
    build.build_binding()
    assert len(builds) == 2
