"""CPU checks of the build: what is rebuilt when, and what is left when a part fails.  The
compilers are stand-ins that write their output file and keep a record of each call."""
import os
import stat

import pytest

import quantized_paged_kv_q8_gb300 as k8
from quantized_paged_kv_q8_gb300 import buildlib

STUB = """#!/bin/sh
echo call >> "{log}"
if [ -e "{log}.fail" ]; then echo "Python.h: No such file" >&2; exit 1; fi
while [ $# -gt 0 ]; do if [ "$1" = "-o" ]; then echo built > "$2"; fi; shift; done
"""


class Tools:
    def __init__(self, where):
        self.where = where
        for name in ("nvcc", "g++"):
            path = os.path.join(where, name)
            with open(path, "w") as f:
                f.write(STUB.format(log=os.path.join(where, name + ".log")))
            os.chmod(path, os.stat(path).st_mode | stat.S_IXUSR)

    def calls(self, name):
        """Calls since the last time this was asked."""
        log = os.path.join(self.where, name + ".log")
        if not os.path.exists(log):
            return 0
        with open(log) as f:
            n = len(f.readlines())
        os.remove(log)
        return n

    def fail(self, name, on):
        mark = os.path.join(self.where, name + ".log.fail")
        if on:
            open(mark, "w").close()
        else:
            os.remove(mark)


@pytest.fixture
def tools(tmp_path, monkeypatch):
    os.makedirs(tmp_path / "bin")
    t = Tools(str(tmp_path / "bin"))
    monkeypatch.setenv("PATH", t.where + os.pathsep + os.environ["PATH"])
    build = str(tmp_path / "_build")
    for name in ("LIB", "BINDING", "BINDING_ERROR"):
        if hasattr(buildlib, name):
            monkeypatch.setattr(buildlib, name, os.path.join(build, os.path.basename(getattr(buildlib, name))))
    monkeypatch.setattr(buildlib, "BUILD", build)
    return t


def test_builds_once(tools):
    assert buildlib.build() == buildlib.LIB
    assert os.path.exists(buildlib.LIB) and os.path.exists(buildlib.BINDING)
    assert tools.calls("nvcc") == len(buildlib.SOURCES) + 1 and tools.calls("g++") == 1
    buildlib.build()
    assert tools.calls("nvcc") == 0 and tools.calls("g++") == 0


def test_the_library_does_not_need_the_extension_module(tools, monkeypatch):
    """Without Python's headers: the C library is built, a warning tells, and the calls that need the module say why."""
    buildlib.build()
    tools.calls("nvcc"), tools.calls("g++")
    os.remove(buildlib.LIB)
    os.utime(buildlib.BINDING, (1, 1))                     # of older sources
    tools.fail("g++", True)
    with pytest.warns(UserWarning, match="Python.h"):
        assert buildlib.build() == buildlib.LIB
    assert os.path.exists(buildlib.LIB) and not os.path.exists(buildlib.BINDING)
    monkeypatch.setattr(k8, "_binding", None)
    monkeypatch.setattr(k8, "lib", lambda: None)
    with pytest.raises(RuntimeError, match="Python.h"):
        k8.spec_accept_k8v4(None, None, None, None, None, None, None)
    # tried again each time, the library left as it is
    tools.calls("nvcc"), tools.calls("g++")
    with pytest.warns(UserWarning, match="Python.h"):
        buildlib.build()
    assert tools.calls("nvcc") == 0 and tools.calls("g++") == 1
    tools.fail("g++", False)
    buildlib.build()
    assert os.path.exists(buildlib.BINDING) and not os.path.exists(buildlib.BINDING_ERROR) and tools.calls("nvcc") == 0


def test_a_library_that_does_not_compile_is_an_error(tools):
    tools.fail("nvcc", True)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        buildlib.build()
    assert not os.path.exists(buildlib.LIB)


def test_the_extension_module_follows_torch_and_python(tools, monkeypatch):
    """A module built against another torch or Python is not taken: their C++ symbols differ."""
    import sysconfig

    import torch
    buildlib.build()
    tools.calls("nvcc"), tools.calls("g++")
    monkeypatch.setattr(torch, "__version__", "9.8.7+other")
    buildlib.build()
    assert tools.calls("nvcc") == 0 and tools.calls("g++") == 1
    buildlib.build()
    assert tools.calls("g++") == 0
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-999" if name == "SOABI" else real(name))
    buildlib.build()
    assert tools.calls("nvcc") == 0 and tools.calls("g++") == 1
    # not built for this pair, and not to be loaded for it
    monkeypatch.setattr(torch, "__version__", "9.8.8")
    monkeypatch.setattr(k8, "_binding", None)
    monkeypatch.setattr(k8, "lib", lambda: None)
    with pytest.raises(RuntimeError, match="not built"):
        k8.spec_accept_k8v4(None, None, None, None, None, None, None)
