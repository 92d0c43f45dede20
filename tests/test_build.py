"""The build of the library and of the Python binding, without compilers."""
import os
import subprocess
import sys

import pytest

from nvfp4_mixture_experts_router_gb300 import build


def fake_tools(monkeypatch, tmp_path, fails):
    """The build in tmp_path with compilers that only write their output file."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        if fails(cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "no headers")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    for name, file in (("OUT", "lib.so"), ("BINDING", "binding.so"), ("BUILD_DIR", "objects")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build.subprocess, "run", run)
    return ran


@pytest.mark.parametrize("what", ["headers", "torch"])
def test_the_library_is_built_without_what_the_binding_needs(monkeypatch, tmp_path, what):
    fake_tools(monkeypatch, tmp_path, lambda cmd: what == "headers" and build.BINDING_SRC in cmd)
    if what == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.raises((RuntimeError, ImportError)):
        build.build()
    assert os.path.exists(build.OUT) and not os.path.exists(build.BINDING)


def test_a_failed_kernel_leaves_no_library(monkeypatch, tmp_path):
    fake_tools(monkeypatch, tmp_path, lambda cmd: any(c.endswith("layer_norm.cu") for c in cmd))
    with pytest.raises(RuntimeError, match="layer_norm"):
        build.build()
    assert not os.path.exists(build.OUT)
    ran = fake_tools(monkeypatch, tmp_path, lambda cmd: False)
    assert build.build() == build.OUT and os.path.exists(build.OUT) and os.path.exists(build.BINDING)
    assert len(ran) == len(build.sources()) + 3
