"""When the build compiles, and what it leaves behind when that fails (no compiler runs here)."""
import os

import pytest
import torch

from scaled_quantize_gemm_amax_gb300 import build as fqbuild


class Process:
    """A compiler that writes its output file, or fails."""
    def __init__(self, cmd, code, started):
        self.cmd, self.returncode, self.waited, self.stopped = cmd, code, False, False
        out = cmd[cmd.index("-o") + 1]
        if code == 0 or "_rowops" in out:
            with open(out, "w") as f:
                f.write("x")
        started.append(self)

    def communicate(self):
        self.waited = True
        return "", None

    def wait(self, timeout=None):
        self.waited = True
        return self.returncode

    def poll(self):
        return self.returncode if self.waited else None

    def kill(self):
        self.stopped = True

    terminate = kill


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build with its outputs in a folder of their own; returns the list of compilers it starts."""
    started = []
    for name in ("LIB", "LIB_DEBUG", "BUILD", "BUILD_DEBUG", "EXT"):
        monkeypatch.setattr(fqbuild, name, str(tmp_path / os.path.basename(getattr(fqbuild, name))))
    codes = {"g++": 0, "nvcc": 0}

    def popen(cmd, **kw):
        return Process(cmd, codes["g++" if cmd[0] == "g++" else "nvcc"], started)

    def run(cmd, **kw):
        Process(cmd, 0, [])

    monkeypatch.setattr(fqbuild.subprocess, "Popen", popen)
    monkeypatch.setattr(fqbuild.subprocess, "run", run)
    return started, codes, tmp_path


def extension_builds(started):
    n = sum(p.cmd[0] == "g++" for p in started)
    started.clear()
    return n


def test_the_extension_is_built_again_for_another_torch(tree, monkeypatch):
    started, _, _ = tree
    fqbuild.build()
    assert extension_builds(started) == 1
    fqbuild.build()
    assert extension_builds(started) == 0
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    fqbuild.build()
    assert extension_builds(started) == 1
    fqbuild.build()
    assert extension_builds(started) == 0


@pytest.mark.parametrize("debug", [False, True])
def test_a_failed_build_leaves_no_compiler_and_no_temporary_file(tree, debug):
    started, codes, folder = tree
    codes["nvcc"] = 1
    with pytest.raises(RuntimeError, match="nvcc failed"):
        fqbuild.build(debug=debug)
    assert started and all(p.waited for p in started)
    assert not [f for f in os.listdir(folder) if ".tmp" in f]


def test_a_failed_extension_leaves_no_temporary_file(tree):
    started, codes, folder = tree
    codes["g++"] = 1
    with pytest.raises(RuntimeError, match="g.. failed"):
        fqbuild.build()
    assert not [f for f in os.listdir(folder) if ".tmp" in f]
    assert not os.path.exists(fqbuild.EXT)
