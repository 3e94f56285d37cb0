"""The package without its C++ binding module: it imports, says so, and its
calls take the Python path; the build makes the module for the torch at hand
and does without it where it cannot."""
import os
import subprocess
import sys
import types

import pytest

from hybrid_mamba_ssm_b200 import build as ssm_build

NAME = "hybrid_mamba_ssm_b200._marshal"
USE = """
import torch, warnings
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    from hybrid_mamba_ssm_b200 import ssm, ssd_chunk_scan, selective_scan_fwd
    assert any("_marshal.so is not used" in str(m.message) for m in w), [str(m.message) for m in w]
assert ssm.selective_scan_saved_size(1, 4096, 64, 16) > 0
t = torch.zeros(4, 8)
calls = [lambda: selective_scan_fwd(t, t, t, t, t), lambda: ssm.selective_scan_bwd(t, t, t, t, t, t, t),
         lambda: ssm.selective_state_update(t, t, t, t, t, t), lambda: ssm.causal_conv1d_bwd(t[None], t[None], t),
         lambda: ssm.ssm_pool_copy(t, t, t), lambda: ssm.ssm_pool_zero(t, t), lambda: ssm.ssm_pool_compact(t, t),
         lambda: ssd_chunk_scan(t, t, t, t, t)]
for f in calls:
    try:
        f()
    except ValueError:
        continue
    raise AssertionError("a CPU tensor was taken")
"""


@pytest.fixture(scope="module")
def built():
    return ssm_build.build()


def run(code):
    p = subprocess.run([sys.executable, "-c", code], cwd=ssm_build.ROOT, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr


def test_imports_without_the_module(built):
    run(f"import sys; sys.modules[{NAME!r}] = None" + USE)


@pytest.mark.parametrize("version", ["'0.1'", "None"])
def test_a_module_of_another_torch_is_not_used(built, version):
    run(f"""
import sys, types
m = types.ModuleType({NAME!r})
if {version}: m.torch_version = {version}
def fail(*a): raise AssertionError("called")
m.scan_fwd = m.scan_bwd = m.state_update = m.conv1d_bwd = m.pool_copy = m.pool_zero = m.pool_compact = fail
import hybrid_mamba_ssm_b200
sys.modules[{NAME!r}] = hybrid_mamba_ssm_b200._marshal = m
""" + USE)


def test_the_built_module_is_used(built):
    import torch
    from hybrid_mamba_ssm_b200 import ssm
    assert isinstance(ssm._marshal, types.ModuleType) and ssm._marshal.torch_version == str(torch.__version__)


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The module's build with its outputs in a folder of the test and a recorder for a compiler."""
    calls = []

    def compile_(cmd, **kw):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(ssm_build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(ssm_build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(ssm_build.subprocess, "check_call", compile_)
    return calls


def test_module_is_rebuilt_for_another_torch(elsewhere, monkeypatch):
    import torch
    ssm_build.build_marshal()
    ssm_build.build_marshal()
    assert len(elsewhere) == 1                              # up to date
    monkeypatch.setattr(torch, "__version__", "0.1+other")
    ssm_build.build_marshal()
    assert len(elsewhere) == 2 and any("0.1+other" in a for a in elsewhere[1])


def test_build_goes_on_without_a_compiler_for_the_module(elsewhere, monkeypatch):
    def fail(cmd, **kw):
        raise subprocess.CalledProcessError(1, cmd)
    open(ssm_build.MARSHAL, "w").close()                    # of an earlier build
    monkeypatch.setattr(ssm_build, "sources", lambda: [])
    monkeypatch.setattr(ssm_build, "_stale", lambda target, deps: target == ssm_build.MARSHAL)
    monkeypatch.setattr(ssm_build.subprocess, "check_call", fail)
    with pytest.warns(RuntimeWarning, match="could not be built"):
        assert ssm_build.build() == ssm_build.LIB
    assert not os.path.exists(ssm_build.MARSHAL)
