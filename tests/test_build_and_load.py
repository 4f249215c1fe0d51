"""The two compiled files of the package are independent: what libgdn2.so serves by itself needs no binding
module, in building and in loading. Everything here runs without a GPU."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "gated_delta_rule_160_b200"


@pytest.fixture(scope="module")
def build():
    from gated_delta_rule_160_b200 import build
    build.build()
    return build


def _copy(tmp_path):
    """The package with libgdn2.so, but without a binding module."""
    to = tmp_path / PACKAGE
    shutil.copytree(os.path.join(ROOT, PACKAGE), to, ignore=shutil.ignore_patterns("__pycache__", "csrc", "_binding*"))
    return to


def _run(where, code):
    return subprocess.run([sys.executable, "-c", code], cwd=where, capture_output=True, text=True, timeout=300,
                          env={**os.environ, "PYTHONPATH": str(where)})


LOADS = f"""
import torch
import {PACKAGE} as g
assert g.__file__.startswith({{where!r}}), g.__file__
assert g.load_library().gdn2_version() >= 210
x = torch.zeros(1, 1, 64)
try:
    g.gdn2_decode_step(x, x, x, x, x, x, torch.zeros(1, 1, 64, 64))
except ValueError as e:  # the check of its own arguments
    assert 'must be a CUDA tensor' in str(e), e
else:
    raise AssertionError('host tensors taken')
for call in (lambda: g.gdn2_state_load(x, x), lambda: g.gdn2_verify_drafts(x, x, x, x, x)):
    try:
        call()
    except ImportError as e:
        assert 'python -m {PACKAGE}.build' in str(e), e
    else:
        raise AssertionError('called without a binding')
print('fine')
"""


@pytest.mark.parametrize("damaged", [False, True])
def test_older_functions_work_without_the_binding(build, tmp_path, damaged):
    """Missing or not loadable: prefill, decode and backward still reach libgdn2.so; the serving operators raise, and
    say what to run."""
    to = _copy(tmp_path)
    if damaged:
        (to / os.path.basename(build.BINDING)).write_bytes(b"not a library")
    r = _run(tmp_path, LOADS.format(where=str(tmp_path)))
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]


def test_library_is_built_before_the_binding(build, tmp_path, monkeypatch):
    """A torch that the binding cannot be compiled against still gets libgdn2.so, and the failure is raised."""
    commands = []

    def compiler(cmd, **kw):
        commands.append(cmd[0])
        if cmd[0] == "g++":
            raise subprocess.CalledProcessError(1, cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgdn2.so"))
    monkeypatch.setattr(build.subprocess, "run", compiler)
    with pytest.raises(subprocess.CalledProcessError):
        build.build(force=True)
    assert os.path.exists(build.LIB) and commands == [build.nvcc(), "g++"]


def test_binding_belongs_to_one_torch_and_python(build, monkeypatch):
    """The module inlines torch's and Python's object layouts: another version of either has another file, and an
    existing file of the old one is not taken for it."""
    import sysconfig

    import torch
    here = build.binding_path()
    assert here == build.BINDING and os.path.exists(here) and os.path.dirname(here) == build.HERE
    seen = {here}
    soabi = sysconfig.get_config_var("SOABI")
    for change in (lambda m: m.setattr(torch, "__version__", "99.1.0+cu1"), lambda m: m.setattr(torch.version, "git_version", "0" * 40),
                   lambda m: m.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI),
                   lambda m: m.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-x" if name == "SOABI" else None)):
        with monkeypatch.context() as m:
            change(m)
            path = build.binding_path()
            assert path not in seen and not os.path.exists(path)
            seen.add(path)
            commands = []
            m.setattr(build.subprocess, "run", lambda cmd, **kw: (commands.append(cmd), open(cmd[cmd.index("-o") + 1], "w").close()))
            m.setattr(build.os, "replace", lambda a, b: (os.remove(a), commands.append(b)))
            assert build.build_binding() == path and len(commands) == 2 and commands[1] == path
    assert sysconfig.get_config_var("SOABI") == soabi and build.binding_path() == here


def test_binding_is_rebuilt_when_its_command_may_have_changed(build, monkeypatch):
    """The flags stand in build.py: a newer one builds again."""
    commands = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: commands.append(cmd))
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    build.build_binding()
    assert not commands
    newer = os.path.getmtime(build.BINDING) + 10
    real = os.path.getmtime
    monkeypatch.setattr(build.os.path, "getmtime", lambda p: newer if os.path.basename(p) == "build.py" else real(p))
    build.build_binding()
    assert len(commands) == 1


def test_a_binding_of_another_torch_is_not_loaded(build, tmp_path):
    to = _copy(tmp_path)
    shutil.copy(build.BINDING, to / os.path.basename(build.BINDING).replace("torch", "torch-0.0.0-"))
    r = _run(tmp_path, LOADS.format(where=str(tmp_path)))
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]
