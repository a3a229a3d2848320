"""The build of the binding's extension."""
import concurrent.futures
import os
import subprocess
import sys
import sysconfig
import threading
import time
import types

import pytest


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build module, its extension in a folder of its own."""
    from combine_movement_gb300 import build
    build.build()
    monkeypatch.setattr(build, "CALLS_PATH", str(tmp_path / os.path.basename(build.CALLS_PATH)))
    return build


def test_the_file_is_this_interpreters(build):
    from combine_movement_gb300 import ep
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert f"{sys.version_info.major}{sys.version_info.minor}" in suffix
    assert os.path.basename(build.CALLS_PATH) == "_calls" + suffix
    assert ep._calls.__file__ == os.path.join(build.PKG, "_calls" + suffix)


def test_another_interpreters_is_not_taken_for_it(build, tmp_path):
    for name in ("_calls.so", "_calls.cpython-30-any.so"):
        (tmp_path / name).write_bytes(b"of another interpreter")
    path = build.build_calls()
    assert path == build.CALLS_PATH and os.path.getsize(path) > 1000
    assert not (tmp_path / "_calls.so").exists()  # which this one would load too
    assert (tmp_path / "_calls.cpython-30-any.so").exists()
    before = os.path.getmtime(path)
    assert build.build_calls() == path and os.path.getmtime(path) == before


@pytest.fixture
def slow_compilers(build, monkeypatch, tmp_path):
    """Compilers that write their output in two parts; gives the outputs that two of
    them wrote at once."""
    busy, lock, clashes = set(), threading.Lock(), []

    def run(cmd, **kind):
        out = cmd[cmd.index("-o") + 1]
        with lock:
            if out in busy:
                clashes.append(out)
            busy.add(out)
        with open(out, "wb") as f:
            f.write(b"one ")
            f.flush()
            time.sleep(0.05)
            f.write(b"two")
        with lock:
            busy.discard(out)
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "OBJ_DIR", str(tmp_path / "_objs"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libep_gb300.so"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return clashes


@pytest.mark.parametrize("call", ["build_calls", "build"])
def test_two_builds_at_once(build, slow_compilers, call):
    with concurrent.futures.ThreadPoolExecutor(3) as ex:
        paths = list(ex.map(lambda _: getattr(build, call)(), range(3)))
    assert not slow_compilers
    for path in paths:
        with open(path, "rb") as f:
            assert f.read() == b"one two"


def test_of_those_that_waited_only_one_compiles(build, slow_compilers, monkeypatch):
    runs, inner = [], build.subprocess.run
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kind: (runs.append(cmd), inner(cmd, **kind))[1])
    with concurrent.futures.ThreadPoolExecutor(4) as ex:
        list(ex.map(lambda _: build.build(), range(4)))
    assert len(runs) == len(build.sources()) + 2  # each source, the library, the extension


def test_nothing_is_written_where_nothing_is_to_be_built(build, slow_compilers, monkeypatch):
    build.build()
    monkeypatch.setattr(build, "OBJ_DIR", os.path.join(build.OBJ_DIR, "not", "there"))
    monkeypatch.setattr(build.os, "makedirs", lambda *a, **k: pytest.fail("a folder was made"))
    assert build.build() == build.LIB_PATH and build.build_calls() == build.CALLS_PATH


def test_without_the_headers_the_library_is_built(build, slow_compilers, monkeypatch, tmp_path):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    with pytest.warns(UserWarning, match="Python.h"):
        assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.CALLS_PATH)


def test_a_broken_extension_does_not_keep_the_library_back(build, slow_compilers, monkeypatch):
    inner = build.subprocess.run
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kind: inner(cmd, **kind) if "nvcc" in cmd[0]
                        else types.SimpleNamespace(returncode=1, stdout="", stderr="broken"))
    with pytest.raises(RuntimeError, match="broken"):
        build.build()
    assert os.path.exists(build.LIB_PATH)


WITHOUT = """
import sys
sys.modules["combine_movement_gb300._calls"] = None  # an import of it fails
import torch
from combine_movement_gb300 import ep, moe
z = torch.zeros
try:
    ep.ep_dispatch(z(4, 8, dtype=torch.bfloat16), z(4, 2, dtype=torch.int32), z(8, 8, dtype=torch.bfloat16))
except ValueError as e:  # what it says of tensors that are not on a GPU
    print("movement:", e)
for call in (lambda: ep.ep_linear(z(4, 8), z(8, 8), z(4, 8)), lambda: moe.route(z(4, 8), 2)):
    try:
        call()
    except ImportError as e:
        print("needs it:", e)
"""


def test_without_the_extension_the_movement_is_there(build):
    r = subprocess.run([sys.executable, "-c", WITHOUT], capture_output=True, text=True, cwd=build.ROOT)
    lines = r.stdout.splitlines()
    assert r.returncode == 0, r.stderr
    assert lines[0].startswith("movement:") and "CUDA" in lines[0]
    assert [l.startswith("needs it:") and "not built" in l for l in lines[1:]] == [True, True]
