"""The build of the binding's extension."""
import os
import sys
import sysconfig

import pytest


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build module, its extension in a folder of its own."""
    from combine_movement_gb300 import build
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
