"""CPU: the library builds without torch and without Python's calls, and a
failure of one part leaves no stale other part behind."""
import os
import shutil
import subprocess
import sys

import pytest

from block_scaled_moe_expert_gb300 import build as BLD


def test_the_library_builds_without_torch():
    """As a C user builds it: the file alone, on a machine without torch."""
    BLD.build()
    code = ("import sys, runpy; sys.modules['torch'] = None; sys.argv = ['build.py']; "
            f"runpy.run_path({BLD.__file__!r}, run_name='__main__')")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert BLD.LIB in r.stdout and "without Python's calls" in r.stdout


@pytest.fixture
def copy(tmp_path, monkeypatch):
    """The built parts in a folder of their own, and calls that do not compile."""
    BLD.build()
    shutil.copytree(BLD.BUILD, tmp_path / "_build")
    for name, path in (("LIB", BLD.LIB), ("CALLS", BLD.CALLS)):
        shutil.copy2(path, tmp_path)
        monkeypatch.setattr(BLD, name, str(tmp_path / os.path.basename(path)))
    monkeypatch.setattr(BLD, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(BLD, "_calls_command", lambda src: [sys.executable, "-c", "raise SystemExit(3)"])
    stamp = tmp_path / "_build" / "calls.torch"
    stamp.write_text("another")
    return stamp


def test_a_library_is_linked_where_only_the_calls_fail(copy):
    os.utime(os.path.join(BLD.BUILD, "sort.o"))  # newer than the library
    before = os.path.getmtime(BLD.LIB)
    with pytest.raises(RuntimeError):
        BLD.build()
    assert os.path.getmtime(BLD.LIB) > before


def test_a_library_older_than_its_objects_is_linked_again(copy, monkeypatch):
    monkeypatch.setattr(BLD, "_calls_command", lambda src: [sys.executable, "-c", f"open({BLD.CALLS!r}, 'w')"])
    BLD.build()
    os.utime(os.path.join(BLD.BUILD, "sort.o"))
    before = os.path.getmtime(BLD.LIB)
    BLD.build()
    assert os.path.getmtime(BLD.LIB) > before


def test_calls_of_another_torch_are_not_taken_for_this_ones(copy):
    """The stamp of a torch is written once its calls are there."""
    for _ in range(2):
        with pytest.raises(RuntimeError):
            BLD.build()
        assert not os.path.exists(BLD.CALLS) and (not copy.exists() or copy.read_text() == "another")
