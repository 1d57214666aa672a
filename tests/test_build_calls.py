"""CPU: when the binding's native module is compiled again."""
import os
import subprocess

import pytest

from streaming_speaker_diarization_b200 import build


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """The compilations asked for, with the module and its record under tmp_path."""
    got = []

    def run(cmd, **_):
        got.append(cmd)
        (tmp_path / "_calls.so").write_text("module")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", run)
    return got


def test_once_for_each_torch_and_source(compiled, monkeypatch, tmp_path):
    build._build_calls()
    build._build_calls()
    assert len(compiled) == 1
    monkeypatch.setattr(build.metadata, "version", lambda name: "99.0")   # torch has been upgraded
    build._build_calls()
    build._build_calls()
    assert len(compiled) == 2
    os.utime(tmp_path / "_calls.so", (1, 1))                              # a source is newer
    build._build_calls()
    assert len(compiled) == 3
    (tmp_path / "calls.versions").unlink()                                # built before the versions were recorded
    build._build_calls()
    assert len(compiled) == 4


def test_a_failed_compilation_is_tried_again(compiled, monkeypatch):
    real = build.subprocess.run
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: subprocess.CompletedProcess(cmd, 1, "", "error"))
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build._build_calls()
    monkeypatch.setattr(build.subprocess, "run", real)
    build._build_calls()
    assert len(compiled) == 1
