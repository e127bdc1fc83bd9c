"""The build script, with a stand-in for the compiler."""
import os

import pytest

from weight_only_quantized_w8a16_amd import build


def stand_in(tmp_path, monkeypatch, text, status):
    exe = tmp_path / "hipcc"
    exe.write_text(f"#!/bin/sh\n{text}\nexit {status}\n")
    exe.chmod(0o755)
    monkeypatch.setattr(build, "HIPCC", str(exe))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))


def test_warnings_of_a_successful_compile_are_shown(tmp_path, monkeypatch, capsys):
    stand_in(tmp_path, monkeypatch, 'echo "mx4.hip:1:1: warning: something" >&2', 0)
    assert build._compile("mx4.hip") == os.path.join(str(tmp_path), "mx4.o")
    err = capsys.readouterr().err
    assert "mx4.hip:1:1: warning: something" in err


def test_a_quiet_compile_shows_nothing(tmp_path, monkeypatch, capsys):
    # nor one whose host pass ignores the device's feature
    note = "'-packed-fp32-ops' is not a recognized feature for this target (ignoring feature)"
    stand_in(tmp_path, monkeypatch, f'echo "{note}" >&2', 0)
    build._compile("mx4.hip")
    out = capsys.readouterr()
    assert out.out == "" and out.err == ""


def test_a_failed_compile_raises_with_its_messages(tmp_path, monkeypatch):
    stand_in(tmp_path, monkeypatch, 'echo "error: no" >&2', 1)
    with pytest.raises(RuntimeError, match="error: no"):
        build._compile("mx4.hip")
