"""The short native way of the binding is optional: the library's build succeeds without it, and leaves no module of
another torch or an older interface behind."""
import os

import pytest

from diffusion_transformer_denoiser_dit_b200 import build


@pytest.fixture
def stale(tmp_path, monkeypatch):
    """A module older than its sources at the place of _fastcall.so, a compiler that fails, and nothing else to build."""
    so, bin = tmp_path / "_fastcall.so", tmp_path / "bin"
    so.write_bytes(b"old")
    os.utime(so, (0, 0))
    bin.mkdir()
    gxx = bin / "g++"
    gxx.write_text("#!/bin/sh\necho no such torch >&2\nexit 1\n")
    gxx.chmod(0o755)
    monkeypatch.setenv("PATH", f"{bin}{os.pathsep}{os.environ['PATH']}")
    monkeypatch.setattr(build, "FASTCALL", str(so))
    monkeypatch.setattr(build, "sources", lambda: [])
    return so


def test_a_compiler_that_fails_only_warns(stale, capsys):
    assert build.build() == build.LIB
    assert not stale.exists()
    out = capsys.readouterr()
    assert "no such torch" in out.err and "_fastcall" in out.err


def test_without_torch_a_stale_module_goes(stale, monkeypatch):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build() == build.LIB
    assert not stale.exists()


def test_a_module_that_is_up_to_date_stays(stale):
    os.utime(stale, None)
    assert build.build() == build.LIB
    assert stale.read_bytes() == b"old"
