"""The build's bookkeeping: the Python extension belongs to one torch and one
interpreter, and the C library does not depend on it (CPU)."""
import os
import sysconfig

import pytest
import torch

from speculative_decoding_verify_split_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build_library(force=not all(os.path.exists(os.path.join(build.BUILD, f + ".o")) for f in build.SOURCES))


def test_another_torch_or_interpreter_makes_the_extension_stale(monkeypatch):
    assert not build.binding_stale()
    here = build.binding_abi()
    for part in torch.__version__, sysconfig.get_config_var("SOABI"):
        assert part in here
    monkeypatch.setattr(build, "binding_abi", lambda: here.replace(torch.__version__, "1.0"))
    assert build.binding_stale() and not build.library_stale()


def test_an_extension_without_a_stamp_is_stale(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "none"))
    assert build.binding_stale()


def test_the_library_is_linked_without_the_extension(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "_compile", lambda src, verbose: os.path.join(build.BUILD, src + ".o"))

    def no_headers(verbose):
        raise RuntimeError("no torch headers")

    monkeypatch.setattr(build, "_compile_binding", no_headers)
    for name in ("LIB", "BINDING", "BINDING_STAMP"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "LIBDIR", str(tmp_path))
    with pytest.raises(RuntimeError, match="no torch headers"):
        build.build_library()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING_STAMP)
