"""The parts of the build: libnt.so needs no torch, and nt_calls.so goes with one torch and one Python (CPU; nvcc)."""
import importlib.util
import os

import pytest

from block_quantized_gemv_nt_gb300 import build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build folder of its own, with one small source in the library's place."""
    src, out = tmp_path / "csrc", tmp_path / "out"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "CSRC", str(src))
    monkeypatch.setattr(build, "BUILD", str(out))
    monkeypatch.setattr(build, "SO", str(out / "libnt.so"))
    return monkeypatch


def _no_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_the_library_is_built_without_torch(elsewhere):
    _no_torch(elsewhere)
    assert build.build() == build.SO and os.path.exists(build.SO)
    assert sorted(os.listdir(build.BUILD)) == ["libnt.so", "one.o"]
    built = os.path.getmtime(build.SO)
    assert build.build() == build.SO and os.path.getmtime(build.SO) == built      # nothing to do


def test_the_library_stands_when_the_module_does_not_compile(elsewhere, tmp_path):
    pytest.importorskip("torch")
    bad = tmp_path / "calls.cpp"
    bad.write_text("#error no module\n")
    elsewhere.setattr(build, "CALLS_SRC", str(bad))
    with pytest.raises(RuntimeError, match="calls.cpp"):
        build.build()
    assert os.path.exists(build.SO)


def test_the_module_is_of_one_torch_and_one_python(monkeypatch):
    """nt_calls.so holds torch's inlined accessors and Python's ABI: another version of either has another file."""
    import sysconfig

    torch = pytest.importorskip("torch")
    here = build.calls_so()
    assert torch.__version__ in os.path.basename(here) and sysconfig.get_config_var("EXT_SUFFIX") in here
    build.build()
    assert os.path.exists(here) and not build._calls_stale()
    with monkeypatch.context() as m:
        m.setattr(build, "_torch_version", lambda: "0.0.1")
        assert build.calls_so() != here and build._calls_stale()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".cpython-399-other.so")
        assert build.calls_so() != here and build._calls_stale()


def test_only_the_calls_that_need_the_module_load_it():
    """The model step's and the 8-bit cache's users import the engine without nt_calls.so."""
    import subprocess
    import sys

    from conftest import ROOT

    pytest.importorskip("torch")
    program = """
from block_quantized_gemv_nt_gb300 import nt
def none():
    raise OSError("no module here")
nt.load_calls = none
from block_quantized_gemv_nt_gb300 import engine
engine.KV8Cache(None, nt.KV8_I8, 1, 64, 64, device="cpu")
for make in (lambda: engine.KV4Cache(None, nt.KV4_I4, 1, 64, 1, device="cpu"),
             lambda: engine.KV4Pages(None, 1, 1, 1, device="cpu"), lambda: engine.Rope(None, 64)):
    try:
        make()
    except OSError as e:
        assert "no module here" in str(e)
    else:
        raise SystemExit("loaded without the module")
"""
    r = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
