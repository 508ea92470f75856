"""The block-scaled FP8 layer's limits, and what its build and binding decide
without a GPU."""

import ctypes
import importlib.metadata
import importlib.util
from types import SimpleNamespace

import pytest

import rotation_bit_ptq_b200 as rbq
from rotation_bit_ptq_b200 import build

FAKE = ctypes.c_void_p(0x10000)                  # never dereferenced
BF, NONE, GELU = rbq.RBQ_BF16, rbq.RBQ_ACT_NONE, rbq.RBQ_ACT_GELU
MOST = 1 << 30


@pytest.fixture(scope="module")
def lib():
    return rbq.lib()


# ---- sizes: no count of blocks leaves 32 bits ---------------------------------------

# the first above the limit, and those whose number of blocks of 128 would wrap
@pytest.mark.parametrize("n", [MOST + 16, (1 << 31) - 128, (1 << 31) - 112, (1 << 31) - 16])
def test_widths_above_the_limit_are_refused(lib, n):
    for rc in (lib.quantize_fp8(FAKE, BF, 1, n, NONE, FAKE, FAKE, None, None, None),
               lib.quantize_fp8(FAKE, BF, 0, n, GELU, FAKE, FAKE, FAKE, FAKE, None),
               lib.quantize_weights_fp8(FAKE, BF, 16, n, FAKE, FAKE, None, None, None),
               lib.quantize_weights_fp8(FAKE, BF, n, 16, FAKE, FAKE, FAKE, FAKE, None),
               lib.qlinear_fp8(FAKE, FAKE, FAKE, FAKE, 1, 8, n, FAKE, None),
               lib.qlinear_fp8(FAKE, FAKE, FAKE, FAKE, 0, 8, n, FAKE, None),
               lib.qlinear_fp8_wgrad(FAKE, FAKE, FAKE, 1, 8, n, FAKE, BF, None),
               lib.gelu_backward_fp8(FAKE, FAKE, FAKE, 1, n, FAKE, None, None, None)):
        assert rc == rbq.RBQ_EINVAL


def test_the_limit_itself_is_allowed(lib):
    """(No rows, so that nothing is launched.)"""
    assert lib.quantize_fp8(None, BF, 0, MOST, NONE, None, None, None, None, None) == rbq.RBQ_OK
    assert lib.quantize_weights_fp8(None, BF, 0, MOST, None, None, None, None, None) == rbq.RBQ_OK
    assert lib.qlinear_fp8(None, None, None, None, 0, MOST, MOST, None, None) == rbq.RBQ_OK
    assert lib.qlinear_fp8_wgrad(None, None, None, MOST, 0, MOST, None, BF, None) == rbq.RBQ_OK
    assert lib.gelu_backward_fp8(None, None, None, 0, MOST, None, None, None, None) == rbq.RBQ_OK


# ---- the native binding's build -----------------------------------------------------

@pytest.fixture
def compiles(monkeypatch, tmp_path):
    """build_binding with files of its own and a compiler that only writes the output; the calls made."""
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_rbq_call.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", run)
    return calls


def test_binding_is_built_again_for_another_torch(compiles, monkeypatch):
    build.build_binding()
    build.build_binding()
    assert len(compiles) == 1                              # up to date
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "9.9.9" if name == "torch" else version(name))
    build.build_binding()
    build.build_binding()
    assert len(compiles) == 2


def test_binding_of_another_torch_is_refused(monkeypatch):
    """A library that loads but was built for another torch, whose objects may be
    laid out differently, is not called."""
    from rotation_bit_ptq_b200 import _fp8
    monkeypatch.setattr(_fp8, "_native", None)
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "9.9.9" if name == "torch" else version(name))
    with pytest.raises(RuntimeError, match="9.9.9"):
        _fp8._ordinary()
    assert _fp8._native is None


def test_the_library_is_built_without_torch(compiles, monkeypatch, capsys):
    """librbq.so needs no torch, so the build ends well where there is none; what is left out is said."""
    find_spec = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find_spec(name, *a))
    assert build.build_binding() is None
    assert compiles == [] and "torch" in capsys.readouterr().err
