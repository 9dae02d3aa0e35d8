"""A tree without the C++ calls (built where Python's headers are missing, or by another
Python): the library is whole, and the same calls go through ctypes with the same checks."""
import os
import warnings

import pytest

import test_native_calls_cpu as calls
import unet_x3_convolution_amd as U
from unet_x3_convolution_amd import build


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(U.LIB_PATH):
        build.build(verbose=False)
    elif not os.path.exists(U.BINDING_PATH):
        build._binding()


@pytest.fixture
def absent(monkeypatch, tmp_path):
    U.lib()
    monkeypatch.setattr(U, "_native", None)
    monkeypatch.setattr(U, "BINDING_PATH", str(tmp_path / "none.so"))
    with pytest.warns(RuntimeWarning, match="none.so is not built"):
        U._calls()


def test_binding_is_of_this_python():
    """Another Python does not find it in place of its own."""
    from importlib.machinery import EXTENSION_SUFFIXES
    assert U.BINDING_PATH == build.BINDING and U.BINDING_PATH.endswith("_binding" + EXTENSION_SUFFIXES[0])
    assert EXTENSION_SUFFIXES[0] != ".so"


def test_build_without_headers(monkeypatch, tmp_path, capfd):
    """Said, and no error: nothing is built, and what an earlier build left is taken away."""
    old = tmp_path / "old.so"
    old.write_bytes(b"")
    monkeypatch.setattr(build, "PYTHON_INCLUDE", str(tmp_path))
    monkeypatch.setattr(build, "BINDING", str(old))
    build._binding()
    assert "Python.h" in capfd.readouterr().err and not old.exists()


def test_build_needs_one_compiler():
    """The one that the library is built with."""
    assert not hasattr(build, "CXX")


def test_a_failing_build_is_an_error(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    with pytest.raises(RuntimeError, match="binding"):
        build._binding()


def test_the_choice_is_made_once(absent):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert U._calls() is U._calls()


def test_calls(absent):
    calls.test_a_native_call_takes_them()
    calls.test_native_calls_are_the_librarys()
    calls.test_a_native_call_counts_its_arguments()


@pytest.mark.parametrize("wrong, error", [({"n": 2 ** 31}, OverflowError), ({"m": 2 ** 63}, OverflowError),
                                          ({"n": 8.0}, TypeError), ({"p": "half"}, TypeError),
                                          ({"x": 4096.0}, AttributeError), ({"x": 2 ** 64}, OverflowError),
                                          ({"stream": calls.Handle(-2 ** 64)}, OverflowError)])
def test_refusals(absent, wrong, error):
    with pytest.raises(error):
        calls.dropout(**wrong)


@pytest.mark.parametrize("scale", [1e300, -1e300, 3.5e38, 2 ** 1000])
def test_floats_past_the_range(absent, scale):
    with pytest.raises(OverflowError):
        calls.residual(scale)


@pytest.mark.parametrize("scale", [1, True, 3.4028235e38, float("inf"), -float("inf"), float("nan"), 1e-300])
def test_floats(absent, scale):
    calls.residual(scale)


def test_unsigned_and_sizes(absent):
    for bad in (-1, 2 ** 32):
        with pytest.raises(OverflowError):
            U.oidn_fp8_pack(4096, 8, 0, 8, 4096, None, U.OIDN_F16, bad, stream=0)
    for bad in (-1, 2 ** 64):
        with pytest.raises(OverflowError):
            U.oidn_norm_backward(None, 8, None, 8, None, None, 0, None, 8, None, None, 0, 8, U.OIDN_NORM_RMS, 1e-5,
                                 U.OIDN_F16, None, bad, stream=0)


def test_both_ways_refuse_alike():
    """The same wrong numbers by the C++ calls, where they are built."""
    if not os.path.exists(U.BINDING_PATH):
        pytest.skip("Python's headers are missing")
    test_unsigned_and_sizes(None)
