"""What the calls that convert their arguments in C++ take, and what they refuse."""
import enum

import pytest

import unet_x3_convolution_amd as U


class Address(enum.IntEnum):
    BUFFER = 4096


class Handle(int):
    pass


class Tensor:
    def data_ptr(self):
        return 8192


class Stream:
    cuda_stream = 77


def dropout(x=4096, m=0, n=8, p=0.5, rng=4096, dtype=U.OIDN_F16, stream=0):
    """No rows: nothing is enqueued, the arguments are only converted."""
    U.oidn_dropout(x, 8, None, 0, x, 8, m, n, p, rng, dtype, stream=stream)


def test_a_native_call_takes_them():
    for x in (4096, Address.BUFFER, Handle(4096), Tensor()):
        for stream in (0, Handle(0), False, Stream()):
            dropout(x, stream=stream)
    dropout(m=False, n=Handle(8), p=0)
    dropout(None)


@pytest.mark.parametrize("wrong, error", [({"n": 2 ** 31}, OverflowError), ({"m": 2 ** 63}, OverflowError),
                                          ({"n": 8.0}, TypeError), ({"p": "half"}, TypeError),
                                          ({"x": 4096.0}, AttributeError), ({"x": 2 ** 64}, OverflowError),
                                          ({"stream": Handle(-2 ** 64)}, OverflowError)])
def test_a_native_call_refuses_what_does_not_convert(wrong, error):
    """Nothing is cut to the parameter's bits."""
    with pytest.raises(error):
        dropout(**wrong)


def test_a_native_call_counts_its_arguments():
    with pytest.raises(TypeError, match="2 arguments given, 12 taken"):
        U._calls().oidn_dropout(4096, 8)


def test_native_calls_are_the_librarys():
    """The same last error, and the same answers, by either way."""
    args = (4096, 8, None, 0, 4096, 8, 0, 8, 2.0, 4096, U.OIDN_F16, 0)
    status = U._calls().oidn_dropout(*args)
    native = U.lib().oidn_last_error()
    assert status == U.lib().oidn_dropout(*args) == U.OIDN_E_INVALID
    assert native == U.lib().oidn_last_error() != b""


def residual(scale):
    U.oidn_norm_residual(4096, 8, None, None, None, 0, 0, 4096, 8, scale, 0.0, None, 4096, 8, None, None, None, 0, 0, 8,
                         U.OIDN_NORM_RMS, U.OIDN_NORM_NONE, 1e-5, U.OIDN_F16, stream=0)


@pytest.mark.parametrize("scale", [1e300, -1e300, 3.5e38, 2 ** 1000])
def test_a_native_call_refuses_floats_past_the_range(scale):
    """Finite numbers that would become infinities of float32."""
    with pytest.raises(OverflowError):
        residual(scale)


@pytest.mark.parametrize("scale", [1, True, 3.4028235e38, float("inf"), -float("inf"), float("nan"), 1e-300])
def test_a_native_call_takes_floats(scale):
    """The largest, infinities and NaN as they are; what is below the range is rounded, as every number is."""
    residual(scale)
