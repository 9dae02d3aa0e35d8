"""What the binding takes as a device address and as a stream."""
import enum

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


def test_addresses():
    assert U._p(None) is None
    assert U._p(4096) == U._p(Address.BUFFER) == U._p(Handle(4096)) == 4096
    assert U._p(Tensor()) == 8192


def test_streams():
    assert U._s(0) == U._s(Handle(0)) == U._s(False) == 0
    assert U._s(Handle(4096)) == U._s(Address.BUFFER) == 4096
    assert U._s(Stream()) == 77


def test_a_call_takes_them():
    """No rows: nothing is enqueued, the arguments are only converted."""
    U.oidn_ckpt_pack(Address.BUFFER, 4, 0, 4, Handle(4096), U.OIDN_F16, stream=Handle(0))
