"""The dense layer in 8-bit floating point on the host: sizes and every refusal
before any device work, and the reference's coding against e4m3's own table.  No GPU
is touched: the pointers are small integers that are only looked at."""
import os

import pytest
import torch

import fp8_reference as R
import unet_x3_convolution_amd as U

P = 4096          # a 16-byte aligned non-null "address"


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not (os.path.exists(U.LIB_PATH) and os.path.exists(U.BINDING_PATH)):
        from unet_x3_convolution_amd import build
        build.build(verbose=False)
    U.lib()


def refused(code, fn, *args, **kw):
    with pytest.raises(U.OidnError) as e:
        fn(*args, **kw)
    assert e.value.code == code, e.value
    assert U.last_error()


def test_reference_rounds_to_the_nearest_code():
    """Every value between two neighbouring codes goes to the nearer one, ties to the even one, as a cast does."""
    v = torch.cat([torch.linspace(-448, 448, 20001), torch.linspace(-0.05, 0.05, 20001),
                   torch.ldexp(torch.arange(1, 512).float() / 16, torch.tensor(-9))]).double()
    assert torch.equal(R.rounded(v), v.float().to(torch.float8_e4m3fn).double())


@pytest.mark.parametrize("top, e", [(448.0, 0), (448.1, 1), (447.0, 0), (224.0, -1), (225.0, 0), (1.75, -8), (1.76, -7),
                                    (1.0, -8), (0.0, 0), (2.0 ** -130, -120), (3.38e38, 120)])
def test_reference_power(top, e):
    assert int(R.power(torch.tensor(top, dtype=torch.float64))) == e


@pytest.mark.parametrize("m, n", [(0, 1), (1, 1), (3, 128), (3, 129), (5, 512), (5, 513), (1000, 112), (1 << 20, 4096)])
def test_packed_bytes(m, n):
    blocks = -(-n // 128)
    assert U.oidn_fp8_bytes(m, n) == -(-m * (blocks * 128 + -(-blocks // 4) * 4) // 256) * 256


def test_packed_bytes_refusals():
    refused(U.OIDN_E_INVALID, U.oidn_fp8_bytes, -1, 4)
    refused(U.OIDN_E_INVALID, U.oidn_fp8_bytes, 4, 0)
    refused(U.OIDN_E_UNSUPPORTED, U.oidn_fp8_bytes, 4, (1 << 24) + 1)
    refused(U.OIDN_E_UNSUPPORTED, U.oidn_fp8_bytes, 1 << 31, 4)
    refused(U.OIDN_E_UNSUPPORTED, U.oidn_fp8_bytes, 1 << 30, 1 << 20)


def pack(**kw):
    a = dict(x=P, ldx=48, m=10, n=48, packed=P, packed_t=P, dtype=U.OIDN_F16, flags=0)
    a.update(kw)
    return U.oidn_fp8_pack(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=P + 1), dict(ldx=47), dict(m=-1), dict(n=0), dict(packed=None, packed_t=None),
    dict(packed=P + 8), dict(packed_t=P + 4), dict(dtype=3), dict(flags=1), dict(flags=8), dict(flags=16)], ids=str)
def test_pack_refuses(bad):
    refused(U.OIDN_E_INVALID, pack, **bad)


def test_pack_limits():
    refused(U.OIDN_E_UNSUPPORTED, pack, m=(1 << 24) + 1)
    refused(U.OIDN_E_UNSUPPORTED, pack, m=(1 << 31) - 1, packed_t=None, n=1)
    refused(U.OIDN_E_UNSUPPORTED, pack, ldx=(1 << 32) + 1)


@pytest.mark.parametrize("bad", [
    dict(packed=None), dict(packed=P + 8), dict(y=None), dict(y=P + 1), dict(ldy=47), dict(m=-1), dict(n=0),
    dict(dtype=7)], ids=str)
def test_unpack_refuses(bad):
    a = dict(packed=P, m=10, n=48, y=P, ldy=48, dtype=U.OIDN_F16)
    a.update(bad)
    refused(U.OIDN_E_INVALID, U.oidn_fp8_unpack, **a, stream=0)


def linear(**kw):
    a = dict(x=P, ldx=160, w8=P, bias=P, residual=P, ldr=48, y=P, ldy=48, z=P, ldz=48, m=100, k=160, n=48,
             act=U.OIDN_ACT_GELU, dtype=U.OIDN_F16, flags=0, workspace=P, ws_bytes=1 << 40)
    a.update(kw)
    return U.oidn_linear_fp8(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(w8=None), dict(y=None), dict(x=P + 1), dict(w8=P + 8), dict(y=P + 1), dict(residual=P + 1),
    dict(z=P + 1), dict(bias=P + 2), dict(ldx=159), dict(ldr=47), dict(ldy=47), dict(ldz=47), dict(m=-1), dict(k=0),
    dict(n=0), dict(act=4), dict(act=-1), dict(dtype=3), dict(flags=U.OIDN_X_CKPT8), dict(flags=U.OIDN_FP8_SQUARE),
    dict(flags=16), dict(flags=U.OIDN_Z_CKPT8, z=None), dict(flags=U.OIDN_X_FP8, x=P + 2), dict(workspace=None),
    dict(workspace=P + 8)], ids=str)
def test_linear_refuses(bad):
    refused(U.OIDN_E_INVALID, linear, **bad)


def test_linear_limits():
    refused(U.OIDN_E_UNSUPPORTED, linear, dtype=U.OIDN_F32)
    refused(U.OIDN_E_UNSUPPORTED, linear, k=(1 << 23) + 1, ldx=1 << 24)
    refused(U.OIDN_E_UNSUPPORTED, linear, n=(1 << 23) + 1, ldy=1 << 24, ldz=1 << 24, ldr=1 << 24)
    refused(U.OIDN_E_UNSUPPORTED, linear, m=1 << 31)
    # more tiles than a launch holds, 64 x 64 each
    refused(U.OIDN_E_UNSUPPORTED, linear, m=(1 << 30) + 1, flags=U.OIDN_X_FP8)
    refused(U.OIDN_E_UNSUPPORTED, U.oidn_linear_fp8_workspace_bytes, (1 << 30) + 1, 64, 48, U.OIDN_F16, U.OIDN_X_FP8)


def test_linear_workspace():
    need = U.oidn_linear_fp8_workspace_bytes(100, 160, 48, U.OIDN_F16, 0)
    assert need >= U.oidn_fp8_bytes(100, 160)
    refused(U.OIDN_E_WORKSPACE, linear, ws_bytes=need - 1)
    assert U.oidn_linear_fp8_workspace_bytes(100, 160, 48, U.OIDN_F16, U.OIDN_X_FP8) < need
    assert U.oidn_linear_fp8_workspace_bytes(0, 64, 48, U.OIDN_F16, 0) == 0
    refused(U.OIDN_E_INVALID, U.oidn_linear_fp8_workspace_bytes, 4, 0, 4, U.OIDN_F16, 0)
    refused(U.OIDN_E_INVALID, U.oidn_linear_fp8_workspace_bytes, 4, 4, 4, U.OIDN_F16, 4)
    refused(U.OIDN_E_UNSUPPORTED, U.oidn_linear_fp8_workspace_bytes, 4, 4, 4, U.OIDN_F32, 0)


def backward(**kw):
    a = dict(dy=P, lddy=48, x=P, ldx=64, z=P, ldz=48, w8t=P, dx=P, lddx=64, dw=P, lddw=64, dbias=P, m=10, k=64, n=48,
             act=U.OIDN_ACT_GELU, dtype=U.OIDN_BF16, flags=0, workspace=P, ws_bytes=1 << 40)
    a.update(kw)
    return U.oidn_linear_fp8_backward(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(x=None), dict(z=None), dict(w8t=None), dict(dy=P + 1), dict(w8t=P + 8), dict(dx=P + 1),
    dict(dw=P + 1), dict(dbias=P + 1), dict(lddy=47), dict(ldx=63), dict(ldz=47), dict(lddx=63), dict(lddw=63),
    dict(m=-1), dict(k=0), dict(n=0), dict(act=9), dict(dtype=-1), dict(flags=1), dict(flags=U.OIDN_FP8_SQUARE),
    dict(workspace=None), dict(flags=U.OIDN_X_FP8, x=P + 2), dict(flags=U.OIDN_Z_CKPT8, z=P + 2)], ids=str)
def test_backward_refuses(bad):
    refused(U.OIDN_E_INVALID, backward, **bad)


def test_backward_limits_and_workspace():
    refused(U.OIDN_E_UNSUPPORTED, backward, dtype=U.OIDN_F32)
    refused(U.OIDN_E_UNSUPPORTED, backward, m=(1 << 23) + 1)
    need = U.oidn_linear_fp8_backward_workspace_bytes(10, 64, 48, U.OIDN_ACT_GELU, U.OIDN_BF16, 0)
    refused(U.OIDN_E_WORKSPACE, backward, ws_bytes=need - 1)
    assert U.oidn_linear_fp8_backward_workspace_bytes(10, 64, 48, U.OIDN_ACT_GELU, U.OIDN_BF16, U.OIDN_X_FP8) < need
    refused(U.OIDN_E_INVALID, U.oidn_linear_fp8_backward_workspace_bytes, 10, 64, 48, 4, U.OIDN_F16, 0)


def test_no_rows_enqueue_nothing():
    pack(m=0, x=None, packed=None, packed_t=None)
    linear(m=0, x=None, y=None)
    U.oidn_fp8_unpack(None, 0, 4, None, 4, U.OIDN_F16, stream=0)
    backward(m=0, dw=None, dbias=None, dy=None, workspace=None)
