"""The dense operators' C ABI on the host: sizes of checkpoints and
workspaces, and every refusal, before any device work.  No GPU is touched:
the pointers are small integers that are only looked at."""
import os

import pytest

import unet_x3_convolution_amd as U

P = 4096          # a 16-byte aligned non-null "address"


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(U.LIB_PATH):
        from unet_x3_convolution_amd import build
        build.build(verbose=False)
    U.lib()


def refused(code, fn, *args, **kw):
    with pytest.raises(U.OidnError) as e:
        fn(*args, **kw)
    assert e.value.code == code, e.value
    assert U.last_error()


@pytest.mark.parametrize("m, n", [(0, 1), (1, 1), (3, 31), (3, 32), (3, 33), (1000, 112), (1 << 20, 4096)])
def test_checkpoint_bytes(m, n):
    blocks = -(-n // 32)
    need = m * blocks * (32 + 2)
    assert U.oidn_ckpt_bytes(m, n) == -(-need // 256) * 256


def test_checkpoint_refusals():
    refused(U.OIDN_E_INVALID, U.oidn_ckpt_bytes, -1, 4)
    refused(U.OIDN_E_INVALID, U.oidn_ckpt_bytes, 4, 0)
    refused(U.OIDN_E_UNSUPPORTED, U.oidn_ckpt_bytes, 4, (1 << 24) + 1)
    refused(U.OIDN_E_UNSUPPORTED, U.oidn_ckpt_bytes, 1 << 31, 4)
    refused(U.OIDN_E_UNSUPPORTED, U.oidn_ckpt_bytes, 1 << 30, 1 << 20)
    for args in [(None, 4, 2, 4, P, U.OIDN_F16), (P, 3, 2, 4, P, U.OIDN_F16), (P, 4, 2, 4, None, U.OIDN_F16),
                 (P, 4, 2, 4, P + 8, U.OIDN_F16), (P + 1, 4, 2, 4, P, U.OIDN_F16), (P, 4, -2, 4, P, U.OIDN_F16),
                 (P, 4, 2, 0, P, U.OIDN_F16), (P, 4, 2, 4, P, 7)]:
        refused(U.OIDN_E_INVALID, U.oidn_ckpt_pack, *args, stream=0)
    for args in [(None, 2, 4, P, 4, U.OIDN_F16), (P + 4, 2, 4, P, 4, U.OIDN_F16), (P, 2, 4, P, 3, U.OIDN_F16),
                 (P, 2, 4, None, 4, U.OIDN_F16), (P, 2, 4, P + 2, 4, U.OIDN_F32)]:
        refused(U.OIDN_E_INVALID, U.oidn_ckpt_unpack, *args, stream=0)


def linear(**kw):
    a = dict(x=P, ldx=64, w=P, ldw=64, bias=P, residual=P, ldr=48, y=P, ldy=48, z=P, ldz=48, m=10, k=64, n=48,
             act=U.OIDN_ACT_GELU, dtype=U.OIDN_F16, flags=0, workspace=P, ws_bytes=1 << 40)
    a.update(kw)
    return U.oidn_linear(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(w=None), dict(y=None), dict(x=P + 1), dict(w=P + 1), dict(y=P + 1), dict(residual=P + 1),
    dict(z=P + 1), dict(bias=P + 2), dict(ldx=63), dict(ldw=63), dict(ldr=47), dict(ldy=47), dict(ldz=47),
    dict(m=-1), dict(k=0), dict(n=0), dict(n=-4), dict(act=4), dict(act=-1), dict(dtype=3), dict(flags=4),
    dict(flags=U.OIDN_X_CKPT8), dict(flags=U.OIDN_Z_CKPT8, z=None), dict(flags=U.OIDN_Z_CKPT8, z=P + 2),
    dict(dtype=U.OIDN_F32, x=P + 2)], ids=str)
def test_linear_refuses(bad):
    refused(U.OIDN_E_INVALID, linear, **bad)


def test_linear_limits():
    refused(U.OIDN_E_UNSUPPORTED, linear, n=(1 << 24) + 1, ldy=1 << 25, ldr=1 << 25, ldz=1 << 25)
    refused(U.OIDN_E_UNSUPPORTED, linear, m=1 << 31)
    refused(U.OIDN_E_UNSUPPORTED, linear, ldx=(1 << 32) + 1)


SPLIT = dict(m=64, k=8192, n=64, ldx=8192, ldw=8192, ldy=64, ldr=64, ldz=64)


def test_linear_workspace():
    need = U.oidn_linear_workspace_bytes(SPLIT["m"], SPLIT["k"], SPLIT["n"], U.OIDN_F16)
    assert need > 0
    refused(U.OIDN_E_WORKSPACE, linear, **SPLIT, ws_bytes=need - 1)
    refused(U.OIDN_E_INVALID, linear, **SPLIT, workspace=None)
    refused(U.OIDN_E_INVALID, linear, **SPLIT, workspace=P + 8)
    assert U.oidn_linear_workspace_bytes(0, 64, 64, U.OIDN_F16) == 0
    refused(U.OIDN_E_INVALID, U.oidn_linear_workspace_bytes, 4, 0, 4, U.OIDN_F16)
    refused(U.OIDN_E_INVALID, U.oidn_linear_workspace_bytes, 4, 4, 4, 9)


def linear_backward(**kw):
    a = dict(dy=P, lddy=48, x=P, ldx=64, z=P, ldz=48, w=P, ldw=64, dx=P, lddx=64, dw=P, lddw=64, dbias=P, m=10,
             k=64, n=48, act=U.OIDN_ACT_GELU, dtype=U.OIDN_F16, flags=0, workspace=P, ws_bytes=1 << 40)
    a.update(kw)
    return U.oidn_linear_backward(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(x=None), dict(z=None), dict(w=None), dict(dy=P + 1), dict(dx=P + 1), dict(dw=P + 1),
    dict(dbias=P + 1), dict(lddy=47), dict(ldx=63), dict(ldz=47), dict(ldw=63), dict(lddx=63), dict(lddw=63),
    dict(m=-1), dict(k=0), dict(n=0), dict(act=9), dict(dtype=-1), dict(flags=8), dict(workspace=None),
    dict(flags=U.OIDN_X_CKPT8, x=P + 2), dict(flags=U.OIDN_Z_CKPT8, z=P + 2)], ids=str)
def test_linear_backward_refuses(bad):
    refused(U.OIDN_E_INVALID, linear_backward, **bad)


def test_linear_backward_workspace():
    need = U.oidn_linear_backward_workspace_bytes(10, 64, 48, U.OIDN_ACT_GELU, U.OIDN_F16, 0)
    refused(U.OIDN_E_WORKSPACE, linear_backward, ws_bytes=need - 1)
    both = U.oidn_linear_backward_workspace_bytes(10, 64, 48, U.OIDN_ACT_GELU, U.OIDN_F16, U.OIDN_X_CKPT8)
    assert both > need
    refused(U.OIDN_E_INVALID, U.oidn_linear_backward_workspace_bytes, 10, 64, 48, 4, U.OIDN_F16, 0)
    refused(U.OIDN_E_INVALID, U.oidn_linear_backward_workspace_bytes, 10, 64, 48, 1, U.OIDN_F16, 16)


def ffn(**kw):
    a = dict(x=P, ldx=64, w_in=P, b_in=P, w_out=P, b_out=P, residual=P, ldr=64, y=P, ldy=64, z=P, m=10, d=64,
             f=80, act=U.OIDN_ACT_SILU, dtype=U.OIDN_BF16, flags=0, workspace=P, ws_bytes=1 << 40)
    a.update(kw)
    return U.oidn_ffn(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(w_in=None), dict(w_out=None), dict(y=None), dict(x=P + 1), dict(w_in=P + 1),
    dict(w_out=P + 1), dict(b_in=P + 1), dict(b_out=P + 1), dict(z=P + 1), dict(ldx=63), dict(ldy=63),
    dict(ldr=63), dict(m=-1), dict(d=0), dict(f=0), dict(act=5), dict(dtype=5), dict(flags=U.OIDN_X_CKPT8),
    dict(flags=U.OIDN_Z_CKPT8, z=P + 4), dict(workspace=None), dict(workspace=P + 8)], ids=str)
def test_ffn_refuses(bad):
    refused(U.OIDN_E_INVALID, ffn, **bad)


def test_ffn_limits_and_workspace():
    refused(U.OIDN_E_UNSUPPORTED, ffn, f=1 << 24)
    refused(U.OIDN_E_WORKSPACE, ffn, ws_bytes=U.oidn_ffn_workspace_bytes(10, 64, 80, U.OIDN_BF16) - 1)
    refused(U.OIDN_E_INVALID, U.oidn_ffn_workspace_bytes, 10, 64, 0, U.OIDN_BF16)
    assert U.oidn_ffn_workspace_bytes(0, 64, 80, U.OIDN_BF16) == 0


def ffn_backward(**kw):
    a = dict(dy=P, lddy=64, x=P, ldx=64, z=P, w_in=P, w_out=P, add=P, ldadd=64, dx=P, lddx=64, dw_in=P, db_in=P,
             dw_out=P, db_out=P, m=10, d=64, f=80, act=U.OIDN_ACT_SILU, dtype=U.OIDN_BF16, flags=0, workspace=P,
             ws_bytes=1 << 40)
    a.update(kw)
    return U.oidn_ffn_backward(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(x=None), dict(z=None), dict(w_in=None), dict(w_out=None), dict(dy=P + 1), dict(dx=P + 1),
    dict(dw_in=P + 1), dict(dw_out=P + 1), dict(db_in=P + 2), dict(db_out=P + 2), dict(add=P + 1), dict(lddy=63),
    dict(ldx=63), dict(lddx=63), dict(ldadd=63), dict(m=-1), dict(d=0), dict(f=-1), dict(act=-2), dict(dtype=3),
    dict(flags=4), dict(flags=U.OIDN_X_CKPT8, x=P + 8), dict(flags=U.OIDN_Z_CKPT8, z=P + 8),
    dict(workspace=None)], ids=str)
def test_ffn_backward_refuses(bad):
    refused(U.OIDN_E_INVALID, ffn_backward, **bad)


def test_ffn_backward_workspace():
    need = U.oidn_ffn_backward_workspace_bytes(10, 64, 80, U.OIDN_BF16, 0)
    refused(U.OIDN_E_WORKSPACE, ffn_backward, ws_bytes=need - 1)
    assert U.oidn_ffn_backward_workspace_bytes(10, 64, 80, U.OIDN_BF16, U.OIDN_X_CKPT8) > need


def test_no_rows_enqueue_nothing():
    """m = 0 forward calls and packs return at once, whatever the pointers."""
    linear(m=0, x=None, y=None)
    ffn(m=0, x=None, y=None)
    U.oidn_ckpt_pack(None, 4, 0, 4, None, U.OIDN_F16, stream=0)
    U.oidn_ckpt_unpack(None, 0, 4, None, 4, U.OIDN_F16, stream=0)
