"""The norms around a block and dropout on the host: sizes of workspaces, every
refusal before any device work, and the generator's published answers.  No GPU is
touched: the pointers are small integers that are only looked at."""
import os

import numpy as np
import pytest

import block_reference as R
import unet_x3_convolution_amd as U

P = 4096          # a 16-byte aligned non-null "address"
NAN, INF = float("nan"), float("inf")


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


@pytest.mark.parametrize("counter, key, want", [
    ([0] * 4, [0] * 2, [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
    ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
     [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1])])
def test_generator(counter, key, want):
    """The oracle's generator against the test vectors published with it."""
    assert [int(v) for v in R.philox([np.array(v, np.uint64) for v in counter], key)] == want


def norm(**kw):
    a = dict(x=P, ldx=48, weight=P, shift=P, y=P, ldy=48, m=10, n=48, norm=U.OIDN_NORM_RMS, eps=1e-5, dtype=U.OIDN_F16)
    a.update(kw)
    return U.oidn_norm(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(y=None), dict(x=P + 1), dict(y=P + 1), dict(weight=P + 2), dict(shift=P + 1), dict(ldx=47),
    dict(ldy=47), dict(m=-1), dict(n=0), dict(n=-3), dict(norm=U.OIDN_NORM_NONE), dict(norm=3), dict(norm=-1),
    dict(eps=-1e-5), dict(eps=NAN), dict(eps=INF), dict(dtype=3), dict(dtype=U.OIDN_F32, x=P + 2)], ids=str)
def test_norm_refuses(bad):
    refused(U.OIDN_E_INVALID, norm, **bad)


def test_norm_limits():
    refused(U.OIDN_E_UNSUPPORTED, norm, n=(1 << 24) + 1, ldx=1 << 25, ldy=1 << 25)
    refused(U.OIDN_E_UNSUPPORTED, norm, m=1 << 31)
    refused(U.OIDN_E_UNSUPPORTED, norm, ldx=(1 << 32) + 1)


def norm_backward(**kw):
    a = dict(dy=P, lddy=48, x=P, ldx=48, weight=P, add=P, ldadd=48, dx=P, lddx=48, dweight=P, dshift=P, m=5000, n=48,
             norm=U.OIDN_NORM_LAYER, eps=1e-5, dtype=U.OIDN_BF16, workspace=P, ws_bytes=1 << 40)
    a.update(kw)
    return U.oidn_norm_backward(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(x=None), dict(dy=P + 1), dict(x=P + 1), dict(dx=P + 1), dict(add=P + 1), dict(weight=P + 1),
    dict(dweight=P + 2), dict(dshift=P + 3), dict(lddy=47), dict(ldx=47), dict(ldadd=47), dict(lddx=47), dict(m=-1),
    dict(n=0), dict(norm=0), dict(norm=7), dict(eps=NAN), dict(dtype=-1), dict(workspace=None),
    dict(workspace=P + 8)], ids=str)
def test_norm_backward_refuses(bad):
    refused(U.OIDN_E_INVALID, norm_backward, **bad)


def residual(**kw):
    a = dict(o=P, ldo=48, weight=P, shift=P, gate=P, ldg=48, gate_rows=4, x=P, ldx=48, scale=0.5, p=0.1, rng=P, u=P,
             ldu=48, next_weight=P, next_shift=P, v=P, ldv=48, m=10, n=48, norm=U.OIDN_NORM_RMS,
             next_norm=U.OIDN_NORM_LAYER, eps=1e-5, dtype=U.OIDN_F16)
    a.update(kw)
    return U.oidn_norm_residual(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(o=None), dict(x=None), dict(u=None), dict(v=None), dict(o=P + 1), dict(x=P + 1), dict(u=P + 1), dict(v=P + 1),
    dict(ldo=47), dict(ldx=47), dict(ldu=47), dict(ldv=47), dict(ldg=47), dict(gate=P + 2), dict(gate_rows=0),
    dict(gate_rows=-4), dict(p=-0.1), dict(p=1.1), dict(p=NAN), dict(rng=None), dict(rng=P + 4), dict(weight=P + 1),
    dict(shift=P + 1), dict(next_weight=P + 1), dict(next_shift=P + 1), dict(m=-1), dict(n=0), dict(norm=3),
    dict(next_norm=-1), dict(next_norm=U.OIDN_NORM_NONE), dict(eps=-1.0), dict(dtype=9)], ids=str)
def test_norm_residual_refuses(bad):
    refused(U.OIDN_E_INVALID, residual, **bad)


def residual_backward(**kw):
    a = dict(du=P, lddu=48, dv=P, lddv=48, o=P, ldo=48, weight=P, shift=P, gate=P, ldg=48, gate_rows=4, u=P, ldu=48,
             scale=0.5, p=0.1, rng=P, next_weight=P, dx=P, lddx=48, d_o=P, lddo=48, dgate=P, lddg=48, dweight=P,
             dshift=P, dnext_weight=P, dnext_shift=P, m=5000, n=48, norm=U.OIDN_NORM_RMS, next_norm=U.OIDN_NORM_LAYER,
             eps=1e-5, dtype=U.OIDN_F16, workspace=P, ws_bytes=1 << 40)
    a.update(kw)
    return U.oidn_norm_residual_backward(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(dv=None), dict(o=None), dict(u=None), dict(du=P + 1), dict(dv=P + 1), dict(o=P + 1), dict(u=P + 1),
    dict(dx=P + 1), dict(d_o=P + 1), dict(lddu=47), dict(lddv=47), dict(ldo=47), dict(ldu=47), dict(lddx=47),
    dict(lddo=47), dict(ldg=47), dict(lddg=47), dict(gate=None), dict(dgate=P + 1), dict(gate_rows=0), dict(p=2.0),
    dict(rng=None), dict(weight=P + 1), dict(dweight=P + 1), dict(dshift=P + 1), dict(dnext_weight=P + 1),
    dict(dnext_shift=P + 1), dict(next_norm=U.OIDN_NORM_NONE), dict(du=None, next_norm=U.OIDN_NORM_NONE, dv=None,
                                                                    dnext_weight=None, dnext_shift=None),
    dict(m=-1), dict(n=0), dict(norm=5), dict(eps=INF), dict(dtype=4), dict(workspace=None)], ids=str)
def test_norm_residual_backward_refuses(bad):
    refused(U.OIDN_E_INVALID, residual_backward, **bad)


def test_workspaces():
    need = U.oidn_norm_backward_workspace_bytes(5000, 48, U.OIDN_BF16)
    refused(U.OIDN_E_WORKSPACE, norm_backward, ws_bytes=need - 1)
    need = U.oidn_norm_residual_backward_workspace_bytes(5000, 48, 4, U.OIDN_F16)
    refused(U.OIDN_E_WORKSPACE, residual_backward, ws_bytes=need - 1)
    assert U.oidn_norm_backward_workspace_bytes(0, 48, U.OIDN_F16) == 0
    assert U.oidn_norm_residual_backward_workspace_bytes(0, 48, 0, U.OIDN_F16) == 0
    refused(U.OIDN_E_INVALID, U.oidn_norm_residual_backward_workspace_bytes, 10, 48, -1, U.OIDN_F16)
    refused(U.OIDN_E_INVALID, U.oidn_norm_backward_workspace_bytes, 10, 0, U.OIDN_F16)
    refused(U.OIDN_E_INVALID, U.oidn_norm_backward_workspace_bytes, 10, 4, 8)
    # a short pass over few rows of partial sums, however many rows there are
    assert U.oidn_norm_residual_backward_workspace_bytes(1 << 30, 32, 1 << 18, U.OIDN_F16) < (1 << 30) * 48


def dropout(**kw):
    a = dict(x=P, ldx=48, residual=P, ldr=48, y=P, ldy=48, m=10, n=48, p=0.5, rng=P, dtype=U.OIDN_F16)
    a.update(kw)
    return U.oidn_dropout(**a, stream=0)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(y=None), dict(x=P + 1), dict(y=P + 1), dict(residual=P + 1), dict(ldx=47), dict(ldr=47),
    dict(ldy=47), dict(m=-1), dict(n=0), dict(p=-1e-9), dict(p=1.0001), dict(p=NAN), dict(rng=None), dict(rng=P + 4),
    dict(dtype=3)], ids=str)
def test_dropout_refuses(bad):
    refused(U.OIDN_E_INVALID, dropout, **bad)


def test_no_rows_enqueue_nothing():
    norm(m=0, x=None, y=None)
    residual(m=0, x=None, o=None, u=None, v=None)
    dropout(m=0, x=None, y=None)
    norm_backward(m=0, dy=None, x=None, dweight=None, dshift=None, workspace=None)
    residual_backward(m=0, du=None, dv=None, o=None, u=None, dweight=None, dshift=None, dnext_weight=None,
                      dnext_shift=None, workspace=None)


@pytest.mark.parametrize("m, n, gate_rows, most", [
    (65536, 32, 65, 1024), (131072, 64, 65, 2048), (16384, 4096, 33, 512), (8192, 8192, 17, 512), (4096, 8256, 9, 512),
    (130560, 32, 170, 768), (16384, 640, 17, 1024), (16384, 640, 40, 1536), (16384, 2048, 48, 768), (16384, 4096, 0, 512),
    (16384, 1024, 0, 1024), (1 << 20, 64, 0, 768), (1 << 20, 4096, 1, 1024)])
def test_sums_are_over_few_chunks(m, n, gate_rows, most):
    """A chunk of rows leaves four rows of partial sums, and one of a gate's where a group has several chunks."""
    assert U.oidn_norm_residual_backward_workspace_bytes(m, n, gate_rows, U.OIDN_F16) - (m * 32 if n > 8192 else 0) <= (
        most * 4 * n * 4 + (most * n * 4 if gate_rows > m // most else 0) + 512)


@pytest.mark.parametrize("groups, rows, n, lanes", [(1024, 8, 32, False), (1024, 16, 32, False), (1536, 8, 32, True),
                                                    (512, 16, 32, False), (1024, 4, 96, True), (768, 4, 96, False),
                                                    (512, 1, 32, True), (2800, 16, 32, True)])
def test_gate_groups_of_few_rows(groups, rows, n, lanes):
    """A workgroup each, or a row lane each, of 64 (up to 32 columns) or 16 (96)."""
    at_once = 64 if n <= 32 else 16
    chunks = -(-groups // at_once) if lanes else groups
    assert U.oidn_norm_residual_backward_workspace_bytes(groups * rows, n, rows, U.OIDN_F16) == -(-chunks * 16 * n // 256) * 256
