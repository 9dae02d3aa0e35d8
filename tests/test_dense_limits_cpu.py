"""Where the dense operators' sizes end: a launch holds less than 2^32 work
items, 256 a tile.  Asked of the sizes and of calls without a workspace, so
that nothing is enqueued on either side of the border."""
import pytest

import unet_x3_convolution_amd as U

P = 4096          # a 16-byte aligned non-null "address"
# tiles go in eights, of 64 rows (32 for a lone plain product in fp32)
TILES = (2 ** 32 - 1) // 256 // 8 * 8


def code(fn, *args, **kw):
    try:
        fn(*args, **kw)
    except U.OidnError as e:
        return e.code
    return U.OIDN_OK


@pytest.mark.parametrize("dtype", [U.OIDN_F32, U.OIDN_F16, U.OIDN_BF16])
@pytest.mark.parametrize("k, n", [(1, 1), (8, 64), (100, 7)])
def test_linear_rows(k, n, dtype):
    last = TILES * 64
    most = max(m for m in (last, last // 2) if code(U.oidn_linear_workspace_bytes, m, k, n, dtype) == U.OIDN_OK)
    assert code(U.oidn_linear_workspace_bytes, most + 1, k, n, dtype) == U.OIDN_E_UNSUPPORTED
    assert code(U.oidn_linear, P, k, P, k, None, None, 0, P, n, None, 0, most + 1, k, n, U.OIDN_ACT_RELU, dtype, 0, P,
                1 << 40, stream=0) == U.OIDN_E_UNSUPPORTED
    assert code(U.oidn_linear_workspace_bytes, 2 ** 31 - 1, k, n, dtype) == U.OIDN_E_UNSUPPORTED


@pytest.mark.parametrize("dtype", [U.OIDN_F32, U.OIDN_F16])
def test_ffn_rows(dtype):
    last = TILES * 64
    most = max(m for m in (last, last // 2) if code(U.oidn_ffn_workspace_bytes, m, 8, 16, dtype) == U.OIDN_OK)
    assert code(U.oidn_ffn_workspace_bytes, most + 1, 8, 16, dtype) == U.OIDN_E_UNSUPPORTED
    assert code(U.oidn_ffn, P, 8, P, None, P, None, None, 0, P, 8, None, most + 1, 8, 16, U.OIDN_ACT_SILU, dtype, 0, P,
                1 << 62, stream=0) == U.OIDN_E_UNSUPPORTED


def backward(m, dtype, flags, dx=P, dw=P, n=4):
    return code(U.oidn_linear_backward, P, n, P, 8, P, n, P, 8, dx, 8, dw, 8, P, m, 8, n, U.OIDN_ACT_GELU, dtype, flags,
                P, 0, stream=0)


def test_gradients_of_many_rows():
    """dx is what takes a tile for 64 rows; the sums over the rows are short of tiles, and a narrow layer's one pass
    takes any number of rows."""
    many = TILES * 64 + 1
    for dtype, flags in ((U.OIDN_F32, 0), (U.OIDN_F16, U.OIDN_X_CKPT8), (U.OIDN_BF16, U.OIDN_Z_CKPT8)):
        assert backward(many // 2, dtype, flags) == U.OIDN_E_WORKSPACE
        assert backward(many, dtype, flags) == U.OIDN_E_UNSUPPORTED
        assert backward(many, dtype, flags, dx=None) == U.OIDN_E_WORKSPACE
        assert backward(many, dtype, flags, dw=None) == U.OIDN_E_UNSUPPORTED
    assert backward(2 ** 31 - 1, U.OIDN_F16, 0) == U.OIDN_E_WORKSPACE


def test_block_gradients_of_many_rows():
    def call(m, dx=None, dw_in=None, db_out=None):
        return code(U.oidn_ffn_backward, P, 4, P, 4, P, P, P, None, 0, dx, 4, dw_in, None, None, db_out, m, 4, 8,
                    U.OIDN_ACT_SILU, U.OIDN_F32, 0, P, 0, stream=0)

    many = TILES * 64 + 1
    assert call(many, dw_in=P) == U.OIDN_E_UNSUPPORTED       # dh
    assert call(many // 2, dw_in=P) == call(many // 2, dx=P) == U.OIDN_E_WORKSPACE
    assert call(many, db_out=P) == U.OIDN_E_WORKSPACE
