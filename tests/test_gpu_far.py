"""Matrices of more than 2^32 elements: rows at their end give what the same rows at the
beginning give, bit for bit, as each row (or tile of rows) is computed alike; and elements
whose place passes 32 bits are dropped by the definition's pattern."""
import numpy as np
import pytest
import torch

import block_reference as R
import unet_x3_convolution_amd as U
from helpers import torch_cuda

pytestmark = pytest.mark.gpu
M, N, SAME = (1 << 20) + 256, 4096, 256
BF = U.OIDN_BF16


@pytest.fixture(autouse=True)
def gpu():
    torch_cuda()
    yield
    torch.cuda.empty_cache()


def bytes_(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def rows(seed, n=N):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(M, n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    x[-SAME:] = x[:SAME]
    return x


def same_ends(y):
    return torch.equal(y[-SAME:].view(torch.int16), y[:SAME].view(torch.int16))


def test_norm_and_gradients():
    x, dy, y = rows(1), rows(2), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    U.oidn_norm(x, N, None, None, y, N, M, N, U.OIDN_NORM_LAYER, 1e-5, BF)
    assert same_ends(y) and bool(y[-1].isfinite().all())
    ws = bytes_(U.oidn_norm_backward_workspace_bytes(M, N, BF))
    dweight = torch.empty(N, device="cuda")
    y.zero_()
    U.oidn_norm_backward(dy, N, x, N, None, None, 0, y, N, dweight, None, M, N, U.OIDN_NORM_RMS, 1e-5, BF, ws, ws.numel())
    assert same_ends(y) and bool(y[-1].any()) and bool(dweight.isfinite().all())


def test_residual_in_place():
    o, x, v = rows(3), rows(4), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    U.oidn_norm_residual(o, N, None, None, None, 0, 0, x, N, 0.5, 0.0, None, x, N, None, None, v, N, M, N,
                         U.OIDN_NORM_RMS, U.OIDN_NORM_LAYER, 1e-5, BF)
    assert same_ends(x) and same_ends(v) and bool(v[-1].any())


def test_layer_in_8_bits():
    k, n = N, 128
    x, dy = rows(5, k), rows(6, n)
    w = torch.randn(n, k, device="cuda").to(torch.bfloat16)
    w8, w8t = bytes_(U.oidn_fp8_bytes(n, k)), bytes_(U.oidn_fp8_bytes(k, n))
    U.oidn_fp8_pack(w, k, n, k, w8, w8t, BF, U.OIDN_FP8_SQUARE)
    y = torch.empty(M, n, dtype=torch.bfloat16, device="cuda")
    ws = bytes_(U.oidn_linear_fp8_workspace_bytes(M, k, n, BF, 0))
    U.oidn_linear_fp8(x, k, w8, None, None, 0, y, n, None, 0, M, k, n, U.OIDN_ACT_NONE, BF, 0, ws, ws.numel())
    assert same_ends(y) and bool(y[-1].any())
    ws = bytes_(U.oidn_linear_fp8_backward_workspace_bytes(M, k, n, U.OIDN_ACT_NONE, BF, 0))
    back = lambda x, dx, dw, dy, m: U.oidn_linear_fp8_backward(  # noqa: E731
        dy, n, x, k, None, 0, w8t, dx, k, dw, k, None, m, k, n, U.OIDN_ACT_NONE, BF, 0, ws, ws.numel())
    dw, last = torch.empty_like(w), torch.empty_like(w)
    # all but the last rows are zeros: the sum over all is the sum over these
    dy[:-SAME] = 0
    back(x, None, dw, dy, M)
    back(x[-SAME:], None, last, dy[-SAME:], SAME)
    assert torch.equal(dw, last) and bool(dw.any())
    dy[:SAME] = dy[-SAME:]
    back(None, x, None, dy, M)
    assert same_ends(x) and bool(x[-1].any())


def test_dropout_of_far_places():
    """Rows of 17 columns take three calls of the generator each, more than 2^32 in all (49 GB,
    in place): the counter's high word is in use."""
    m, n, seed, offset, p, last = (1 << 32) // 3 + 100, 17, 11, 5, 0.3, 200
    x = torch.ones(m, n, dtype=torch.float16, device="cuda")
    rng = torch.tensor([seed, offset], dtype=torch.int64, device="cuda")
    U.oidn_dropout(x, n, None, 0, x, n, m, n, p, rng, U.OIDN_F16)
    got = x[-last:].cpu() != 0
    at = np.arange(3 * (m - last), 3 * m, dtype=np.uint64)
    zeros = np.zeros_like(at)
    words = R.philox([at & np.uint64(0xffffffff), at >> np.uint64(32), zeros + np.uint64(offset), zeros], [seed, 0])
    bits = np.stack([v for w in words for v in (w & np.uint64(0xffff), w >> np.uint64(16))], 1)
    want = torch.from_numpy(bits.reshape(last, 24)[:, :n].astype(np.int64)) >= round(p * 65536)
    assert int(at[0]) < 1 << 32 < int(at[-1]) and torch.equal(got, want)
