"""8-bit products where the large ones of each eight cancel: what is left is off by what the
matrix cores cut below the large ones, 7 * 2^-13 of the largest product for each eight
(fp8_reference), however small it is itself; never by more."""
import pytest
import torch

import fp8_reference as R
import unet_x3_convolution_amd as U
from dense_reference import check, given, t
from helpers import torch_cuda
from test_gpu_fp8 import HALVES, packed, reference, run_back, run_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    torch_cuda()


def cancelling(g, rows, cols, along, most, sign):
    """Codes of four significant bits below 1 but for two of each eight along a dimension, +-most: with sign they
    cancel against a matrix of the same call without."""
    v = torch.randint(-15, 16, (rows, cols), generator=g).double() / 16
    v = v if along else v.T
    v[:, 0::8] = most
    v[:, 1::8] = -most if sign else most
    return (v if along else v.T).contiguous()


@pytest.mark.parametrize("precision", HALVES)
@pytest.mark.parametrize("m, k, n", [(1, 512, 40), (4, 4096, 64), (20, 1024, 48), (70, 128, 72), (300, 96, 264),
                                     (200, 1024, 136), (2100, 512, 2304), (4200, 264, 4360)])
def test_large_products_cancel(m, k, n, precision):
    g = torch.Generator().manual_seed(m + k)
    dev = lambda v: v.to({"f16": torch.float16, "bf16": torch.bfloat16}[precision]).cuda()  # noqa: E731
    x, w = dev(cancelling(g, m, k, True, 16.0, False)), dev(cancelling(g, n, k, True, 1.0, True))
    want = reference(x, w, None, None, "none")[0]
    # the codes are the values themselves, so that the bound is the products' alone
    assert torch.equal(want[0], given(x)[0] @ given(w)[0].T) and float(want[0].abs().max()) < 16 * k / 4
    w8 = packed(w, U.OIDN_FP8_SQUARE)
    check(run_linear(x, w8, n, None, None, "none", precision).get(), want, precision, "y")
    y = run_linear(packed(x), w8, n, None, None, "none", precision, flags=U.OIDN_X_FP8, m=m, k=k)
    check(y.get(), want, precision, "y from packed x")


@pytest.mark.parametrize("m, k, n", [(64, 72, 128), (1024, 136, 264), (2048, 1032, 2304)])
def test_gradients_large_products_cancel(m, k, n):
    """dw sums over the rows, dx over the outputs."""
    g = torch.Generator().manual_seed(m)
    dev = lambda v: v.half().cuda()  # noqa: E731
    for name in ("dw", "dx"):
        if name == "dw":
            dy, x = dev(cancelling(g, m, n, False, 16.0, False)), dev(cancelling(g, m, k, False, 1.0, True))
            w, q, p = dev(torch.zeros(n, k)), t(given(dy)), t(given(x))
        else:
            dy, w = dev(cancelling(g, m, n, True, 16.0, False)), dev(cancelling(g, n, k, False, 1.0, True))
            x, q, p = dev(torch.zeros(m, k)), given(dy), t(given(w))
        dx, dw, _ = run_back(dy, x, None, w, "none", "f16")
        check((dx if name == "dx" else dw).get(), R.product(q, p), "f16", name)
