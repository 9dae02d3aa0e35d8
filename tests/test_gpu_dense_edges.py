"""Dense operators at their edges: the narrowest operands, whose 16-byte loads
span several rows, as dense as they can lie."""
import pytest
import torch

import unet_x3_convolution_amd as U
from dense_reference import TORCH, check, given, linear_backward
from helpers import DT, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    torch_cuda()


def bytes_(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("precision", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m", [33, 34, 65, 66, 70, 129, 134, 8193])
@pytest.mark.parametrize("k, n", [(1, 1), (2, 1), (1, 3), (3, 3), (3, 129), (129, 2), (5, 7)])
def test_gradients_of_the_narrowest_layers(m, k, n, precision):
    """Rows of one to three elements without padding, lengths just past a tile, in one pass and in separate products."""
    ty, dt = TORCH[precision], DT[precision]
    g = torch.Generator().manual_seed(m + 10 * k + 100 * n)
    new = lambda *s: torch.randn(*s, generator=g).to(ty).cuda()  # noqa: E731
    x, w, dy, z = new(m, k), new(n, k), new(m, n), new(m, n)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(n, device="cuda")
    ws = bytes_(U.oidn_linear_backward_workspace_bytes(m, k, n, U.OIDN_ACT_SILU, dt, 0))
    U.oidn_linear_backward(dy, n, x, k, z, n, w, k, dx, k, dw, k, db, m, k, n, U.OIDN_ACT_SILU, dt, 0, ws, ws.numel())
    want = linear_backward(given(dy), given(x), given(z), given(w), "silu", precision)
    check(dx, want[0], precision, "dx")
    check(dw, want[1], precision, "dw")
    check(db, want[2], "f32", "dbias")
