"""Dense operators at their edges: the narrowest operands, whose 16-byte loads
span several rows, as dense as they can lie."""
import ctypes
import math

import pytest
import torch

import unet_x3_convolution_amd as U
from dense_reference import HALF, TINY, TORCH, check, given, linear, linear_backward
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


def last_values(precision):
    """Blocks whose largest magnitudes are the type's last finite values, a few steps below, and of both signs."""
    top = torch.tensor(torch.finfo(TORCH[precision]).max, dtype=torch.float64)
    down = torch.linspace(0, 0.01, 33, dtype=torch.float64).view(-1, 1)
    x = (top * (1 - down)).repeat(1, 64)
    x[:, 1::3] *= -1
    x[:, 2::3] *= 0.25
    return x.to(TORCH[precision])


@pytest.mark.parametrize("precision", ["f32", "f16", "bf16"])
def test_checkpoints_of_the_largest_values_stay_finite(precision):
    """A finite value reads back within half a step of its block's scale, and a step is max / 127 and its rounding."""
    x = last_values(precision)
    m, n = x.shape
    blob, y = bytes_(U.oidn_ckpt_bytes(m, n)), torch.empty_like(x, device="cuda")
    U.oidn_ckpt_pack(x.cuda(), n, m, n, blob, DT[precision])
    U.oidn_ckpt_unpack(blob, m, n, y, n, DT[precision])
    y, x = y.cpu().double(), x.double()
    assert y.isfinite().all()
    step = x.abs().amax(1, keepdim=True) / 127 * (1 + 2.0 ** -8)
    assert ((y - x).abs() <= (0.5 + 2.0 ** -14) * step + torch.finfo(TORCH[precision]).eps / 2 * x.abs()).all()


@pytest.mark.parametrize("precision", ["f32", "f16", "bf16"])
def test_weight_gradients_from_checkpoints_of_the_largest_values(precision):
    """x from 8 bits beside the slope pass and beside the block's backward product: one row in, so dw is x scaled."""
    ty, dt = TORCH[precision], DT[precision]
    x = last_values(precision)[:1]
    n = x.shape[1]
    x8 = bytes_(U.oidn_ckpt_bytes(1, n))
    U.oidn_ckpt_pack(x.cuda(), n, 1, n, x8, dt)
    small = torch.full((1, 1), 2.0 ** -12, dtype=ty, device="cuda")
    one, dw = torch.ones(1, 1, dtype=ty, device="cuda"), torch.empty(1, n, dtype=ty, device="cuda")
    ws = bytes_(U.oidn_linear_backward_workspace_bytes(1, n, 1, U.OIDN_ACT_RELU, dt, U.OIDN_X_CKPT8))
    U.oidn_linear_backward(small, 1, x8, 0, one, 1, None, n, None, n, dw, n, None, 1, n, 1, U.OIDN_ACT_RELU, dt,
                           U.OIDN_X_CKPT8, ws, ws.numel())
    want, bound = x.double() * 2.0 ** -12, x.double().abs().max() * 2.0 ** -12 / 127
    assert ((dw.cpu().double() - want).abs() <= bound).all()
    dy = torch.zeros(1, n, dtype=ty, device="cuda")
    dy[0, 0] = 2.0 ** -12
    z, w_out = torch.ones(1, 2, dtype=ty, device="cuda"), torch.ones(n, 1, dtype=ty, device="cuda")
    dw_in = torch.empty(2, n, dtype=ty, device="cuda")
    ws = bytes_(U.oidn_ffn_backward_workspace_bytes(1, n, 1, dt, U.OIDN_X_CKPT8))
    U.oidn_ffn_backward(dy, n, x8, 0, z, None, w_out, None, 0, None, n, dw_in, None, None, None, 1, n, 1,
                        U.OIDN_ACT_RELU, dt, U.OIDN_X_CKPT8, ws, ws.numel())
    assert ((dw_in.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("precision", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activations_keep_their_relative_accuracy_where_they_vanish(kind, precision):
    """act(z) and act'(z) of negative z against 64 bits, off by a part of their own magnitude: fp32 by the exponential's
    argument (half a step of z^2 / 2 or of z, twice) and 16 units of erfc, the 16-bit gelu by its formula (2^-15, and
    2^-11 past the range of fp16); then the output's rounding."""
    ty, dt, act = TORCH[precision], DT[precision], U.OIDN_ACT_GELU if kind == "gelu" else U.OIDN_ACT_SILU
    x = (-torch.linspace(0, 13 if kind == "gelu" else 80, 5003)).to(ty).cuda().view(-1, 1)
    m, one = x.shape[0], torch.ones(1, 1, dtype=ty, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    ws = bytes_(max(U.oidn_linear_workspace_bytes(m, 1, 1, dt), U.oidn_linear_backward_workspace_bytes(m, 1, 1, act, dt, 0)))
    U.oidn_linear(x, 1, one, 1, None, None, 0, y, 1, None, 0, m, 1, 1, act, dt, 0, ws, ws.numel())
    U.oidn_linear_backward(torch.ones_like(x), 1, x, 1, x, 1, one, 1, dx, 1, None, 1, None, m, 1, 1, act, dt, 0, ws, ws.numel())
    z = x.cpu().double()
    if kind == "gelu":
        p, d = torch.special.erfc(-z / math.sqrt(2)) / 2, torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        part = 2.0 ** -19 + z * z * 2.0 ** -22
        if precision != "f32":
            part = part + torch.where(z > -5.75, 2.0 ** -15, 2.0 ** -11)
    else:
        p = 1 / (1 + torch.exp(-z))
        d, part = p * (1 - p), 2.0 ** -20 - z * 2.0 ** -22
    for got, want, size in ((y, z * p, z.abs() * p), (dx, p + z * d, p + z.abs() * d)):
        bound = part * size
        bound = bound + HALF[precision] * (want.abs() + bound) + TINY[precision]
        bad = ~((got.cpu().double() - want).abs() <= bound)
        assert not bad.any(), (int(bad.sum()), float(z[bad][0]), float(got.cpu()[bad][0]), float(want[bad][0]))


def test_checkpoint_of_more_units_than_a_launch_has_threads():
    """2^30 rows of one column take 2^32 units of eight codes.  Each value is its block's largest: q = +-127."""
    m, part = 2 ** 30 + 3, 2 ** 27
    g = torch.Generator(device="cuda").manual_seed(1)
    x, y = torch.empty(m, 1, dtype=torch.float16, device="cuda"), torch.full((m, 1), float("nan"), dtype=torch.float16, device="cuda")
    for i in range(0, m, part):
        x[i:i + part].normal_(generator=g)
    blob = bytes_(U.oidn_ckpt_bytes(m, 1))
    U.oidn_ckpt_pack(x, 1, m, 1, blob, U.OIDN_F16)
    U.oidn_ckpt_unpack(blob, m, 1, y, 1, U.OIDN_F16)
    del blob
    for i in range(0, m, part):
        a, b = x[i:i + part].float(), y[i:i + part].float()
        step = a.abs() / 127 * (1 + 2.0 ** -8)
        assert ((b - a).abs() <= (0.5 + 2.0 ** -13) * step + a.abs() * 2.0 ** -11 + 2.0 ** -25).all()
    torch.cuda.empty_cache()


def recorded(call):
    """Nodes of a graph that records the call."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    count = ctypes.c_size_t()
    assert U.lib().hipGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(count)) == 0
    return count.value


def test_gradients_of_no_rows_take_one_launch_each():
    """dw inside a wider buffer too: 300 rows of 7 of its 9 columns are zeros, the others as they were."""
    k, n, ld = 7, 300, 9
    dw, db = torch.full((n, ld), 3.0, device="cuda"), torch.full((n,), 3.0, device="cuda")

    def call():
        U.oidn_linear_backward(None, n, None, k, None, n, None, k, None, k, dw, ld, db, 0, k, n, U.OIDN_ACT_GELU, U.OIDN_F32,
                               0, None, 0)

    call()
    assert not dw[:, :k].any() and (dw[:, k:] == 3).all() and not db.any()
    assert recorded(call) == 2


# the largest subnormal, and weights that bring its multiples back into the middle of the range
SUBNORMAL = {"f32": (2.0 ** -127, 2.0 ** 100), "f16": (2.0 ** -15, 2.0 ** 12), "bf16": (2.0 ** -127, 2.0 ** 100)}


@pytest.mark.parametrize("precision", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m, k, n", [(1, 72, 48), (2, 515, 48), (3, 72, 48), (4, 1040, 48), (3, 72, 4104), (5, 72, 48), (33, 72, 48), (300, 129, 200)])
def test_subnormal_inputs_count(m, k, n, precision):
    """Every kernel of a forward product takes subnormals as what they are."""
    size, scale = SUBNORMAL[precision]
    ty, dt = TORCH[precision], DT[precision]
    g = torch.Generator().manual_seed(m + k + n)
    x = ((torch.rand(m, k, generator=g, dtype=torch.float64) * 2 - 1) * size).to(ty)
    w = (torch.randn(n, k, generator=g, dtype=torch.float64) * scale * k ** -0.5).to(ty)
    assert x.any() and x.abs().max().double() <= size
    y = torch.empty(m, n, dtype=ty, device="cuda")
    ws = bytes_(U.oidn_linear_workspace_bytes(m, k, n, dt))
    U.oidn_linear(x.cuda(), k, w.cuda(), k, None, None, 0, y, n, None, 0, m, k, n, U.OIDN_ACT_NONE, dt, 0, ws, ws.numel())
    check(y, linear(given(x), given(w), None, None, "none")[0], precision, "y")


@pytest.mark.parametrize("precision", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m, k, n", [(50, 40, 24), (50, 136, 144), (9000, 24, 40)])
def test_subnormal_gradients_count(m, k, n, precision):
    """dy subnormal, in one pass and in separate products."""
    size, scale = SUBNORMAL[precision]
    ty, dt = TORCH[precision], DT[precision]
    g = torch.Generator().manual_seed(m + k + n)
    dy = ((torch.rand(m, n, generator=g, dtype=torch.float64) * 2 - 1) * size).to(ty)
    x, w = ((torch.randn(r, k, generator=g, dtype=torch.float64) * scale * 2.0 ** -6).to(ty) for r in (m, n))
    dx, dw = torch.empty(m, k, dtype=ty, device="cuda"), torch.empty(n, k, dtype=ty, device="cuda")
    ws = bytes_(U.oidn_linear_backward_workspace_bytes(m, k, n, U.OIDN_ACT_NONE, dt, 0))
    U.oidn_linear_backward(dy.cuda(), n, x.cuda(), k, None, n, w.cuda(), k, dx, k, dw, k, None, m, k, n, U.OIDN_ACT_NONE, dt,
                           0, ws, ws.numel())
    want = linear_backward(given(dy), given(x), None, given(w), "none", precision)
    check(dx, want[0], precision, "dx")
    check(dw, want[1], precision, "dw")
