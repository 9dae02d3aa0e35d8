"""Norms and their gradients where a workgroup goes through several rows: the next row's
loads, the sums that stay in registers from row to row and the ends of gate groups inside a
chunk, for every count of lanes that a row takes, against 64 bits (block_reference)."""
import pytest
import torch

import block_reference as R
import unet_x3_convolution_amd as U
from dense_reference import TORCH, check, given
from helpers import DT, torch_cuda
from test_gpu_dense import GUARD, bytes_
from test_gpu_norm import EPS, EPS32, KIND, back_case, reference, residual_case, run_back, run_residual, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    torch_cuda()


def gated(c, gate_rows):
    """The case with a gate for every gate_rows rows (0: none)."""
    m, n = c["m"], c["n"]
    c["gate_rows"] = gate_rows
    c["gate"] = torch.randn(-(-m // gate_rows), n + c["pad"], device="cuda")[:, :n] if gate_rows else None
    return c


# rows enough for three to five a chunk: 4 to 64 lanes a row, whose workgroups take several rows at once, and
# 128, 256, 512, 1024 lanes and the rows past what registers hold, which are taken one at a time
CHUNKS = [(16400, 30), (9000, 56), (7000, 120), (5000, 200), (4200, 400), (4300, 600), (4300, 1024), (1600, 1032),
          (1600, 2040), (1100, 2056), (1100, 4096), (1030, 4099), (1030, 8192), (1030, 8200)]


@pytest.mark.parametrize("gate_rows", [0, 1, 2, 4, 70, "m"])
@pytest.mark.parametrize("m, n", CHUNKS)
def test_gradients_over_several_rows(m, n, gate_rows):
    """All of them with dropout, and without the shifts', which other kernels take: the same bits."""
    kinds, precision = [("rms", "layer"), ("layer", "rms"), ("none", "layer")], ["bf16", "f32", "f16"]
    turn = (m + n + (gate_rows if gate_rows != "m" else 5)) % 3
    c = gated(back_case(m, n, *kinds[turn], precision[turn], 26), m if gate_rows == "m" else gate_rows)
    want, outs = reference(c), run_back(c)
    for name, o in outs.items():
        got = o.get() if name in ("dx", "d_o", "dgate") else o.get()[0]
        check(got, want[name], c["precision"] if name in ("dx", "d_o") else "f32", name)
    some = run_back(c, [name for name in outs if name not in ("dshift", "dnext_shift")])
    for name, o in some.items():
        left = name in ("dshift", "dnext_shift")
        assert torch.equal(o.get(), torch.full_like(o.get(), GUARD) if left else outs[name].get()), name


@pytest.mark.parametrize("m, n, gate_rows", [(1020, 4096, 5), (1020, 4099, 5), (1020, 8200, 5), (44000, 30, 16),
                                             (12003, 30, 8), (900, 56, 1), (3001, 120, 2), (5003, 24, 4), (66000, 24, 1)])
def test_gradients_of_parted_and_shared_groups(m, n, gate_rows):
    """Groups in fewer parts than their rows ask for; groups of few rows, one a row lane and one a workgroup."""
    test_gradients_over_several_rows(m, n, gate_rows)


@pytest.mark.parametrize("m, n", CHUNKS)
def test_norm_gradients_over_several_rows(m, n):
    """The gradients of a norm by itself, as parts of a call without a branch."""
    c = back_case(m, n, "none", ["rms", "layer"][n // 8 % 2], ["bf16", "f32"][m // 100 % 2], 26)
    ty, dt = TORCH[c["precision"]], DT[c["precision"]]
    dx, dw, ds = (torch.empty(*shape, dtype=t, device="cuda") for shape, t in
                  (((m, n), ty), ((n,), torch.float32), ((n,), torch.float32)))
    ws = bytes_(U.oidn_norm_backward_workspace_bytes(m, n, dt))
    U.oidn_norm_backward(c["dv"], c["dv"].stride(0), c["u"], c["u"].stride(0), c["next_weight"], c["du"],
                         c["du"].stride(0), dx, n, dw, ds, m, n, KIND[c["following"]], EPS, dt, ws, ws.numel())
    want = R.back(given(c["du"]), given(c["dv"]), None, given(c["u"]), None, None, None, 0, 1.0, None, "none",
                  wide(c["next_weight"]), c["following"], EPS32)
    check(dx, want["dx"], c["precision"], "dx")
    check(dw, want["dnext_weight"], "f32", "dweight")
    check(ds, want["dnext_shift"], "f32", "dshift")


# more rows than a launch's workgroups take at once
@pytest.mark.parametrize("m, n", [(132000, 20), (66000, 64), (33000, 128), (17000, 250), (8300, 300), (4200, 600),
                                  (2100, 1032), (1100, 2049), (1100, 4096), (600, 8192), (600, 8191)])
def test_forward_passes_over_several_rows(m, n):
    turn = (m + n) % 3
    c = gated(residual_case(m, n, *[("rms", "layer"), ("layer", "rms"), ("none", "layer")][turn],
                            ["bf16", "f32", "f16"][turn], 26), [3, m, 37][turn])
    c["next_shift"] = torch.randn(n, device="cuda")
    u, v = run_residual(c)
    want = R.after(given(c["o"]), wide(c["weight"]), wide(c["shift"]), wide(c["gate"]), c["gate_rows"], given(c["x"]),
                   c["scale"], c["keep"], c["kind"], EPS32)
    check(u.get(), want, c["precision"], "u")
    check(v.get(), R.before(given(u.get()), wide(c["next_weight"]), wide(c["next_shift"]), c["following"], EPS32),
          c["precision"], "v")


def test_weight_gradient_of_many_rows():
    """More than 2^32 elements, 2049 rows a chunk.  A term dy hat carries the row's statistic (sums of 4096 squares
    by 512 lanes of eight, 8 + 6 + 8 additions in a chain, and a square root) and its own products, fewer than 64
    roundings in all; it then passes at most 2049 additions in its chunk and 512 over the chunks."""
    m, n, at_once = (1 << 20) + 256, 4096, 1 << 15
    g = torch.Generator(device="cuda").manual_seed(8)
    x, dy = (torch.empty(m, n, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    ws = bytes_(U.oidn_norm_backward_workspace_bytes(m, n, U.OIDN_BF16))
    dw, ds = (torch.empty(n, device="cuda") for _ in range(2))
    U.oidn_norm_backward(dy, n, x, n, None, None, 0, None, n, dw, ds, m, n, U.OIDN_NORM_RMS, EPS, U.OIDN_BF16, ws,
                         ws.numel())
    sums = torch.zeros(4, n, dtype=torch.float64, device="cuda")
    for i in range(0, m, at_once):
        a, b = x[i:i + at_once].double(), dy[i:i + at_once].double()
        hat = a * (a.square().mean(1, keepdim=True) + EPS32).rsqrt()
        for k, term in enumerate((b * hat, b)):
            sums[k] += term.sum(0)
            sums[k + 2] += term.abs().sum(0)
    for k, got in enumerate((dw, ds)):
        assert ((got.double() - sums[k]).abs() <= (2049 + 512 + 64) * 2.0 ** -24 * sums[k + 2]).all()
