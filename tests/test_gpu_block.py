"""A residual block as a program runs it: the norm before it, a dense layer in 8-bit
floating point, the residual sum after it with its norm, gate and dropout, the next
block's norm in the same pass; two such blocks in a row, forward and backward, on one
workspace.  Each result is checked against its definition on what the pass before it
stored; then the whole step is captured into a graph."""
import pytest
import torch

import block_reference as R
import fp8_reference as F
import unet_x3_convolution_amd as U
from dense_reference import TORCH, act, add, check, given, mul, slope, total
from helpers import DT, torch_cuda

pytestmark = pytest.mark.gpu
EPS = 1e-5
EPS32 = float(torch.tensor(EPS))
RMS, LAYER = U.OIDN_NORM_RMS, U.OIDN_NORM_LAYER


@pytest.fixture(autouse=True)
def gpu():
    torch_cuda()


def bytes_(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


class Blocks:
    """v0 = norm(x0); for each block  o = gelu(v w^T + b),  u = 0.9 x + gate drop(norm(o) wn),  v = norm(u)."""

    def __init__(self, m, d, images, p, precision):
        self.m, self.d, self.p, self.precision, self.dt = m, d, p, precision, DT[precision]
        g = torch.Generator(device="cuda").manual_seed(d)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        half = lambda t: t.to(TORCH[precision])  # noqa: E731
        rows = lambda: torch.empty(m, d, dtype=TORCH[precision], device="cuda")  # noqa: E731
        self.gate_rows = -(-m // images)
        self.x0, self.first = half(rnd(m, d)), 1 + 0.1 * rnd(d)
        self.du = half(rnd(m, d))
        self.v0 = rows()
        self.dx0, self.dfirst = rows(), torch.empty(d, device="cuda")
        packed = lambda a, b: bytes_(U.oidn_fp8_bytes(a, b))  # noqa: E731
        self.blocks = []
        for k in range(2):
            b = dict(w=half(rnd(d, d) * d ** -0.5), bias=0.1 * rnd(d), weight=1 + 0.1 * rnd(d), gate=rnd(images, d),
                     next=1 + 0.1 * rnd(d), rng=torch.tensor([17, 100 * k], dtype=torch.int64, device="cuda"))
            b.update({name: rows() for name in ("z", "o", "u", "v", "dx", "do", "dv")})
            b.update(w8=packed(d, d), w8t=packed(d, d), v8=packed(m, d), v8t=packed(d, m), dw=torch.empty_like(b["w"]))
            b.update({"d" + name: torch.empty_like(b[name]) for name in ("bias", "weight", "gate", "next")})
            self.blocks.append(b)
        act = U.OIDN_ACT_GELU
        self.ws = bytes_(max(U.oidn_linear_fp8_workspace_bytes(m, d, d, self.dt, U.OIDN_X_FP8),
                             U.oidn_linear_fp8_backward_workspace_bytes(m, d, d, act, self.dt, U.OIDN_X_FP8),
                             U.oidn_norm_residual_backward_workspace_bytes(m, d, self.gate_rows, self.dt),
                             U.oidn_norm_backward_workspace_bytes(m, d, self.dt)))

    def step(self):
        m, d, dt, ws, act = self.m, self.d, self.dt, self.ws, U.OIDN_ACT_GELU
        U.oidn_norm(self.x0, d, self.first, None, self.v0, d, m, d, LAYER, EPS, dt)
        x, v = self.x0, self.v0
        for b in self.blocks:
            U.oidn_fp8_pack(b["w"], d, d, d, b["w8"], b["w8t"], dt, U.OIDN_FP8_SQUARE)
            U.oidn_fp8_pack(v, d, m, d, b["v8"], b["v8t"], dt, 0)
            U.oidn_linear_fp8(b["v8"], 0, b["w8"], b["bias"], None, 0, b["o"], d, b["z"], d, m, d, d, act, dt,
                              U.OIDN_X_FP8, ws, ws.numel())
            U.oidn_norm_residual(b["o"], d, b["weight"], None, b["gate"], d, self.gate_rows, x, d, 0.9, self.p,
                                 b["rng"], b["u"], d, b["next"], None, b["v"], d, m, d, RMS, LAYER, EPS, dt)
            x, v = b["u"], b["v"]
        du, dv = None, self.du                 # the loss reads the last v
        for b in reversed(self.blocks):
            U.oidn_norm_residual_backward(du, d, dv, d, b["o"], d, b["weight"], None, b["gate"], d, self.gate_rows,
                                          b["u"], d, 0.9, self.p, b["rng"], b["next"], b["dx"], d, b["do"], d,
                                          b["dgate"], d, b["dweight"], None, b["dnext"], None, m, d, RMS, LAYER, EPS, dt,
                                          ws, ws.numel())
            U.oidn_linear_fp8_backward(b["do"], d, b["v8t"], 0, b["z"], d, b["w8t"], b["dv"], d, b["dw"], d, b["dbias"],
                                       m, d, d, act, dt, U.OIDN_X_FP8, ws, ws.numel())
            du, dv = b["dx"], b["dv"]
        U.oidn_norm_backward(dv, d, self.x0, d, self.first, du, d, self.dx0, d, self.dfirst, None, m, d, LAYER, EPS, dt,
                             ws, ws.numel())
        for b in self.blocks:                  # the next step drops others
            b["rng"][1].add_(1)

    def results(self):
        out = {"v0": self.v0, "dx0": self.dx0, "dfirst": self.dfirst}
        for k, b in enumerate(self.blocks):
            out.update({f"{name}{k}": b[name] for name in ("z", "o", "u", "v", "dx", "do", "dv", "dw", "dbias", "dgate",
                                                           "dweight", "dnext")})
        return out


def turned(a):
    return a[0].T.contiguous(), a[1].T.contiguous()


@pytest.mark.parametrize("precision", ["f16", "bf16"])
@pytest.mark.parametrize("m, d", [(1, 40), (70, 96), (300, 264)])
def test_two_blocks(m, d, precision):
    n = Blocks(m, d, min(m, 3), 0.2, precision)
    offsets = [int(b["rng"][1]) for b in n.blocks]
    n.step()
    torch.cuda.synchronize()
    w = lambda t: t.cpu().double()  # noqa: E731
    ok = lambda got, want, label, p=precision: check(got, want, p, label)  # noqa: E731
    ok(n.v0, R.before(given(n.x0), w(n.first), None, "layer", EPS32), "v0")
    x, v = n.x0, n.v0
    for k, b in enumerate(n.blocks):
        z = F.product(F.coded(given(v)), F.coded(given(b["w"]), True))
        z = add(z, (w(b["bias"]).expand_as(z[0]), torch.zeros_like(z[0])))
        ok(b["z"], z, f"z{k}")
        ok(b["o"], act("gelu", z), f"o{k}")
        keep = R.kept(m, d, n.p, 17, offsets[k])
        ok(b["u"], R.after(given(b["o"]), w(b["weight"]), None, w(b["gate"]), n.gate_rows, given(x), 0.9, keep, "rms",
                           EPS32), f"u{k}")
        ok(b["v"], R.before(given(b["u"]), w(b["next"]), None, "layer", EPS32), f"v{k}")
        x, v = b["u"], b["v"]
    du, dv = None, n.du
    for k in (1, 0):
        b = n.blocks[k]
        want = R.back(given(du) if du is not None else None, given(dv), given(b["o"]), given(b["u"]), w(b["weight"]),
                      None, w(b["gate"]), n.gate_rows, 0.9, R.kept(m, d, n.p, 17, offsets[k]), "rms", w(b["next"]),
                      "layer", EPS32)
        ok(b["dx"], want["dx"], f"dx{k}")
        ok(b["do"], want["d_o"], f"do{k}")
        for name, key in (("dgate", "dgate"), ("dweight", "dweight"), ("dnext", "dnext_weight")):
            ok(b[name], want[key], f"{name}{k}", "f32")
        dz = mul(given(b["do"]), slope("gelu", given(b["z"])))
        v = n.blocks[k - 1]["v"] if k else n.v0
        ok(b["dv"], F.product(F.coded(dz), turned(F.coded(given(b["w"]), True))), f"dv{k}")
        ok(b["dw"], F.product(F.coded(turned(dz)), F.coded(turned(given(v)))), f"dw{k}")
        ok(b["dbias"], total(dz), f"dbias{k}", "f32")
        du, dv = b["dx"], b["dv"]
    want = R.back(given(du), given(dv), None, given(n.x0), None, None, None, 0, 1.0, None, "none", w(n.first), "layer",
                  EPS32)
    ok(n.dx0, want["dx"], "dx0")
    ok(n.dfirst, want["dnext_weight"], "dfirst", "f32")


def test_a_captured_step():
    """Replays of the whole step, on inputs and weights changed in place and with other elements dropped, against the
    eager step; eager steps in between use the same workspace."""
    n, eager = Blocks(300, 96, 3, 0.2, "bf16"), Blocks(300, 96, 3, 0.2, "bf16")
    n.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n.step()
    eager.ws = n.ws
    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(4):
        for t, other in [(n.x0, eager.x0), (n.du, eager.du)] + [(a["w"], b["w"]) for a, b in zip(n.blocks, eager.blocks)]:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda") * 0.5)
            other.copy_(t)
        for a, b in zip(n.blocks, eager.blocks):
            b["rng"].copy_(a["rng"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager.step()
        torch.cuda.synchronize()
        for name, got in n.results().items():
            assert torch.equal(got, eager.results()[name]), name
