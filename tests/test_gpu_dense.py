"""The dense operators on the GPU against their definitions in 64 bits, with
error bounds carried through every step (dense_reference)."""
import math

import pytest
import torch

import unet_x3_convolution_amd as U
from dense_reference import (ACTS, HALF, TORCH, act, check, ffn, ffn_backward, given, linear, linear_backward,
                             slope, stored, t, total)
from helpers import DT, torch_cuda

pytestmark = pytest.mark.gpu

PRECISIONS = ["f32", "f16", "bf16"]
ACT = {"none": U.OIDN_ACT_NONE, "relu": U.OIDN_ACT_RELU, "silu": U.OIDN_ACT_SILU, "gelu": U.OIDN_ACT_GELU}
GUARD = -7.0     # what surrounds every output; exact in each type


@pytest.fixture(autouse=True)
def gpu():
    torch_cuda()


class Maker:
    def __init__(self, seed, precision):
        self.g = torch.Generator().manual_seed(seed)
        self.type = TORCH[precision]

    def rows(self, m, n, pad=0, scale=1.0, shift=0):
        """m x n normal values; the pitch has `pad` more columns, which hold NaN, and the base is `shift` elements in."""
        v = (torch.randn(m, n, generator=self.g) * scale).to(self.type)
        buf = torch.full((m * (n + pad) + shift + 8,), float("nan"), dtype=self.type)
        out = buf.cuda()[shift:shift + m * (n + pad)].view(m, n + pad)[:, :n]
        out.copy_(v)
        return out

    def vec(self, n):
        return (torch.randn(n, generator=self.g) * 0.5).cuda()


class Out:
    """A guarded output: rows x cols at a padded pitch, guards before and after."""

    def __init__(self, m, n, dtype, pad=0, shift=0):
        self.m, self.n, self.ld = m, n, n + pad
        self.buf = torch.full((m * self.ld + shift + 64,), GUARD, dtype=dtype, device="cuda")
        self.lo = 32 + shift
        self.view = self.buf[self.lo:self.lo + m * self.ld].view(m, self.ld)

    def get(self):
        torch.cuda.synchronize()
        b = self.buf.clone()
        b[self.lo:self.lo + self.m * self.ld].view(self.m, self.ld)[:, :self.n] = GUARD
        assert (b == GUARD).all(), "written outside the output"
        return self.view[:, :self.n]


def bytes_(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def ptr(o):
    return o.view if isinstance(o, Out) else o


def run_linear(x, w, bias, residual, kind, precision, z=None, flags=0, pad=0, shift=0, stream=None):
    m, k, n, dt = x.shape[0], x.shape[1], w.shape[0], DT[precision]
    y = Out(m, n, TORCH[precision], pad, shift)
    ws = bytes_(U.oidn_linear_workspace_bytes(m, k, n, dt))
    U.oidn_linear(x, x.stride(0), w, w.stride(0), bias, residual, residual.stride(0) if residual is not None else 0,
                  y.view, y.ld, ptr(z), z.ld if isinstance(z, Out) else 0, m, k, n, ACT[kind], dt, flags, ws,
                  ws.numel(), stream=stream)
    return y


# m, k, n: single elements and rows, sizes around the tiles and fragments, long sums that are cut in slices
LINEAR = [(1, 1, 1), (1, 8, 8), (1, 1000, 300), (2, 4096, 40), (3, 5, 7), (5, 64, 64), (8, 512, 96), (16, 64, 32),
          (17, 33, 130), (63, 65, 33), (64, 1024, 64), (100, 96, 384), (129, 130, 127), (257, 72, 264),
          (300, 1000, 8), (640, 40, 520), (1025, 24, 1025)]


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, k, n", LINEAR)
def test_linear(m, k, n, precision):
    seed = m * 7 + k * 3 + n
    mk = Maker(seed, precision)
    kind = ACTS[seed % 4]
    pad, shift = [(0, 0), (8, 0), (3, 0), (8, 1)][(m + k) % 4]
    x, w = mk.rows(m, k, pad, shift=shift), mk.rows(n, k, pad, k ** -0.5)
    bias = mk.vec(n) if seed % 3 else None
    residual = mk.rows(m, n, pad, shift=shift) if seed % 2 else None
    z = Out(m, n, TORCH[precision], pad) if seed % 5 else None
    y = run_linear(x, w, bias, residual, kind, precision, z, pad=pad, shift=shift)
    want, want_z = linear(given(x), given(w), given(bias) if bias is not None else None,
                          given(residual) if residual is not None else None, kind)
    check(y.get(), want, precision, "y")
    if z is not None:
        check(z.get(), want_z, precision, "z")


@pytest.mark.parametrize("precision", PRECISIONS)
def test_linear_many_tiles(precision):
    """More tiles than compute units, ragged in both directions."""
    mk = Maker(5, precision)
    m, k, n = 2113, 136, 2310
    x, w, bias, r = mk.rows(m, k), mk.rows(n, k, scale=k ** -0.5), mk.vec(n), mk.rows(m, n)
    y = run_linear(x, w, bias, r, "gelu", precision)
    check(y.get(), linear(given(x), given(w), given(bias), given(r), "gelu")[0], precision, "y")


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, k, n", [(1, 24, 16), (40, 24, 48), (7, 2048, 24), (130, 24, 72)])
def test_linear_in_place_residual(m, k, n, precision):
    mk = Maker(11, precision)
    x, w = mk.rows(m, k), mk.rows(n, k, scale=k ** -0.5)
    y = mk.rows(m, n)
    want, _ = linear(given(x), given(w), None, given(y), "relu")
    ws = bytes_(U.oidn_linear_workspace_bytes(m, k, n, DT[precision]))
    U.oidn_linear(x, k, w, k, None, y, n, y, n, None, 0, m, k, n, U.OIDN_ACT_RELU, DT[precision], 0, ws, ws.numel())
    check(y, want, precision, "y")


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("kind", ACTS)
def test_activations_and_slopes_over_their_range(kind, precision):
    """k = 1 and weight 1: y = act(x) and dx = dy act'(x) at any x, infinities, NaN and the ends among them."""
    x = torch.cat([torch.linspace(-12, 12, 4001), torch.linspace(-200, 200, 801),
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e4, -3e4, float("inf"), float("-inf"), float("nan")])])
    x = x.to(TORCH[precision]).cuda().view(-1, 1)
    one = torch.ones(1, 1, dtype=x.dtype, device="cuda")
    m, dt = x.shape[0], DT[precision]
    y = run_linear(x, one, None, None, kind, precision).get()
    dx = Out(m, 1, x.dtype)
    ws = bytes_(U.oidn_linear_backward_workspace_bytes(m, 1, 1, ACT[kind], dt, 0))
    U.oidn_linear_backward(torch.ones_like(x), 1, x, 1, x, 1, one, 1, dx.view, 1, None, 0, None, m, 1, 1, ACT[kind],
                           dt, 0, ws, ws.numel())
    dx = dx.get()
    fin = x.isfinite().view(-1)
    z = given(x[fin])
    check(y[fin], act(kind, z), precision, "y")
    check(dx[fin], slope(kind, z), precision, "slope")
    inf, ninf, nan = m - 3, m - 2, m - 1
    assert y[inf].item() == math.inf and y[nan].isnan().item()
    assert y[ninf].item() == (-math.inf if kind == "none" else 0)
    assert dx[inf].item() == 1 and dx[ninf].item() == (1 if kind == "none" else 0)
    assert kind == "none" or dx[nan].isnan().item()


@pytest.mark.parametrize("precision", PRECISIONS)
def test_linear_keeps_rows_apart(precision):
    """A NaN or an infinity in a row reaches that row's outputs only, and NaN past the rows' ends reach none."""
    mk = Maker(3, precision)
    m, k, n = 70, 100, 66
    x, w = mk.rows(m, k, 4), mk.rows(n, k, 4)
    x[10, 3] = float("nan")
    x[33, 99] = float("inf")
    y = run_linear(x, w, None, None, "none", precision).get()
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    bad[[10, 33]] = True
    assert y[10].isnan().all() and not y[33].isfinite().any()
    assert y[~bad].isfinite().all()


BACK = [(1, 1, 1), (1, 64, 40), (3, 5, 7), (33, 64, 64), (64, 65, 31), (100, 96, 384), (257, 40, 72),
        (1000, 33, 17), (4097, 32, 64), (700, 264, 136)]


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, k, n", BACK)
def test_linear_backward(m, k, n, precision):
    seed = m + 3 * k + 7 * n
    mk, kind, dt = Maker(seed, precision), ACTS[seed % 4], DT[precision]
    pad = [0, 8, 3][seed % 3]
    x, w, dy, z = mk.rows(m, k, pad), mk.rows(n, k, pad, k ** -0.5), mk.rows(m, n, pad), mk.rows(m, n, pad)
    dx, dw = Out(m, k, TORCH[precision], pad), Out(n, k, TORCH[precision], pad)
    db = Out(1, n, torch.float32)
    ws = bytes_(U.oidn_linear_backward_workspace_bytes(m, k, n, ACT[kind], dt, 0))
    U.oidn_linear_backward(dy, dy.stride(0), x, x.stride(0), z, z.stride(0), w, w.stride(0), dx.view, dx.ld, dw.view,
                           dw.ld, db.view, m, k, n, ACT[kind], dt, 0, ws, ws.numel())
    want = linear_backward(given(dy), given(x), given(z), given(w), kind, precision)
    check(dx.get(), want[0], precision, "dx")
    check(dw.get(), want[1], precision, "dw")
    check(db.get()[0], want[2], "f32", "dbias")


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("asked", ["dx", "dw", "dbias", "nothing"])
def test_linear_backward_parts(asked, precision):
    """Each gradient alone: the same bits as all at once; what it does not need may be null."""
    mk, dt = Maker(21, precision), DT[precision]
    m, k, n = 150, 72, 40
    x, w, dy, z = mk.rows(m, k), mk.rows(n, k), mk.rows(m, n), mk.rows(m, n)
    ws = bytes_(U.oidn_linear_backward_workspace_bytes(m, k, n, U.OIDN_ACT_SILU, dt, 0))

    def run(want):
        o = {"dx": Out(m, k, x.dtype), "dw": Out(n, k, x.dtype), "dbias": Out(1, n, torch.float32)}
        p = {key: v.view if key in want else None for key, v in o.items()}
        U.oidn_linear_backward(dy, n, x if p["dw"] is not None else None, k, z, n, w if p["dx"] is not None else None, k,
                               p["dx"], k, p["dw"], k, p["dbias"], m, k, n, U.OIDN_ACT_SILU, dt, 0, ws, ws.numel())
        return {key: v.get() for key, v in o.items()}

    both, some = run(["dx", "dw", "dbias"]), run([asked])
    for key in both:
        assert torch.equal(some[key], both[key] if key == asked else torch.full_like(both[key], GUARD)), key


@pytest.mark.parametrize("precision", PRECISIONS)
def test_gradients_of_no_rows_are_zero(precision):
    dt, ty = DT[precision], TORCH[precision]
    dw, db = Out(5, 7, ty, 2), Out(1, 5, torch.float32)
    U.oidn_linear_backward(None, 5, None, 7, None, 5, None, 7, None, 7, dw.view, dw.ld, db.view, 0, 7, 5,
                           U.OIDN_ACT_GELU, dt, 0, None, 0)
    assert not dw.get().any() and not db.get().any()
    w_in, w_out, b_in, b_out = Out(12, 9, ty), Out(9, 6, ty), Out(1, 12, torch.float32), Out(1, 9, torch.float32)
    U.oidn_ffn_backward(None, 9, None, 9, None, None, None, None, 0, None, 9, w_in.view, b_in.view, w_out.view,
                        b_out.view, 0, 9, 6, U.OIDN_ACT_GELU, dt, 0, None, 0)
    for o in (w_in, w_out, b_in, b_out):
        assert not o.get().any()


def run_ffn(x, w_in, b_in, w_out, b_out, residual, kind, precision, z=None, flags=0, pad=0, stream=None):
    m, d, f, dt = x.shape[0], x.shape[1], w_out.shape[1], DT[precision]
    y = Out(m, d, TORCH[precision], pad)
    ws = bytes_(U.oidn_ffn_workspace_bytes(m, d, f, dt))
    U.oidn_ffn(x, x.stride(0), w_in, b_in, w_out, b_out, residual, residual.stride(0) if residual is not None else 0,
               y.view, y.ld, ptr(z), m, d, f, ACT[kind], dt, flags, ws, ws.numel(), stream=stream)
    return y


FFN = [(1, 1, 1), (1, 64, 80), (2, 2048, 96), (3, 5, 7), (16, 96, 256), (33, 40, 65), (64, 72, 33), (65, 24, 130),
       (130, 100, 64), (300, 64, 200), (600, 16, 1000)]


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, d, f", FFN)
def test_ffn(m, d, f, precision):
    seed = 5 * m + d + 3 * f
    mk, kind, pad = Maker(seed, precision), ACTS[seed % 4], [0, 3, 8][seed % 3]
    x, w_in, w_out = mk.rows(m, d, pad), mk.rows(2 * f, d, 0, d ** -0.5), mk.rows(d, f, 0, f ** -0.5)
    b_in, b_out = (mk.vec(2 * f), mk.vec(d)) if seed % 2 else (None, None)
    residual = mk.rows(m, d, pad) if seed % 3 else None
    z = Out(m, 2 * f, TORCH[precision]) if seed % 4 else None
    y = run_ffn(x, w_in, b_in, w_out, b_out, residual, kind, precision, z, pad=pad)
    g = lambda v: given(v) if v is not None else None  # noqa: E731
    want, want_z = ffn(given(x), given(w_in), g(b_in), given(w_out), g(b_out), g(residual), kind, precision)
    check(y.get(), want, precision, "y")
    if z is not None:
        check(z.get(), want_z, precision, "z")


FFN_BACK = [(1, 1, 1), (1, 64, 80), (3, 5, 7), (33, 40, 65), (64, 72, 32), (130, 24, 100), (513, 96, 256), (1500, 17, 40)]


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, d, f", FFN_BACK)
def test_ffn_backward(m, d, f, precision):
    seed = m + d + f
    mk, kind, pad, dt = Maker(seed, precision), ACTS[seed % 4], [0, 3, 8][m % 3], DT[precision]
    x, dy, z = mk.rows(m, d, pad), mk.rows(m, d, pad), mk.rows(m, 2 * f)
    w_in, w_out = mk.rows(2 * f, d, 0, d ** -0.5), mk.rows(d, f, 0, f ** -0.5)
    extra = mk.rows(m, d, pad) if seed % 2 else None
    ty = TORCH[precision]
    o = [Out(m, d, ty, pad), Out(2 * f, d, ty), Out(d, f, ty), Out(1, 2 * f, torch.float32), Out(1, d, torch.float32)]
    ws = bytes_(U.oidn_ffn_backward_workspace_bytes(m, d, f, dt, 0))
    U.oidn_ffn_backward(dy, dy.stride(0), x, x.stride(0), z, w_in, w_out, extra,
                        extra.stride(0) if extra is not None else 0, o[0].view, o[0].ld, o[1].view, o[3].view,
                        o[2].view, o[4].view, m, d, f, ACT[kind], dt, 0, ws, ws.numel())
    want = ffn_backward(given(dy), given(x), given(z), given(w_in), given(w_out),
                        given(extra) if extra is not None else None, kind, precision)
    for got, w, name in zip(o[:3], want[:3], ["dx", "dw_in", "dw_out"]):
        check(got.get(), w, precision, name)
    check(o[3].get()[0], want[3], "f32", "db_in")
    check(o[4].get()[0], want[4], "f32", "db_out")


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("asked", ["dx", "dw_in", "dw_out", "db_in", "db_out"])
def test_ffn_backward_parts(asked, precision):
    mk, dt, ty = Maker(8, precision), DT[precision], TORCH[precision]
    m, d, f = 90, 48, 72
    x, dy, z = mk.rows(m, d), mk.rows(m, d), mk.rows(m, 2 * f)
    w_in, w_out = mk.rows(2 * f, d), mk.rows(d, f)
    ws = bytes_(U.oidn_ffn_backward_workspace_bytes(m, d, f, dt, 0))

    def run(want):
        o = {"dx": Out(m, d, ty), "dw_in": Out(2 * f, d, ty), "dw_out": Out(d, f, ty),
             "db_in": Out(1, 2 * f, torch.float32), "db_out": Out(1, d, torch.float32)}
        p = {key: v.view if key in want else None for key, v in o.items()}
        U.oidn_ffn_backward(dy, d, x, d, z, w_in, w_out, None, 0, p["dx"], d, p["dw_in"], p["db_in"], p["dw_out"],
                            p["db_out"], m, d, f, U.OIDN_ACT_GELU, dt, 0, ws, ws.numel())
        return {key: v.get() for key, v in o.items()}

    both, some = run(["dx", "dw_in", "dw_out", "db_in", "db_out"]), run([asked])
    for key in both:
        assert torch.equal(some[key], both[key] if key == asked else torch.full_like(both[key], GUARD)), key


# ------------------------------------------------------------- differences
def central(fn, at, direction, eps=1e-5):
    """Directional derivative of fn (to a float) by differences, in 64 bits."""
    return (fn(at + eps * direction) - fn(at - eps * direction)) / (2 * eps)


@pytest.mark.parametrize("kind", ["silu", "gelu", "none"])
def test_gradients_match_differences(kind):
    """<gradient, direction> of the fp32 gradients against the change of sum(dy * y) along the direction.  The
    difference is off by about eps^2 and 2^-53 / eps, below 1e-9 of the scale; the gradients by the fp32 sums."""
    g = torch.Generator().manual_seed(17)
    m, d, f = 37, 24, 40
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, w_in, b_in = rnd(m, d), rnd(2 * f, d) * d ** -0.5, rnd(2 * f) * 0.3
    w_out, b_out, dy = rnd(d, f) * f ** -0.5, rnd(d), rnd(m, d)
    dev = [v.cuda() for v in (x, w_in, b_in, w_out, b_out, dy)]
    X, WI, BI, WO, BO, DY = dev
    z = torch.empty(m, 2 * f, device="cuda")
    run_ffn(X, WI, BI, WO, BO, X, kind, "f32", z)
    o = {"dx": torch.empty_like(X), "w_in": torch.empty_like(WI), "b_in": torch.empty_like(BI),
         "w_out": torch.empty_like(WO), "b_out": torch.empty_like(BO)}
    ws = bytes_(U.oidn_ffn_backward_workspace_bytes(m, d, f, U.OIDN_F32, 0))
    U.oidn_ffn_backward(DY, d, X, d, z, WI, WO, DY, d, o["dx"], d, o["w_in"], o["b_in"], o["w_out"], o["b_out"], m, d,
                        f, ACT[kind], U.OIDN_F32, 0, ws, ws.numel())

    def loss(x, w_in, b_in, w_out, b_out):
        a, b = (x @ w_in.T + b_in).chunk(2, 1)
        h = act(kind, (a, torch.zeros_like(a)))[0] * b
        return float(((h @ w_out.T + b_out + x) * dy.double()).sum())

    base = dict(x=x.double(), w_in=w_in.double(), b_in=b_in.double(), w_out=w_out.double(), b_out=b_out.double())
    for name, got in (("x", o["dx"]), ("w_in", o["w_in"]), ("b_in", o["b_in"]), ("w_out", o["w_out"]), ("b_out", o["b_out"])):
        v = torch.randn(base[name].shape, generator=g, dtype=torch.float64)
        want = central(lambda p: loss(**{**base, name: p}), base[name], v)
        have = float((got.cpu().double() * v).sum())
        scale = float((got.cpu().double() * v).abs().sum())
        assert abs(have - want) <= 1e-5 * scale, (name, have, want, scale)


# ------------------------------------------------------- 8-bit checkpoints
def decode(blob, m, n):
    """(values, scales per column) of a checkpoint from its documented layout, in 64 bits."""
    pitch = -(-n // 32) * 32
    b = blob.cpu()
    codes = b[:m * pitch].view(torch.int8).view(m, pitch).double()
    scales = b[m * pitch:m * pitch + m * pitch // 16].view(torch.bfloat16).view(m, pitch // 32).double()
    s = scales.repeat_interleave(32, 1)
    return (codes * s)[:, :n], s[:, :n], codes


def check_codes(blob, want, m, n, label):
    """Scales within a rounding of max / 127, values within half a step (and the value's own bound)."""
    v, e = want
    values, s, codes = decode(blob, m, n)
    assert not codes[:, n:].any(), "padding is not zero"
    wide = lambda a: torch.nn.functional.pad(a, (0, -n % 32)).view(m, -1, 32).amax(2).repeat_interleave(32, 1)[:, :n]  # noqa: E731
    top, slack = wide(v.abs()), wide(e)
    # the division, the bf16 rounding and the largest value's own error
    assert (torch.abs(s - top / 127) <= (2.0 ** -8 + 2.0 ** -22) * (top + slack) / 127 + slack / 127 + 1e-36).all(), label
    bad = ~((values - v).abs() <= (0.5 + 2.0 ** -14) * s + e + 1e-34)
    assert not bad.any(), (label, int(bad.sum()))


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, n", [(1, 1), (1, 33), (2, 8), (3, 31), (5, 32), (7, 100), (64, 112), (333, 257), (1000, 96)])
def test_checkpoint(m, n, precision):
    mk = Maker(m + n, precision)
    pad = [0, 8, 5][m % 3]
    x = mk.rows(m, n, pad)
    x *= torch.exp(torch.randn(m, 1, generator=mk.g) * 2).cuda().to(x.dtype)
    blob = torch.full((U.oidn_ckpt_bytes(m, n) + 64,), 99, dtype=torch.uint8, device="cuda")
    U.oidn_ckpt_pack(x, x.stride(0), m, n, blob, DT[precision])
    torch.cuda.synchronize()
    pitch = -(-n // 32) * 32
    assert (blob[m * pitch + m * pitch // 16:] == 99).all(), "written past the checkpoint"
    check_codes(blob, given(x), m, n, "pack")
    y = Out(m, n, TORCH[precision], pad)
    U.oidn_ckpt_unpack(blob, m, n, y.view, y.ld, DT[precision])
    values = decode(blob, m, n)[0]
    # a product of an int8 and a bf16 is exact in fp32
    assert torch.equal(y.get().cpu(), values.float().to(TORCH[precision]))


@pytest.mark.parametrize("precision", PRECISIONS)
def test_checkpoint_special_blocks(precision):
    """All zeros, one value, values too small to scale, infinities and NaN: each block on its own."""
    x = torch.randn(8, 96, generator=torch.Generator().manual_seed(2)).to(TORCH[precision])
    x[0] = 0
    x[1, :32] = 0
    x[1, 5] = -3.5
    x[2, 32:64] = 1e-38 if precision != "f16" else 0.0
    x[3, 40] = float("inf")
    x[4, 95] = float("nan")
    x[5, 0] = float("-inf")
    x[6, 64:] = torch.finfo(TORCH[precision]).max
    x[7, :32] = torch.finfo(TORCH[precision]).tiny
    x = x.cuda()
    blob = bytes_(U.oidn_ckpt_bytes(8, 96))
    y = torch.empty_like(x)
    U.oidn_ckpt_pack(x, 96, 8, 96, blob, DT[precision])
    U.oidn_ckpt_unpack(blob, 8, 96, y, 96, DT[precision])
    y = y.float().cpu()
    assert not y[0].any() and not y[1, :32][[k for k in range(32) if k != 5]].any()
    assert abs(y[1, 5] + 3.5) <= 3.5 * 2.0 ** -8
    assert not y[2, 32:64].any() and y[2, :32].any()
    nan = torch.zeros(8, 96, dtype=torch.bool)
    nan[3, 32:64] = nan[4, 64:] = nan[5, :32] = True
    # the largest bf16 or fp16 value may round up past the type when it is unpacked
    assert torch.equal(y.isnan(), nan)
    assert (y[6, 64:] >= torch.finfo(TORCH[precision]).max * (1 - 2.0 ** -7)).all()
    assert (y[7, :32].abs() <= torch.finfo(TORCH[precision]).tiny * (1 + 2.0 ** -7)).all()


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, k, n", [(1, 8, 8), (5, 16, 33), (70, 40, 96), (64, 2048, 40), (300, 24, 200)])
def test_linear_saves_in_8_bits(m, k, n, precision):
    mk = Maker(m + k, precision)
    x, w, bias = mk.rows(m, k), mk.rows(n, k, scale=k ** -0.5), mk.vec(n)
    z = bytes_(U.oidn_ckpt_bytes(m, n))
    y = run_linear(x, w, bias, None, "gelu", precision, z, U.OIDN_Z_CKPT8)
    want, want_z = linear(given(x), given(w), given(bias), None, "gelu")
    check(y.get(), want, precision, "y")
    check_codes(z, want_z, m, n, "z")


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, k, n", [(1, 8, 8), (5, 16, 33), (70, 41, 96), (300, 24, 200)])
def test_linear_backward_from_8_bits(m, k, n, precision):
    mk, dt, ty = Maker(m * n, precision), DT[precision], TORCH[precision]
    x, z, dy, w = mk.rows(m, k), mk.rows(m, n), mk.rows(m, n), mk.rows(n, k)
    x8, z8 = bytes_(U.oidn_ckpt_bytes(m, k)), bytes_(U.oidn_ckpt_bytes(m, n))
    U.oidn_ckpt_pack(x, k, m, k, x8, dt)
    U.oidn_ckpt_pack(z, n, m, n, z8, dt)
    dx, dw, db = Out(m, k, ty), Out(n, k, ty), Out(1, n, torch.float32)
    flags = U.OIDN_X_CKPT8 | U.OIDN_Z_CKPT8
    ws = bytes_(U.oidn_linear_backward_workspace_bytes(m, k, n, U.OIDN_ACT_SILU, dt, flags))
    U.oidn_linear_backward(dy, n, x8, 0, z8, 0, w, k, dx.view, k, dw.view, k, db.view, m, k, n, U.OIDN_ACT_SILU, dt,
                           flags, ws, ws.numel())
    kept_x = stored(given(decode(x8, m, k)[0]), precision)
    want = linear_backward(given(dy), kept_x, given(decode(z8, m, n)[0]), given(w), "silu", precision)
    check(dx.get(), want[0], precision, "dx")
    check(dw.get(), want[1], precision, "dw")
    check(db.get()[0], want[2], "f32", "dbias")


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, d, f", [(1, 8, 8), (5, 16, 33), (70, 41, 96), (513, 96, 256)])
def test_ffn_step_in_8_bits(m, d, f, precision):
    """Forward keeps 8 bits; backward reads them: its gradients are those of the kept values."""
    mk, dt, ty = Maker(m * f, precision), DT[precision], TORCH[precision]
    x, dy = mk.rows(m, d), mk.rows(m, d)
    w_in, w_out = mk.rows(2 * f, d, 0, d ** -0.5), mk.rows(d, f, 0, f ** -0.5)
    one = U.oidn_ckpt_bytes(m, f)
    x8, z8 = bytes_(U.oidn_ckpt_bytes(m, d)), bytes_(2 * one)
    U.oidn_ckpt_pack(x, d, m, d, x8, dt)
    y = run_ffn(x, w_in, None, w_out, None, x, "gelu", precision, z8, U.OIDN_Z_CKPT8)
    want, want_z = ffn(given(x), given(w_in), None, given(w_out), None, given(x), "gelu", precision)
    check(y.get(), want, precision, "y")
    for k, part in enumerate((z8[:one], z8[one:])):
        check_codes(part, (want_z[0][:, k * f:(k + 1) * f], want_z[1][:, k * f:(k + 1) * f]), m, f, "z")
    o = [Out(m, d, ty), Out(2 * f, d, ty), Out(d, f, ty)]
    db = Out(1, 2 * f, torch.float32)
    flags = U.OIDN_X_CKPT8 | U.OIDN_Z_CKPT8
    ws = bytes_(U.oidn_ffn_backward_workspace_bytes(m, d, f, dt, flags))
    U.oidn_ffn_backward(dy, d, x8, 0, z8, w_in, w_out, dy, d, o[0].view, d, o[1].view, db.view, o[2].view, None, m, d,
                        f, U.OIDN_ACT_GELU, dt, flags, ws, ws.numel())
    kept = torch.cat([decode(z8[:one], m, f)[0], decode(z8[one:], m, f)[0]], 1)
    kept_x = stored(given(decode(x8, m, d)[0]), precision)
    grads = ffn_backward(given(dy), kept_x, given(kept), given(w_in), given(w_out), given(dy), "gelu", precision)
    for got, w, name in zip(o, grads[:3], ["dx", "dw_in", "dw_out"]):
        check(got.get(), w, precision, name)
    check(db.get()[0], grads[3], "f32", "db_in")


# ------------------------------------------------ how a program calls them
def test_offsets_past_32_bits():
    """Rows far apart: element offsets pass 2^32 in x, y and z."""
    m, k, n, pitch = 70000, 16, 24, 65600
    buf = torch.empty(m * pitch, dtype=torch.float16, device="cuda")
    x, y = buf.view(m, pitch)[:, :k], buf.view(m, pitch)[:, 64:64 + n]
    g = torch.Generator(device="cuda").manual_seed(1)
    x.copy_(torch.randn(m, k, generator=g, device="cuda"))
    w = torch.randn(n, k, generator=g, device="cuda").half()
    ws = bytes_(U.oidn_linear_workspace_bytes(m, k, n, U.OIDN_F16))
    U.oidn_linear(x, pitch, w, k, None, None, 0, y, pitch, None, 0, m, k, n, U.OIDN_ACT_RELU, U.OIDN_F16, 0, ws,
                  ws.numel())
    check(y, linear(given(x), given(w), None, None, "relu")[0], "f16", "y")
    dw = torch.empty(n, k, dtype=torch.float16, device="cuda")
    db = torch.empty(n, device="cuda")
    ws = bytes_(U.oidn_linear_backward_workspace_bytes(m, k, n, U.OIDN_ACT_NONE, U.OIDN_F16, 0))
    U.oidn_linear_backward(y, pitch, x, pitch, None, 0, None, k, None, k, dw, k, db, m, k, n, U.OIDN_ACT_NONE,
                           U.OIDN_F16, 0, ws, ws.numel())
    want = linear_backward(given(y), given(x), None, given(w), "none", "f16")
    check(dw, want[1], "f16", "dw")
    check(db, want[2], "f32", "dbias")
    blob = bytes_(U.oidn_ckpt_bytes(m, n))
    U.oidn_ckpt_pack(y, pitch, m, n, blob, U.OIDN_F16)
    check_codes(blob, given(y), m, n, "pack")


@pytest.mark.parametrize("precision", PRECISIONS)
def test_calls_repeat_their_bits_on_any_stream(precision):
    """The same call gives the same bits, on another stream too, ordered by events alone."""
    mk = Maker(4, precision)
    m, d, f = 200, 64, 96
    x, w_in, w_out = mk.rows(m, d), mk.rows(2 * f, d), mk.rows(d, f)
    a = run_ffn(x, w_in, None, w_out, None, x, "silu", precision).get().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = run_ffn(x, w_in, None, w_out, None, x, "silu", precision)
        c = run_ffn(x, w_in, None, w_out, None, x, "silu", precision, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b.get()) and torch.equal(a, c.get())


@pytest.mark.parametrize("precision", PRECISIONS)
def test_training_step_in_a_graph(precision):
    """Forward and backward of both operators recorded once and replayed on new inputs, each replay against an eager run."""
    dt, ty = DT[precision], TORCH[precision]
    m, d, f = 4200, 32, 48          # the weight gradients' sums are cut in slices
    g = torch.Generator(device="cuda").manual_seed(9)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda").to(ty)  # noqa: E731
    x, w, w_in, w_out, dy = new(m, d), new(d, d), new(2 * f, d), new(d, f), new(m, d)
    flags = U.OIDN_X_CKPT8 | U.OIDN_Z_CKPT8
    ws = bytes_(max(U.oidn_linear_workspace_bytes(m, d, d, dt), U.oidn_ffn_workspace_bytes(m, d, f, dt),
                    U.oidn_ffn_backward_workspace_bytes(m, d, f, dt, flags),
                    U.oidn_linear_backward_workspace_bytes(m, d, d, U.OIDN_ACT_GELU, dt, 0)))
    hid, z, y, dhid = (torch.empty(m, d, dtype=ty, device="cuda") for _ in range(4))
    h8, z8 = bytes_(U.oidn_ckpt_bytes(m, d)), bytes_(2 * U.oidn_ckpt_bytes(m, f))
    outs = [y, dhid] + [torch.empty_like(v) for v in (x, w, w_in, w_out)] + [torch.empty(n, device="cuda") for n in (d, 2 * f, d)]
    _, _, dx, dw, dw_in, dw_out, db, db_in, db_out = outs

    def step():
        n = ws.numel()
        U.oidn_linear(x, d, w, d, None, None, 0, hid, d, z, d, m, d, d, U.OIDN_ACT_GELU, dt, 0, ws, n)
        U.oidn_ckpt_pack(hid, d, m, d, h8, dt)
        U.oidn_ffn(hid, d, w_in, None, w_out, None, hid, d, y, d, z8, m, d, f, U.OIDN_ACT_SILU, dt, U.OIDN_Z_CKPT8, ws, n)
        U.oidn_ffn_backward(dy, d, h8, 0, z8, w_in, w_out, dy, d, dhid, d, dw_in, db_in, dw_out, db_out, m, d, f,
                            U.OIDN_ACT_SILU, dt, flags, ws, n)
        U.oidn_linear_backward(dhid, d, x, d, z, d, w, d, dx, d, dw, d, db, m, d, d, U.OIDN_ACT_GELU, dt, 0, ws, n)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for v in (x, w, dy):
            v.copy_(new(*v.shape))
        step()
        eager = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o, e)


@pytest.mark.parametrize("precision", ["f16", "bf16"])
@pytest.mark.parametrize("k, n", [(24, 40), (100, 64), (33, 128), (128, 97)])
def test_narrow_linear_backward_of_many_rows(k, n, precision):
    """More blocks of rows than workgroups: each takes several, the last block is ragged."""
    m, dt, ty = 33333, DT[precision], TORCH[precision]
    mk, kind = Maker(k * n, precision), "silu"
    x, w, dy, z = mk.rows(m, k, 8), mk.rows(n, k, 0, k ** -0.5), mk.rows(m, n, 3), mk.rows(m, n)
    dx, dw, db = Out(m, k, ty, 5), Out(n, k, ty, 1), Out(1, n, torch.float32)
    ws = bytes_(U.oidn_linear_backward_workspace_bytes(m, k, n, ACT[kind], dt, 0))
    U.oidn_linear_backward(dy, dy.stride(0), x, x.stride(0), z, n, w, k, dx.view, dx.ld, dw.view, dw.ld, db.view, m, k, n,
                           ACT[kind], dt, 0, ws, ws.numel())
    want = linear_backward(given(dy), given(x), given(z), given(w), kind, precision)
    check(dx.get(), want[0], precision, "dx")
    check(dw.get(), want[1], precision, "dw")
    check(db.get()[0], want[2], "f32", "dbias")


@pytest.mark.parametrize("precision", ["f16", "bf16"])
@pytest.mark.parametrize("m, k, n", [(8191, 65, 96), (8192, 65, 96), (8193, 128, 128), (16385, 112, 72),
                                     (20001, 40, 64), (20001, 70, 64)])
def test_narrow_linear_backward_around_its_limits(m, k, n, precision):
    """Either side of the row count from which wide ones take one pass, of one and of two blocks a workgroup."""
    dt, ty = DT[precision], TORCH[precision]
    mk, kind = Maker(m + k * n, precision), "gelu"
    x, w, dy, z = mk.rows(m, k, 3), mk.rows(n, k, 0, k ** -0.5), mk.rows(m, n, 8), mk.rows(m, n)
    dx, dw, db = Out(m, k, ty, 1), Out(n, k, ty, 5), Out(1, n, torch.float32)
    ws = bytes_(U.oidn_linear_backward_workspace_bytes(m, k, n, ACT[kind], dt, 0))
    U.oidn_linear_backward(dy, dy.stride(0), x, x.stride(0), z, n, w, k, dx.view, dx.ld, dw.view, dw.ld, db.view, m, k, n,
                           ACT[kind], dt, 0, ws, ws.numel())
    want = linear_backward(given(dy), given(x), given(z), given(w), kind, precision)
    check(dx.get(), want[0], precision, "dx")
    check(dw.get(), want[1], precision, "dw")
    check(db.get()[0], want[2], "f32", "dbias")


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, k, n", [(2, 264, 4096), (3, 264, 4095), (3, 267, 4096), (4, 1032, 4099), (4, 72, 4090), (5, 72, 4096)])
def test_few_rows_of_many_columns(m, k, n, precision):
    """Either side of the column and row counts between the two kernels of few rows."""
    mk, kind = Maker(m + k + n, precision), "silu"
    x, w, bias, r = mk.rows(m, k, 3), mk.rows(n, k, 0, k ** -0.5), mk.vec(n), mk.rows(m, n, 1)
    z = Out(m, n, TORCH[precision], 5)
    y = run_linear(x, w, bias, r, kind, precision, z, pad=3, shift=1)
    want, want_z = linear(given(x), given(w), given(bias), given(r), kind)
    check(y.get(), want, precision, "y")
    check(z.get(), want_z, precision, "z")


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, k, n", [(33, 64, 64), (95, 67, 63), (97, 515, 300), (512, 512, 520), (1021, 128, 771),
                                     (2041, 112, 97)])
def test_linear_of_few_tiles(m, k, n, precision):
    """Rows that end inside 32-row and 64-row tiles, sums without and with slices, z in both forms."""
    mk, kind = Maker(m + 3 * k + n, precision), "gelu"
    x, w, bias, r = mk.rows(m, k, 1), mk.rows(n, k, 0, k ** -0.5), mk.vec(n), mk.rows(m, n, 3)
    z = Out(m, n, TORCH[precision], 2)
    y = run_linear(x, w, bias, r, kind, precision, z, pad=1)
    want, want_z = linear(given(x), given(w), given(bias), given(r), kind)
    check(y.get(), want, precision, "y")
    check(z.get(), want_z, precision, "z")
    kept = bytes_(U.oidn_ckpt_bytes(m, n))
    y8 = run_linear(x, w, bias, r, kind, precision, kept, U.OIDN_Z_CKPT8, pad=1)
    assert torch.equal(y8.get(), y.get())
    check_codes(kept, want_z, m, n, "z in 8 bits")
