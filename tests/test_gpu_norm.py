"""The norms around a block and dropout on the GPU against their definitions in
64 bits, with error bounds carried through every step (block_reference)."""
import pytest
import torch

import block_reference as R
import unet_x3_convolution_amd as U
from dense_reference import TORCH, check, given
from helpers import DT, torch_cuda
from test_gpu_dense import GUARD, PRECISIONS, Maker, Out, bytes_

pytestmark = pytest.mark.gpu

KIND = {"none": U.OIDN_NORM_NONE, "rms": U.OIDN_NORM_RMS, "layer": U.OIDN_NORM_LAYER}
EPS = 1e-5
EPS32 = float(torch.tensor(EPS))      # as the kernels take it
SUMS = ("dweight", "dshift", "dnext_weight", "dnext_shift")


@pytest.fixture(autouse=True)
def gpu():
    torch_cuda()


def state(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def wide(v):
    return None if v is None else v.cpu().double()


def pitch(v):
    return 0 if v is None else v.stride(0)


# ---------------------------------------------------------------- dropout
@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("m, n, p", [(1, 1, 0.5), (1, 7, 0.1), (3, 8, 0.9), (5, 9, 0.5), (17, 33, 0.25), (64, 96, 0.1),
                                     (300, 112, 0.5), (7, 4099, 0.1), (2, 40, 1.0), (9, 24, 0.0), (9, 24, 1e-6)])
def test_dropout(m, n, p, precision):
    """Which elements are kept is equal to the definition's, and each value is off by its roundings alone."""
    mk, pad, shift = Maker(m + n, precision), [0, 3, 8][n % 3], n % 2
    x = mk.rows(m, n, pad, shift=shift)
    residual = mk.rows(m, n, pad) if m % 2 else None
    seed, offset = -(m << 40) - 12345, (n << 33) + 77
    keep = R.kept(m, n, p, seed, offset)
    y = Out(m, n, TORCH[precision], pad, shift)
    U.oidn_dropout(x, x.stride(0), residual, pitch(residual), y.view, y.ld, m, n, p, state(seed, offset), DT[precision])
    want = R.scaled(given(x), keep)
    if residual is not None:
        want = R.add(want, given(residual))
    check(y.get(), want, precision, "y")
    if residual is None:
        assert torch.equal(y.get().cpu() != 0, (keep != 0) & (x.cpu() != 0))


@pytest.mark.parametrize("precision", PRECISIONS)
def test_dropped_places_may_hold_anything(precision):
    m, n, p = 40, 50, 0.5
    x = torch.full((m, n), float("nan"), dtype=TORCH[precision], device="cuda")
    x[::2] = float("inf")
    y = torch.empty_like(x)
    U.oidn_dropout(x, n, None, 0, y, n, m, n, p, state(1, 2), DT[precision])
    keep = R.kept(m, n, p, 1, 2) != 0
    assert (y.cpu()[~keep] == 0).all() and not y.cpu()[keep].isfinite().any()


def test_dropout_in_place_and_its_gradient():
    """y in x's place, then in the residual's; the gradient's mask is the forward pass's, at any pitch and type."""
    mk = Maker(4, "f32")
    m, n, p, s = 33, 70, 0.3, state(5, 6)
    x, r = mk.rows(m, n), mk.rows(m, n)
    want = torch.empty_like(x)
    U.oidn_dropout(x, n, r, n, want, n, m, n, p, s, U.OIDN_F32)
    a, b = x.clone(), r.clone()
    U.oidn_dropout(a, n, r, n, a, n, m, n, p, s, U.OIDN_F32)
    U.oidn_dropout(x, n, b, n, b, n, m, n, p, s, U.OIDN_F32)
    assert torch.equal(a, want) and torch.equal(b, want)
    keep = R.kept(m, n, p, 5, 6)
    for precision in PRECISIONS:
        dy = torch.ones(m, n + 5, dtype=TORCH[precision], device="cuda")[:, :n]
        dx = torch.empty(m, n, dtype=TORCH[precision], device="cuda")
        U.oidn_dropout(dy, n + 5, None, 0, dx, n, m, n, p, s, DT[precision])
        assert torch.equal(dx.cpu(), keep.to(TORCH[precision]))


def test_dropout_share():
    """The share kept is p's: within five standard deviations of 2^22 independent draws, and so are the pairs of
    neighbours (in a row, in a column) that are both kept."""
    m, n, p = 2048, 2048, 0.25
    x = torch.ones(m, n, device="cuda")
    y = torch.empty_like(x)
    U.oidn_dropout(x, n, None, 0, y, n, m, n, p, state(11, 12), U.OIDN_F32)
    k = (y != 0).double().cpu()
    for share, want in ((k.mean(), 0.75), ((k[:, 1:] * k[:, :-1]).mean(), 0.75 ** 2), ((k[1:] * k[:-1]).mean(), 0.75 ** 2)):
        # neighbouring pairs share elements: their mean varies at most three times as much
        assert abs(float(share) - want) < 5 * (3 * want * (1 - want) / (m * (n - 1))) ** 0.5
    assert float(y.max()) == pytest.approx(4 / 3, rel=2 ** -23)


# ------------------------------------------------------------------- norms
# rows, columns: single ones, sizes around 8, a wave's and a workgroup's columns, rows past what registers hold
SIZES = [(1, 1), (3, 1), (1, 8), (5, 7), (70, 9), (130, 31), (64, 32), (67, 33), (300, 64), (33, 96), (41, 112),
         (20, 128), (19, 200), (9, 257), (7, 512), (6, 513), (5, 1000), (9, 1024), (4, 2048), (5, 2056), (3, 4096),
         (2, 4099), (3, 8192), (2, 8193), (2, 20001)]


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("m, n", SIZES)
def test_norm(m, n, kind, precision):
    mk, pad, shift = Maker(m + n, precision), [0, 3, 8][(m + n) % 3], n % 2
    x = mk.rows(m, n, pad, 3.0, shift=shift)
    weight, extra = (mk.vec(n) + 1 if m % 2 else None), (mk.vec(n) if n % 4 else None)
    y = Out(m, n, TORCH[precision], pad, shift)
    U.oidn_norm(x, x.stride(0), weight, extra, y.view, y.ld, m, n, KIND[kind], EPS, DT[precision])
    check(y.get(), R.before(given(x), wide(weight), wide(extra), kind, EPS32), precision, "y")


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("n", [24, 200, 1500, 9000])
def test_rows_of_zeros_and_equal_values(n, precision):
    """A row of zeros gives the shift; equal values give it with the layer norm, and 1 / sqrt(1 + eps / x^2) without."""
    x = torch.zeros(4, n, dtype=TORCH[precision], device="cuda")
    x[1], x[2], x[3] = 2.0, -0.25, 2.0 ** -14
    for kind in ("rms", "layer"):
        y = torch.empty_like(x)
        shift = torch.full((n,), 0.5, device="cuda")
        U.oidn_norm(x, n, None, shift, y, n, 4, n, KIND[kind], EPS, DT[precision])
        check(y, R.before(given(x), None, wide(shift), kind, EPS32), precision, kind)
        assert (y[0] == 0.5).all()


@pytest.mark.parametrize("n", [40, 300, 3000, 10000])
def test_layer_norm_far_from_zero(n):
    """A mean 10^4 times the spread: the deviations are formed before they are squared."""
    g = torch.Generator().manual_seed(n)
    x = (torch.randn(5, n, generator=g) + 1e4).cuda()
    y = torch.empty_like(x)
    U.oidn_norm(x, n, None, None, y, n, 5, n, U.OIDN_NORM_LAYER, EPS, U.OIDN_F32)
    check(y, R.before(given(x), None, None, "layer", EPS32), "f32", "y")
    d = x.cpu().double() - x.cpu().double().mean(1, keepdim=True)
    assert (y.cpu().double() - d / d.square().mean(1, keepdim=True).sqrt()).abs().max() < 0.01


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("n", [12, 100, 700, 5000, 9001])
def test_rows_stay_apart(n, precision):
    """NaN and infinities stay in their row, and what lies past the rows' ends reaches none."""
    mk, m = Maker(n, precision), 21
    x, o = mk.rows(m, n, 5), mk.rows(m, n, 5)
    x[3, n // 2], o[11, n - 1], x[20, 0] = float("nan"), float("inf"), float("-inf")
    u, v = (torch.empty(m, n, dtype=x.dtype, device="cuda") for _ in range(2))
    U.oidn_norm_residual(o, n + 5, None, None, None, 0, 0, x, n + 5, 1.0, 0.0, None, u, n, None, None, v, n, m, n,
                         U.OIDN_NORM_RMS, U.OIDN_NORM_LAYER, EPS, DT[precision])
    bad = torch.zeros(m, dtype=torch.bool)
    bad[[3, 11, 20]] = True
    assert v[~bad].isfinite().all() and u[~bad].isfinite().all() and v[bad].isnan().any(1).all()


def residual_case(m, n, kind, following, precision, seed):
    """Inputs of the residual form: what is there goes by the seed."""
    mk = Maker(seed, precision)
    pad = [0, 3, 8][seed % 3]
    c = dict(m=m, n=n, kind=kind, following=following, precision=precision, pad=pad, scale=[1.0, 0.7][seed % 2],
             p=[0.0, 0.2, 0.5][seed % 3], seed=seed * 1000003, offset=-seed)
    rows = lambda: mk.rows(m, n, pad)  # noqa: E731
    c.update(o=rows(), x=rows(), weight=mk.vec(n) + 1 if seed % 4 else None, shift=mk.vec(n) if seed % 3 else None)
    c["gate_rows"] = [0, 1, 3, m, m + 5, max(1, m // 2)][seed % 6]
    c["gate"] = torch.randn(-(-m // c["gate_rows"]), n + pad, generator=mk.g).cuda()[:, :n] if c["gate_rows"] else None
    c.update(next_weight=mk.vec(n) + 1 if seed % 5 else None, next_shift=mk.vec(n) if seed % 2 else None)
    c["rng"] = state(c["seed"], c["offset"])
    c["keep"] = R.kept(m, n, c["p"], c["seed"], c["offset"])
    return c


def run_residual(c, **kw):
    m, n, ty = c["m"], c["n"], TORCH[c["precision"]]
    u, v = Out(m, n, ty, c["pad"]), Out(m, n, ty, c["pad"]) if c["following"] != "none" else None
    U.oidn_norm_residual(c["o"], c["o"].stride(0), c["weight"], c["shift"], c["gate"], pitch(c["gate"]), c["gate_rows"],
                         c["x"], c["x"].stride(0), c["scale"], c["p"], c["rng"], u.view, u.ld, c["next_weight"],
                         c["next_shift"], v.view if v else None, v.ld if v else 0, m, n, KIND[c["kind"]],
                         KIND[c["following"]], EPS, DT[c["precision"]], **kw)
    return u, v


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("kind", R.NORMS)
@pytest.mark.parametrize("m, n", SIZES)
def test_norm_residual(m, n, kind, precision):
    seed = 3 * m + n + R.NORMS.index(kind)
    following = R.NORMS[(m + n) % 3]
    c = residual_case(m, n, kind, following, precision, seed)
    u, v = run_residual(c)
    want = R.after(given(c["o"]), wide(c["weight"]), wide(c["shift"]), wide(c["gate"]), c["gate_rows"], given(c["x"]),
                   c["scale"], c["keep"], kind, EPS32)
    check(u.get(), want, precision, "u")
    if v:     # of u as stored
        check(v.get(), R.before(given(u.get()), wide(c["next_weight"]), wide(c["next_shift"]), following, EPS32),
              precision, "v")


@pytest.mark.parametrize("n", [40, 500, 3000, 9000])
@pytest.mark.parametrize("where", ["x", "o"])
def test_norm_residual_in_place(n, where):
    c = residual_case(37, n, "layer", "rms", "bf16", 7)
    c["pad"] = 0
    c["o"], c["x"] = c["o"].contiguous(), c["x"].contiguous()
    want = [t.get().clone() for t in run_residual(c)]
    v = torch.empty_like(c["x"])
    U.oidn_norm_residual(c["o"], n, c["weight"], c["shift"], c["gate"], pitch(c["gate"]), c["gate_rows"], c["x"], n,
                         c["scale"], c["p"], c["rng"], c[where], n, c["next_weight"], c["next_shift"], v, n, 37, n,
                         KIND["layer"], KIND["rms"], EPS, U.OIDN_BF16)
    assert torch.equal(c[where], want[0]) and torch.equal(v, want[1])
    y = c["x"].clone()
    U.oidn_norm(y, n, None, None, y, n, 37, n, KIND["layer"], EPS, U.OIDN_BF16)
    other = torch.empty_like(y)
    U.oidn_norm(c["x"], n, None, None, other, n, 37, n, KIND["layer"], EPS, U.OIDN_BF16)
    assert torch.equal(y, other)


# --------------------------------------------------------------- gradients
def back_case(m, n, kind, following, precision, seed):
    c = residual_case(m, n, kind, following, precision, seed)
    mk = Maker(seed + 1, precision)
    rows = lambda: mk.rows(m, n, c["pad"])  # noqa: E731
    c.update(u=rows(), dv=rows() if following != "none" else None,
             du=rows() if following == "none" or seed % 7 else None)
    return c


def run_back(c, asked=None, ws=None, **kw):
    m, n, ty, pad = c["m"], c["n"], TORCH[c["precision"]], c["pad"]
    dt, following = DT[c["precision"]], c["following"] != "none"
    outs = {"dx": Out(m, n, ty, pad), "d_o": Out(m, n, ty, pad), "dweight": Out(1, n, torch.float32),
            "dshift": Out(1, n, torch.float32)}
    if c["gate"] is not None:
        outs["dgate"] = Out(c["gate"].shape[0], n, torch.float32, pad)
    if following:
        outs.update(dnext_weight=Out(1, n, torch.float32), dnext_shift=Out(1, n, torch.float32))
    at = {k: o.view if asked is None or k in asked else None for k, o in outs.items()}
    if ws is None:
        ws = bytes_(U.oidn_norm_residual_backward_workspace_bytes(m, n, c["gate_rows"], dt))
    U.oidn_norm_residual_backward(
        c["du"], pitch(c["du"]), c["dv"], pitch(c["dv"]), c["o"], c["o"].stride(0), c["weight"], c["shift"], c["gate"],
        pitch(c["gate"]), c["gate_rows"], c["u"] if following else None, c["u"].stride(0), c["scale"], c["p"], c["rng"],
        c["next_weight"], at["dx"], n + pad, at["d_o"], n + pad, at.get("dgate"), n + pad, at["dweight"], at["dshift"],
        at.get("dnext_weight"), at.get("dnext_shift"), m, n, KIND[c["kind"]], KIND[c["following"]], EPS, dt, ws,
        ws.numel(), **kw)
    return outs


def reference(c):
    return R.back(given(c["du"]) if c["du"] is not None else None, given(c["dv"]) if c["dv"] is not None else None,
                  given(c["o"]), given(c["u"]), wide(c["weight"]), wide(c["shift"]), wide(c["gate"]), c["gate_rows"],
                  c["scale"], c["keep"], c["kind"], wide(c["next_weight"]), c["following"], EPS32)


# the same and lengths that take several chunks of rows
BACK = SIZES + [(2500, 17), (700, 100), (4100, 33), (150, 1032)]


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("kind", R.NORMS)
@pytest.mark.parametrize("m, n", BACK)
def test_norm_residual_backward(m, n, kind, precision):
    seed = m + 2 * n + R.NORMS.index(kind)
    c = back_case(m, n, kind, R.NORMS[(m + n + seed) % 3], precision, seed)
    want, outs = reference(c), run_back(c)
    for name, o in outs.items():
        if name in ("dx", "d_o"):
            check(o.get(), want[name], precision, name)
        else:
            check(o.get() if name == "dgate" else o.get()[0], want[name], "f32", name)


@pytest.mark.parametrize("gate_rows", [1, 2, 15, 16, 17, 100, 333, 1000, 1500])
@pytest.mark.parametrize("m, n", [(1000, 24), (333, 520), (120, 4800), (50, 8200)])
def test_gate_groups(m, n, gate_rows):
    """Groups shorter and longer than a workgroup's rows, the last one short."""
    c = back_case(m, n, "rms", "rms", "f32", 25)
    c["gate_rows"], c["pad"] = gate_rows, 3
    c["gate"] = torch.randn(-(-m // gate_rows), n + 3, device="cuda")[:, :n]
    want, outs = reference(c), run_back(c)
    check(outs["dgate"].get(), want["dgate"], "f32", "dgate")
    check(outs["dweight"].get()[0], want["dweight"], "f32", "dweight")
    check(outs["d_o"].get(), want["d_o"], "f32", "d_o")


@pytest.mark.parametrize("m, n, gate_rows", [(3001, 24, 1), (3001, 24, 3), (3001, 24, 5), (2600, 30, 5), (8193, 31, 16),
                                             (1201, 96, 2), (1201, 200, 1), (1201, 200, 2), (1101, 512, 1),
                                             (512 * 4, 64, 4), (513 * 4, 64, 4)])
def test_many_gate_groups(m, n, gate_rows):
    test_gate_groups(m, n, gate_rows)


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("m, n", BACK)
def test_norm_backward(m, n, kind, precision):
    mk, dt, ty, pad = Maker(m + n, precision), DT[precision], TORCH[precision], [0, 3, 8][n % 3]
    x, dy = mk.rows(m, n, pad, 2.0), mk.rows(m, n, pad)
    extra = mk.rows(m, n, pad) if m % 2 else None
    weight = mk.vec(n) + 1 if n % 3 else None
    dx, dw, ds = Out(m, n, ty, pad), Out(1, n, torch.float32), Out(1, n, torch.float32)
    ws = bytes_(U.oidn_norm_backward_workspace_bytes(m, n, dt))
    U.oidn_norm_backward(dy, dy.stride(0), x, x.stride(0), weight, extra, pitch(extra), dx.view, dx.ld, dw.view, ds.view,
                         m, n, KIND[kind], EPS, dt, ws, ws.numel())
    want = R.back(given(extra) if extra is not None else None, given(dy), None, given(x), None, None, None, 0, 1.0, None,
                  "none", wide(weight), kind, EPS32)
    check(dx.get(), want["dx"], precision, "dx")
    check(dw.get()[0], want["dnext_weight"], "f32", "dweight")
    check(ds.get()[0], want["dnext_shift"], "f32", "dshift")
    if extra is not None:      # add in dx's place
        again = Out(m, n, ty, pad)
        again.view[:, :n] = extra
        U.oidn_norm_backward(dy, dy.stride(0), x, x.stride(0), weight, again.view, again.ld, again.view, again.ld,
                             dw.view, ds.view, m, n, KIND[kind], EPS, dt, ws, ws.numel())
        assert torch.equal(again.get(), dx.get())
        check(dw.get()[0], want["dnext_weight"], "f32", "dweight")


@pytest.mark.parametrize("n", [40, 700, 1600, 4800, 9000])
@pytest.mark.parametrize("asked", ["dx", "d_o", "dgate", "dweight", "dshift", "dnext_weight", "dnext_shift", "nothing"])
def test_backward_parts(asked, n):
    """Each gradient alone: the same bits as all at once."""
    c = back_case(130, n, "layer", "rms", "bf16", 26)
    assert c["gate"] is not None and c["p"]
    both, some = run_back(c), run_back(c, [asked])
    for name, o in both.items():
        want = o.get() if name == asked else torch.full_like(o.get(), GUARD)
        assert torch.equal(some[name].get(), want), name


@pytest.mark.parametrize("n", [40, 700, 9000])
def test_dropped_rows_have_no_gradient(n):
    """p = 1: the branch is cut off, whatever it holds; u is the scaled input."""
    c = back_case(20, n, "none", "rms", "f32", 26)
    c.update(p=1.0, keep=torch.zeros(20, n, dtype=torch.float64))
    c["o"][3, 5] = float("nan")
    u, _ = run_residual(c)
    assert torch.equal(u.get(), c["x"] * c["scale"])
    outs = run_back(c)
    for name in ("d_o", "dgate", "dweight", "dshift"):
        assert not outs[name].get().any(), name
    check(outs["dx"].get(), reference(c)["dx"], "f32", "dx")


def test_gradients_of_no_rows_are_zero():
    dw, ds = Out(1, 12, torch.float32), Out(1, 12, torch.float32)
    U.oidn_norm_backward(None, 12, None, 12, None, None, 0, None, 12, dw.view, ds.view, 0, 12, KIND["rms"], EPS,
                         U.OIDN_F16, None, 0)
    assert not dw.get().any() and not ds.get().any()
    four = [Out(1, 9, torch.float32) for _ in SUMS]
    U.oidn_norm_residual_backward(None, 9, None, 9, None, 9, None, None, None, 0, 0, None, 9, 1.0, 0.0, None, None, None,
                                  9, None, 9, None, 0, *[o.view for o in four], 0, 9, KIND["rms"], KIND["rms"], EPS,
                                  U.OIDN_F32, None, 0)
    assert not any(o.get().any() for o in four)


@pytest.mark.parametrize("kind, following", [("rms", "layer"), ("layer", "rms"), ("none", "layer")])
def test_gradients_match_differences(kind, following):
    """<gradient, direction> of the fp32 gradients against the change of sum(du u + dv v) along the direction.  The
    difference is off by about eps^2 and 2^-53 / eps; the gradients by the fp32 sums."""
    m, n = 29, 44
    c = back_case(m, n, kind, following, "f32", 20)
    c.update(p=0.2, keep=R.kept(m, n, 0.2, c["seed"], c["offset"]), weight=torch.rand(n).cuda() + 0.5,
             shift=torch.randn(n).cuda(), next_weight=torch.rand(n).cuda() + 0.5, next_shift=torch.randn(n).cuda())
    assert c["gate"] is not None and c["du"] is not None
    u, _ = run_residual(c)
    c["u"] = u.get().clone()
    outs = run_back(c)
    base = dict(o=wide(c["o"]), x=wide(c["x"]), weight=wide(c["weight"]), shift=wide(c["shift"]), gate=wide(c["gate"]),
                next_weight=wide(c["next_weight"]), next_shift=wide(c["next_shift"]))

    def loss(**kw):
        b = dict(base, **kw)
        u = R.after(R.exact(b["o"]), b["weight"], b["shift"], b["gate"], c["gate_rows"], R.exact(b["x"]), c["scale"],
                    c["keep"], kind, EPS32)[0]
        v = R.before(R.exact(u), b["next_weight"], b["next_shift"], following, EPS32)[0]
        return float((wide(c["du"]) * u + wide(c["dv"]) * v).sum())

    g = torch.Generator().manual_seed(3)
    for name, out in (("o", "d_o"), ("x", "dx"), ("weight", "dweight"), ("shift", "dshift"), ("gate", "dgate"),
                      ("next_weight", "dnext_weight"), ("next_shift", "dnext_shift")):
        way = torch.randn(base[name].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        slope = (loss(**{name: base[name] + h * way}) - loss(**{name: base[name] - h * way})) / (2 * h)
        got = outs[out].get().cpu().double().view(base[name].shape)
        # fp32 gradients: relative 2^-24 a rounding, some tens of them, over the sum's terms
        assert abs(float((got * way).sum()) - slope) <= 64 * 2.0 ** -24 * float((got * way).abs().sum()) + 1e-7


# -------------------------------------------------- streams, graphs, reuse
def test_another_stream_and_the_same_bits_again():
    c = back_case(513, 96, "layer", "rms", "f16", 44)
    want_u, want_v = [t.get().clone() for t in run_residual(c)]
    want = {k: o.get().clone() for k, o in run_back(c).items()}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        u, v = run_residual(c, stream=stream)
        outs = run_back(c, stream=stream)
        stream.synchronize()
        assert torch.equal(u.get(), want_u) and torch.equal(v.get(), want_v)
        assert all(torch.equal(o.get(), want[k]) for k, o in outs.items())


@pytest.mark.parametrize("m, n", [(300, 96), (40, 1500), (5, 9000)])
def test_graph_replays_drop_other_elements(m, n):
    """A captured forward and backward pass, replayed with the state changed in between: each replay is the eager
    result of that state, and of inputs changed in place."""
    c = back_case(m, n, "rms", "layer", "bf16", 26)
    c.update(p=0.3)
    ws = bytes_(U.oidn_norm_residual_backward_workspace_bytes(m, n, c["gate_rows"], DT["bf16"]))
    run_residual(c), run_back(c, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        u, v = run_residual(c)
        outs = run_back(c, ws=ws)
        c["rng"][1].add_(1)
    first = int(c["rng"][1])
    for k in range(4):
        c["o"].copy_(torch.randn(m, n, device="cuda"))
        torch.cuda.synchronize()
        at = int(c["rng"][1])
        assert at == first + k
        graph.replay()
        torch.cuda.synchronize()
        now = {**{name: o.get().clone() for name, o in outs.items()}, "u": u.get().clone(), "v": v.get().clone()}
        c["rng"][1] = at
        eager_u, eager_v = run_residual(c)
        eager = {**{name: o.get() for name, o in run_back(c).items()}, "u": eager_u.get(), "v": eager_v.get()}
        c["rng"][1] = at + 1
        assert all(torch.equal(now[name], eager[name]) for name in now)
