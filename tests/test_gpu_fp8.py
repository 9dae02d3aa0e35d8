"""The dense layer in 8-bit floating point on the GPU: codes bit for bit, products and
gradients against their definitions in 64 bits with error bounds (fp8_reference)."""
import pytest
import torch

import fp8_reference as R
import unet_x3_convolution_amd as U
from dense_reference import ACTS, TORCH, act, add, check, given, mul, slope, total
from helpers import DT, torch_cuda
from test_gpu_dense import ACT, GUARD, PRECISIONS, Maker, Out, bytes_, ptr

pytestmark = pytest.mark.gpu
HALVES = ["f16", "bf16"]


@pytest.fixture(autouse=True)
def gpu():
    torch_cuda()


def packed(x, flags=0, turned=False, rows=True, dt=None):
    m, n = x.shape
    dt = {torch.float32: U.OIDN_F32, torch.float16: U.OIDN_F16, torch.bfloat16: U.OIDN_BF16}[x.dtype]
    a = bytes_(U.oidn_fp8_bytes(m, n)) if rows else None
    b = bytes_(U.oidn_fp8_bytes(n, m)) if turned else None
    U.oidn_fp8_pack(x, x.stride(0), m, n, a, b, dt, flags)
    return (a, b) if rows and turned else a if rows else b


def unpacked(blob, m, n, precision="f32"):
    y = Out(m, n, TORCH[precision], 3)
    U.oidn_fp8_unpack(blob, m, n, y.view, y.ld, DT[precision])
    return y.get()


def fields(blob, m, n):
    """Codes and scales as they lie in the buffer."""
    blocks = -(-n // 128)
    words = -(-blocks // 4) * 4
    b = blob.cpu()
    return b[:m * blocks * 128].view(m, blocks * 128), b[m * blocks * 128:m * (blocks * 128 + words)].view(m, words)[:, :blocks]


# ------------------------------------------------------------ packed form
PACK = [(1, 1), (1, 128), (1, 129), (3, 7), (5, 515), (64, 96), (127, 130), (128, 128), (129, 127), (300, 384), (260, 1000)]


@pytest.mark.parametrize("precision", PRECISIONS)
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("m, n", PACK)
def test_pack(m, n, square, precision):
    """Both forms bit for bit: codes, padding, scales; and their values."""
    mk = Maker(m + n, precision)
    x = mk.rows(m, n, [0, 3, 8][n % 3], shift=m % 2)
    x *= torch.exp(2 * torch.randn(m, 1, generator=mk.g)).to(x.dtype).cuda()
    flags = U.OIDN_FP8_SQUARE if square else 0
    both = packed(x, flags, turned=True)
    v = x.cpu().double()
    for blob, t, alone in ((both[0], v, packed(x, flags)), (both[1], v.T.contiguous(), packed(x, flags, True, False))):
        want, power = R.code(t, square)
        for b in (blob, alone):
            codes, scales = fields(b, *t.shape)
            assert torch.equal(scales.long() - 127, power)
            got = codes.view(torch.float8_e4m3fn).double()
            assert not got[:, t.shape[1]:].any()
            scaled = got[:, :t.shape[1]] * torch.ldexp(torch.ones(1, dtype=torch.float64),
                                                       power.repeat_interleave(128, 1)[:, :t.shape[1]])
            assert torch.equal(scaled, want)
        assert torch.equal(unpacked(blob, *t.shape).cpu().double(), want)
    if square:
        assert torch.equal(unpacked(both[0], m, n), unpacked(both[1], n, m).T)


def test_pack_borders():
    """Blocks of zeros, of one value, largest values at and past 448 2^k, the ends of float32, negative zeros."""
    x = torch.zeros(16, 128, device="cuda")
    top = [0.0, 448.0, 448.00003, 447.9, 1.75 * 2.0 ** -20, 1.7500002 * 2.0 ** -20, 3.4028234e38, 2.0 ** -126, 1e-44, 1e-30,
           2.0 ** -112, 464.0, 2.0 ** -111]
    for i, t in enumerate(top):
        x[i, 3 * i] = t
        x[i, 3 * i + 1] = -t / 3
        x[i, 100] = t * 2.0 ** -16
    x[13] = 5.0
    x[14] = -0.0
    want, power = R.code(x.cpu().double())
    blob = packed(x)
    _, scales = fields(blob, 16, 128)
    assert torch.equal(scales.long() - 127, power)
    got = unpacked(blob, 16, 128).cpu().double()
    # float32's own end: the rounding carries 2^128 (1 - 2^-24) to 2^128, read back as the largest value
    want = want.clamp(-float(torch.finfo(torch.float32).max), float(torch.finfo(torch.float32).max))
    # float32's subnormals may be read as zeros: half of 2^-126 at most
    assert ((got - want).abs() <= 2.0 ** -127).all()


@pytest.mark.parametrize("precision", PRECISIONS)
def test_not_finite_becomes_nan_alone(precision):
    x = torch.randn(130, 260, device="cuda").to(TORCH[precision])
    x[3, 5], x[64, 200], x[129, 259] = float("nan"), float("inf"), float("-inf")
    for flags in (0, U.OIDN_FP8_SQUARE):
        a, b = packed(x, flags, turned=True)
        for blob, t in ((a, x), (b, x.T)):
            got = unpacked(blob, *t.shape).cpu().double()
            want, _ = R.code(t.cpu().double().contiguous(), bool(flags))
            assert torch.equal(got.isnan(), want.isnan()) and int(got.isnan().sum()) == 3
            assert torch.equal(got[~got.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("precision", PRECISIONS)
def test_finite_reads_back_finite(precision):
    most = float(torch.finfo(TORCH[precision]).max)
    x = torch.full((2, 40), most, device="cuda").to(TORCH[precision])
    x[1] = -x[1]
    assert torch.equal(unpacked(packed(x), 2, 40, precision), x)


# ------------------------------------------------------------------ layer
def run_linear(x, w8, n, bias, residual, kind, precision, z=None, flags=0, pad=0, shift=0, m=None, k=None, stream=None):
    m, k, dt = m or x.shape[0], k or x.shape[1], DT[precision]
    y = Out(m, n, TORCH[precision], pad, shift)
    ws = bytes_(U.oidn_linear_fp8_workspace_bytes(m, k, n, dt, flags))
    U.oidn_linear_fp8(x, x.stride(0) if not flags & U.OIDN_X_FP8 else 0, w8, bias, residual,
                      residual.stride(0) if residual is not None else 0, y.view, y.ld, ptr(z),
                      z.ld if isinstance(z, Out) else 0, m, k, n, ACT[kind], dt, flags, ws, ws.numel(), stream=stream)
    return y


def reference(x, w, bias, residual, kind):
    z = R.product(R.coded(given(x)), R.coded(given(w), True))
    if bias is not None:
        z = add(z, (bias.cpu().double().expand_as(z[0]), torch.zeros_like(z[0])))
    y = act(kind, z)
    return (add(y, given(residual)) if residual is not None else y), z


# m, k, n: single elements and rows, sizes around blocks, tiles and fragments, long sums that are cut in slices
LINEAR = [(1, 1, 1), (1, 8, 8), (1, 1000, 300), (2, 4096, 40), (3, 5, 7), (5, 64, 64), (8, 512, 96), (16, 64, 32),
          (17, 33, 130), (31, 200, 64), (33, 128, 64), (63, 129, 33), (64, 1024, 64), (65, 640, 48), (100, 96, 384),
          (129, 130, 127), (257, 72, 264), (300, 1000, 8), (70, 8192, 72), (640, 40, 520), (1025, 24, 1025)]


@pytest.mark.parametrize("precision", HALVES)
@pytest.mark.parametrize("m, k, n", LINEAR)
def test_linear(m, k, n, precision):
    seed = m * 7 + k * 3 + n
    mk, kind = Maker(seed, precision), ACTS[seed % 4]
    pad, shift = [(0, 0), (8, 0), (3, 0), (8, 1)][(m + k) % 4]
    x, w = mk.rows(m, k, pad, shift=shift), mk.rows(n, k, pad, k ** -0.5)
    bias = mk.vec(n) if seed % 3 else None
    residual = mk.rows(m, n, pad, shift=shift) if seed % 2 else None
    z = Out(m, n, TORCH[precision], pad) if seed % 5 else None
    w8 = packed(w, U.OIDN_FP8_SQUARE)
    y = run_linear(x, w8, n, bias, residual, kind, precision, z, pad=pad, shift=shift)
    want, want_z = reference(x, w, bias, residual, kind)
    check(y.get(), want, precision, "y")
    if z is not None:
        check(z.get(), want_z, precision, "z")
    # x packed beforehand
    again = run_linear(packed(x), w8, n, bias, residual, kind, precision, flags=U.OIDN_X_FP8, pad=pad, m=m, k=k)
    check(again.get(), want, precision, "y from packed x")


@pytest.mark.parametrize("precision", HALVES)
@pytest.mark.parametrize("m, k, n", [(2113, 136, 2310), (1500, 1100, 1290), (4100, 260, 4200)])
def test_linear_many_tiles(m, k, n, precision):
    """More tiles than compute units, ragged in both directions, in tiles of each size."""
    mk = Maker(5, precision)
    x, w, bias, r = mk.rows(m, k), mk.rows(n, k, scale=k ** -0.5), mk.vec(n), mk.rows(m, n)
    y = run_linear(x, packed(w, U.OIDN_FP8_SQUARE), n, bias, r, "gelu", precision)
    check(y.get(), reference(x, w, bias, r, "gelu")[0], precision, "y")


def whole(g, *shape, most=8):
    return torch.randint(-most, most + 1, shape, generator=g).float()


@pytest.mark.parametrize("m, k, n", [(1, 64, 48), (16, 300, 33), (40, 130, 70), (200, 513, 90), (300, 256, 264)])
def test_whole_numbers_are_exact(m, k, n):
    """Small whole numbers are codes, and sums of their products are exact in any order: y, dx and dw bit for bit, and
    the change of sum(dy y) along a whole-numbered step is the gradients' product with it."""
    g = torch.Generator().manual_seed(m)
    x, w, dy, step_x, step_w = whole(g, m, k), whole(g, n, k, most=1), whole(g, m, n, most=1), whole(g, m, k, most=1), whole(g, n, k, most=1)
    dev = lambda v: v.half().cuda()  # noqa: E731
    run = lambda x, w: run_linear(dev(x), packed(dev(w), U.OIDN_FP8_SQUARE), n, None, None, "none", "f16").get().cpu().double()  # noqa: E731
    y = run(x, w)
    assert torch.equal(y, x.double() @ w.double().T)
    dx, dw, db = (t.get().cpu().double() for t in run_back(dev(dy), dev(x), None, dev(w), "none", "f16"))
    assert torch.equal(dx, dy.double() @ w.double()) and torch.equal(dw, dy.double().T @ x.double())
    assert torch.equal(db[0], dy.double().sum(0))
    loss = lambda v: float((dy.double() * v).sum())  # noqa: E731
    assert loss(run(x + step_x, w)) - loss(y) == float((dx * step_x).sum())
    assert loss(run(x, w + step_w)) - loss(y) == float((dw * step_w).sum())


@pytest.mark.parametrize("m, k, n", [(8200, 2056, 4104), (130568, 72, 136), (2056, 8200, 264)])
def test_whole_numbers_in_large_tiles(m, k, n):
    """The same over many tiles of each size, partial ones at every edge, against products in fp32 (sums below 2^24 are
    exact there; results below 2^11 are exact in fp16)."""
    g = torch.Generator(device="cuda").manual_seed(k)
    rand = lambda most, *shape: torch.randint(-most, most + 1, shape, generator=g, device="cuda").half()  # noqa: E731
    share = lambda t, of: t * (torch.rand(t.shape, generator=g, device="cuda") < of)  # noqa: E731
    x, w, dy = share(rand(2, m, k), 400 / max(m, k, 400)), rand(1, n, k), share(rand(1, m, n), 400 / max(m, n, 400))
    want = [x.float() @ w.float().T, dy.float() @ w.float(), dy.float().T @ x.float()]
    assert all(float(t.abs().max()) <= 2048 for t in want)
    y = run_linear(x, packed(w, U.OIDN_FP8_SQUARE), n, None, None, "none", "f16").get()
    dx, dw, db = (t.get() for t in run_back(dy, x, None, w, "none", "f16"))
    for got, v in zip((y, dx, dw, db[0]), want + [dy.float().sum(0)]):
        assert torch.equal(got.float(), v)
    y = run_linear(packed(x), packed(w, U.OIDN_FP8_SQUARE), n, None, None, "relu", "f16", flags=U.OIDN_X_FP8, m=m, k=k).get()
    assert torch.equal(y.float(), want[0].clamp_min(0))


@pytest.mark.parametrize("precision", HALVES)
@pytest.mark.parametrize("m", [1, 20, 70])
def test_linear_keeps_rows_apart(m, precision):
    """A NaN or an infinity in a row makes that row's outputs NaN and no other's, and NaN past the rows' ends reach none."""
    mk, k, n = Maker(3, precision), 300, 66
    x, w = mk.rows(m, k, 4), mk.rows(n, k, 4)
    x[m // 2, 3], x[m - 1, 299] = float("nan"), float("inf")
    y = run_linear(x, packed(w, U.OIDN_FP8_SQUARE), n, None, None, "none", precision).get()
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    bad[[m // 2, m - 1]] = True
    assert y[bad].isnan().all() and y[~bad].isfinite().all()


@pytest.mark.parametrize("m, k, n", [(5, 200, 96), (40, 200, 100), (100, 96, 70), (300, 130, 264)])
def test_z_in_eight_bits(m, k, n):
    mk = Maker(9, "f16")
    x, w, bias = mk.rows(m, k), mk.rows(n, k, scale=k ** -0.5), mk.vec(n)
    w8, w8t = packed(w, U.OIDN_FP8_SQUARE, turned=True)
    z8 = bytes_(U.oidn_ckpt_bytes(m, n))
    y = run_linear(x, w8, n, bias, None, "silu", "f16", z8, U.OIDN_Z_CKPT8)
    want, want_z = reference(x, w, bias, None, "silu")
    check(y.get(), want, "f16", "y")
    z = torch.empty(m, n, dtype=torch.float16, device="cuda")
    U.oidn_ckpt_unpack(z8, m, n, z, n, U.OIDN_F16)
    top = torch.nn.functional.pad(want_z[0].abs() + want_z[1], (0, -n % 32)).view(m, -1, 32).amax(2)
    # half a step of the block's scale, whose own rounding adds 2^-8 of it to the largest code
    assert ((z.cpu().double() - want_z[0]).abs() <= want_z[1] + (top / 127).repeat_interleave(32, 1)[:, :n] * 1.02).all()
    # the gradients read it: the same as from its values in fp32
    dy = mk.rows(m, n)
    a = run_back(dy, x, z8, w, "silu", "f16", flags=U.OIDN_Z_CKPT8)
    wide = torch.empty(m, n, device="cuda")
    U.oidn_ckpt_unpack(z8, m, n, wide, n, U.OIDN_F32)
    want = back_reference(dy, x, given(wide), w, "silu")
    for got, v, name, p in zip(a, want, ("dx", "dw", "dbias"), ("f16", "f16", "f32")):
        check(got.get() if name != "dbias" else got.get()[0], v, p, name)


# -------------------------------------------------------------- gradients
def run_back(dy, x, z, w, kind, precision, flags=0, pad=0, asked=("dx", "dw", "dbias"), stream=None, ws=None):
    (m, n), k, dt, ty = dy.shape, w.shape[1], DT[precision], TORCH[precision]
    dx, dw, db = Out(m, k, ty, pad), Out(n, k, ty, pad), Out(1, n, torch.float32)
    if ws is None:
        ws = bytes_(U.oidn_linear_fp8_backward_workspace_bytes(m, k, n, ACT[kind], dt, flags))
    w8t = packed(w, U.OIDN_FP8_SQUARE, True, False)
    at = lambda name, o: o.view if name in asked else None  # noqa: E731
    U.oidn_linear_fp8_backward(dy, dy.stride(0), x if "dw" in asked else None,
                               x.stride(0) if not flags & U.OIDN_X_FP8 else 0, z,
                               z.stride(0) if z is not None and z.dim() == 2 else 0, w8t if "dx" in asked else None,
                               at("dx", dx), dx.ld, at("dw", dw), dw.ld, at("dbias", db), m, k, n, ACT[kind], dt, flags,
                               ws, ws.numel(), stream=stream)
    return dx, dw, db


def back_reference(dy, x, z, w, kind):
    dz = given(dy) if kind == "none" else mul(given(dy), slope(kind, z))
    turned = lambda a: (a[0].T.contiguous(), a[1].T.contiguous())  # noqa: E731
    dx = R.product(R.coded(dz), turned(R.coded(given(w), True)))
    dw = R.product(R.coded(turned(dz)), R.coded(turned(given(x))))
    return dx, dw, total(dz)


BACK = [(1, 1, 1), (1, 64, 40), (3, 5, 7), (33, 64, 64), (64, 65, 31), (100, 96, 384), (128, 128, 128), (257, 40, 72),
        (1000, 33, 17), (4097, 32, 64), (700, 264, 136), (1300, 600, 520)]


@pytest.mark.parametrize("precision", HALVES)
@pytest.mark.parametrize("m, k, n", BACK)
def test_backward(m, k, n, precision):
    seed = m + 3 * k + 7 * n
    mk, kind, pad = Maker(seed, precision), ACTS[seed % 4], [0, 8, 3][seed % 3]
    x, w, dy, z = mk.rows(m, k, pad), mk.rows(n, k, pad, k ** -0.5), mk.rows(m, n, pad), mk.rows(m, n, pad)
    got = run_back(dy, x, z, w, kind, precision, pad=pad)
    want = back_reference(dy, x, given(z), w, kind)
    check(got[0].get(), want[0], precision, "dx")
    check(got[1].get(), want[1], precision, "dw")
    check(got[2].get()[0], want[2], "f32", "dbias")
    # x as its packed transpose: the same bits
    again = run_back(dy, packed(x, 0, True, False), z, w, kind, precision, U.OIDN_X_FP8, pad)
    assert all(torch.equal(a.get(), b.get()) for a, b in zip(again, got))


@pytest.mark.parametrize("asked", ["dx", "dw", "dbias", "nothing"])
def test_backward_parts(asked):
    mk, m, k, n = Maker(21, "bf16"), 290, 72, 140
    x, w, dy, z = mk.rows(m, k), mk.rows(n, k), mk.rows(m, n), mk.rows(m, n)
    both, some = run_back(dy, x, z, w, "silu", "bf16"), run_back(dy, x, z, w, "silu", "bf16", asked=[asked])
    for name, a, b in zip(("dx", "dw", "dbias"), both, some):
        assert torch.equal(b.get(), a.get() if name == asked else torch.full_like(a.get(), GUARD)), name


def test_gradients_of_no_rows_are_zero():
    dw, db = Out(5, 7, torch.float16, 2), Out(1, 5, torch.float32)
    U.oidn_linear_fp8_backward(None, 5, None, 7, None, 5, None, None, 7, dw.view, dw.ld, db.view, 0, 7, 5,
                               U.OIDN_ACT_GELU, U.OIDN_F16, 0, None, 0)
    assert not dw.get().any() and not db.get().any()


# --------------------------------------------------------- streams, graphs
@pytest.mark.parametrize("m, k, n", [(4, 640, 96), (300, 200, 264)])
def test_streams_and_the_same_bits_again(m, k, n):
    mk = Maker(31, "bf16")
    x, w, dy, z = mk.rows(m, k), mk.rows(n, k), mk.rows(m, n), mk.rows(m, n)
    w8 = packed(w, U.OIDN_FP8_SQUARE)
    want = [run_linear(x, w8, n, None, dy, "gelu", "bf16").get()] + [t.get() for t in run_back(dy, x, z, w, "gelu", "bf16")]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(stream):
            got = [run_linear(x, w8, n, None, dy, "gelu", "bf16")] + list(run_back(dy, x, z, w, "gelu", "bf16"))
        stream.synchronize()
        assert all(torch.equal(a.get(), b) for a, b in zip(got, want))


@pytest.mark.parametrize("m, k, n", [(4, 640, 96), (300, 2000, 264)])
def test_graph_replays(m, k, n):
    """Packing, a forward and a backward pass captured; each replay on new inputs equals the eager calls."""
    mk = Maker(41, "f16")
    x, w, dy, z = mk.rows(m, k), mk.rows(n, k, scale=k ** -0.5), mk.rows(m, n), mk.rows(m, n)
    ws = bytes_(U.oidn_linear_fp8_backward_workspace_bytes(m, k, n, ACT["silu"], DT["f16"], 0))

    def step():
        w8 = packed(w, U.OIDN_FP8_SQUARE)
        return [run_linear(x, w8, n, None, dy, "silu", "f16")] + list(run_back(dy, x, z, w, "silu", "f16", ws=ws))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(4):
        for t in (x, w, dy, z):
            t.copy_(torch.randn(t.shape, device="cuda") * 0.3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        now = [o.get().clone() for o in outs]
        assert all(torch.equal(a, b.get()) for a, b in zip(now, step()))
