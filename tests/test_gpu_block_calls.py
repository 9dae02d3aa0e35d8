"""Calls around a block that the interface allows and that no other test makes: the residual
in y's place, in place at a padded pitch, two calls at once on two streams, a gate in a wider
buffer's columns, one input read in several places."""
import pytest
import torch

import unet_x3_convolution_amd as U
from dense_reference import TORCH
from helpers import DT, torch_cuda
from test_gpu_dense import ACT, Maker, Out, bytes_
from test_gpu_fp8 import HALVES, packed, run_back, run_linear
from test_gpu_norm import EPS, KIND, back_case, residual_case, run_back as norm_back, run_residual

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def gpu():
    torch_cuda()


# one row, rows coded on the way, few packed ones, one block of inputs, tiles, slices, tiles of each size
LAYERS = [(1, 300, 44), (4, 520, 100), (20, 600, 72), (90, 100, 75), (300, 128, 264), (70, 8192, 72), (300, 260, 200),
          (1100, 520, 1030), (8192, 1200, 2056)]


@pytest.mark.parametrize("precision", HALVES)
@pytest.mark.parametrize("pad, shift", [(0, 0), (3, 1)])
@pytest.mark.parametrize("m, k, n", LAYERS)
def test_layer_adds_to_y(m, k, n, pad, shift, precision):
    """The same bits as from a residual of its own, and nothing written past the rows."""
    mk, dt = Maker(m + n, precision), DT[precision]
    x, w, bias, r = mk.rows(m, k, pad), mk.rows(n, k, 0, k ** -0.5), mk.vec(n), mk.rows(m, n, pad, shift=shift)
    w8 = packed(w, U.OIDN_FP8_SQUARE)
    for given, flags in ((x, 0), (packed(x), U.OIDN_X_FP8)):
        want = run_linear(given, w8, n, bias, r, "silu", precision, flags=flags, pad=pad, shift=shift, m=m, k=k).get()
        y = Out(m, n, TORCH[precision], pad, shift)
        y.view[:, :n] = r
        ws = bytes_(U.oidn_linear_fp8_workspace_bytes(m, k, n, dt, flags))
        U.oidn_linear_fp8(given, 0 if flags else x.stride(0), w8, bias, y.view, y.ld, y.view, y.ld, None, 0, m, k, n,
                          ACT["silu"], dt, flags, ws, ws.numel())
        assert torch.equal(y.get(), want)


@pytest.mark.parametrize("n", [31, 40, 257, 700, 2049, 5000, 9001])
@pytest.mark.parametrize("where", ["x", "o"])
def test_in_place_at_a_pitch(n, where):
    """u over x or o inside a wider buffer, rows enough that a workgroup takes several."""
    m, seed = max(40, 66000 // n), 26
    c = residual_case(m, n, "rms", "layer", "f16", seed)
    assert c["gate"] is not None and c["p"]
    want_u, want_v = [t.get().clone() for t in run_residual(c)]
    u = Out(m, n, torch.float16, c["pad"])
    u.view[:, :n] = c[where]
    at = dict(c, **{where: u.view[:, :n]})
    v = Out(m, n, torch.float16, c["pad"])
    U.oidn_norm_residual(at["o"], at["o"].stride(0), c["weight"], c["shift"], c["gate"], c["gate"].stride(0),
                         c["gate_rows"], at["x"], at["x"].stride(0), c["scale"], c["p"], c["rng"], u.view, u.ld,
                         c["next_weight"], c["next_shift"], v.view, v.ld, m, n, KIND["rms"], KIND["layer"], EPS, U.OIDN_F16)
    assert torch.equal(u.get(), want_u) and torch.equal(v.get(), want_v)


def test_two_calls_at_once():
    """Forward and backward passes of both operators on two streams, each with its own workspace: the bits of one
    after the other."""
    mk = Maker(2, "bf16")
    m, k, n = 700, 520, 1030
    x, w, dy, z = mk.rows(m, k), mk.rows(n, k, 0, k ** -0.5), mk.rows(m, n), mk.rows(m, n)
    w8 = packed(w, U.OIDN_FP8_SQUARE)
    c = back_case(1200, 1000, "layer", "rms", "bf16", 26)

    def layer(stream=None):
        return [run_linear(x, w8, n, None, None, "gelu", "bf16", stream=stream),
                *run_back(dy, x, z, w, "silu", "bf16", stream=stream)]

    def norms(stream=None):
        return [*run_residual(c, stream=stream), *norm_back(c, stream=stream).values()]

    want = [[o.get().clone() for o in f()] for f in (layer, norms)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for turn in range(6):
        for s, f, to in zip(streams, (layer, norms) if turn % 2 else (norms, layer), (got[turn % 2 == 0], got[turn % 2])):
            # the wrappers' fills run on the stream that their kernels take
            with torch.cuda.stream(s):
                to.append(f())
    torch.cuda.synchronize()
    for outs, wanted in zip(got, want):
        assert len(outs) == 6 and all(torch.equal(o.get(), v) for run in outs for o, v in zip(run, wanted))


def test_the_same_input_in_several_places():
    """o and x the same rows; dv and du; weight and next_weight; a gate for all rows from a row of a wider table."""
    m, n = 300, 264
    c = residual_case(m, n, "rms", "rms", "f32", 26)
    table = torch.randn(3, 5 * n, device="cuda")
    alone = dict(c, x=c["o"].clone(), next_weight=c["weight"].clone(), next_shift=None, gate_rows=100,
                 gate=table[:, 2 * n:3 * n].contiguous())
    shared = dict(c, x=c["o"], next_weight=c["weight"], next_shift=None, gate_rows=100, gate=table[:, 2 * n:3 * n])
    for a, b in zip(run_residual(alone), run_residual(shared)):
        assert torch.equal(a.get(), b.get())
    b = back_case(m, n, "rms", "rms", "f32", 26)
    alone.update(u=b["u"].clone(), du=b["dv"].clone(), dv=b["dv"].clone())
    shared.update(u=b["u"].clone(), du=b["dv"], dv=b["dv"])
    one, two = norm_back(alone), norm_back(shared)
    assert all(torch.equal(o.get(), two[name].get()) for name, o in one.items())


@pytest.mark.parametrize("n", [24, 1000, 9000])
def test_far_apart_rows(n):
    """A pitch of 2^31 elements: the third row begins 2^32 elements in (no memory lies between but one buffer's)."""
    ld, m = 1 << 31, 3
    buf = torch.empty(2 * ld + n, dtype=torch.float16, device="cuda")
    out = torch.empty(2 * ld + n, dtype=torch.float16, device="cuda")
    far, to = buf.as_strided((m, n), (ld, 1)), out.as_strided((m, n), (ld, 1))
    x = torch.randn(m, n, device="cuda").half()
    far.copy_(x)
    near = torch.empty(m, n, dtype=torch.float16, device="cuda")
    for call in (lambda a, lda, y, ldy: U.oidn_norm(a, lda, None, None, y, ldy, m, n, KIND["layer"], EPS, U.OIDN_F16),
                 lambda a, lda, y, ldy: U.oidn_dropout(a, lda, None, 0, y, ldy, m, n, 0.5, rng, U.OIDN_F16),
                 lambda a, lda, y, ldy: unpack(a, lda, y, ldy)):
        rng = torch.tensor([1, 2], device="cuda")
        blob = bytes_(U.oidn_fp8_bytes(m, n))

        def unpack(a, lda, y, ldy):
            U.oidn_fp8_pack(a, lda, m, n, blob, None, U.OIDN_F16, 0)
            U.oidn_fp8_unpack(blob, m, n, y, ldy, U.OIDN_F16)

        call(x, n, near, n)
        call(far, ld, to, ld)
        assert torch.equal(near, to)
    del buf, out, far, to
    torch.cuda.empty_cache()
