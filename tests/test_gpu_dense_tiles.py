"""The dense operators' large tiles, 128 x 128 and 256 x 256, in each of their
forms: operands straight to LDS and through registers, every epilogue, ragged
rows, columns and sums, what is kept in the storage type and in 8 bits.  A graph
that records the call names the kernels it launches, so that a case whose plan
has moved to other tiles says so.  All elements are compared, with the bounds of
dense_reference on the GPU in 64 bits."""
import ctypes
import re

import pytest
import torch

import unet_x3_convolution_amd as U
from dense_reference import HALF, TINY, TORCH, ffn, ffn_backward, linear, linear_backward, stored
from helpers import DT, torch_cuda

pytestmark = pytest.mark.gpu

ACT = {"none": U.OIDN_ACT_NONE, "relu": U.OIDN_ACT_RELU, "silu": U.OIDN_ACT_SILU, "gelu": U.OIDN_ACT_GELU}


@pytest.fixture(autouse=True)
def gpu():
    torch_cuda()
    yield
    torch.cuda.empty_cache()


class Dim3(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint), ("y", ctypes.c_uint), ("z", ctypes.c_uint)]


class KernelNode(ctypes.Structure):
    _fields_ = [("block", Dim3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("grid", Dim3),
                ("args", ctypes.c_void_p), ("lds", ctypes.c_uint)]


def names(call):
    """The kernels that `call` launches, by their mangled names."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    hip, raw, count = U.lib(), ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t()
    assert hip.hipGraphGetNodes(raw, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert hip.hipGraphGetNodes(raw, nodes, ctypes.byref(count)) == 0
    hip.hipKernelNameRefByPtr.restype = ctypes.c_char_p
    found = []
    for node in nodes:
        params = KernelNode()
        assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(params)) == 0
        found.append(hip.hipKernelNameRefByPtr(ctypes.c_void_p(params.func), None).decode())
    return found


def launches(call):
    """(kernel, tile, straight to LDS) of the 16-bit tile kernels that `call` launches."""
    found = []
    for name in names(call):
        m = re.search(r"dense_gemm16(_gated_back|_group)?ILb[01]E(?:Li0ELi([02])E)?Li(\d+)E(?:Li\d+E)?Lb([01])E", name)
        if m:
            kind = {"_gated_back": "gated back", "_group": "group"}.get(m[1]) or ("linear" if m[2] == "0" else "gated")
            found.append((kind, int(m[3]), m[4] == "1"))
    return found


def wide(t):
    return (t.double(), torch.zeros(t.shape, dtype=torch.float64, device=t.device)) if t is not None else None


def agree(got, want, precision, label):
    v, e = stored(want, precision)
    bad = ~((got.double() - v).abs() <= e)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} off, first at {at}: got {got[at].item():.9g}, "
                             f"want {v[at].item():.9g} +- {e[at].item():.3g}")


class Maker:
    """Rows of buffers `pad` columns wider, which hold NaN."""

    def __init__(self, seed, precision, pad):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.type, self.pad = TORCH[precision], pad

    def rows(self, m, n, scale=1.0, pad=None):
        pad = self.pad if pad is None else pad
        buf = torch.full((m, n + pad), float("nan"), dtype=self.type, device="cuda")
        buf[:, :n] = torch.randn(m, n, generator=self.g, device="cuda") * scale
        return buf[:, :n]

    def vec(self, n):
        return torch.randn(n, generator=self.g, device="cuda") * 0.5

    def out(self, m, n):
        """Rows to be written, inside a buffer of sevens."""
        return torch.full((m, n + self.pad), 7.0, dtype=self.type, device="cuda")

    def intact(self, buf, n):
        assert (buf[:, n:] == 7).all(), "written past the rows' ends"
        return buf[:, :n]


def bytes_(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def kept(blob, m, n):
    """A checkpoint's values (products of an int8 and a bf16, exact in fp32)."""
    y = torch.empty(m, n, device="cuda")
    U.oidn_ckpt_unpack(blob, m, n, y, n, U.OIDN_F32)
    return y


def agree8(blob, want, label):
    """Half a step of the block's scale, of which the largest magnitude and the roundings of the scale decide."""
    v, e = want
    m, n = v.shape
    top = torch.nn.functional.pad(v.abs() + e, (0, -n % 32)).view(m, -1, 32).amax(2).repeat_interleave(32, 1)[:, :n]
    bad = ~((kept(blob, m, n).double() - v).abs() <= (0.5 + 2.0 ** -13) * (1 + 2.0 ** -8) * top / 127 + e)
    assert not bad.any(), (label, int(bad.sum()))


# m, k, n, the tile, and the one where rows lie at odd pitches
LINEAR = [(3001, 264, 1030, (128, True), (128, False)), (6150, 264, 2054, (256, True), (128, False)),
          (6145, 320, 2049, (256, True), (128, False)), (1030, 8192, 1030, (128, True), (128, False)),
          (3001, 263, 1030, (128, False), (128, False)), (8001, 1032, 510, (128, True), (128, False)),
          (13101, 264, 4102, (256, True), (128, False))]


@pytest.mark.parametrize("precision", ["f16", "bf16"])
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("m, k, n, whole, odd", LINEAR)
def test_linear(m, k, n, whole, odd, pad, precision):
    mk, dt, kind = Maker(m + k + n, precision, pad), DT[precision], "gelu" if m % 2 else "silu"
    x, w, r, bias = mk.rows(m, k), mk.rows(n, k, k ** -0.5, 0), mk.rows(m, n), mk.vec(n)
    y, z, z8 = mk.out(m, n), mk.out(m, n), bytes_(U.oidn_ckpt_bytes(m, n))
    ws = bytes_(U.oidn_linear_workspace_bytes(m, k, n, dt))

    def call(z, flags=0):
        U.oidn_linear(x, x.stride(0), w, k, bias, r, r.stride(0), y, y.stride(0), z, n + pad, m, k, n, ACT[kind], dt, flags, ws,
                      ws.numel())

    assert launches(lambda: call(z)) == [("linear", *(odd if pad == 3 else whole))]
    call(z)
    want, want_z = linear(wide(x), wide(w), wide(bias), wide(r), kind)
    agree(mk.intact(y, n), want, precision, "y")
    agree(mk.intact(z, n), want_z, precision, "z")
    first = y.clone()
    y.fill_(7)
    call(z8, U.OIDN_Z_CKPT8)
    assert torch.equal(y, first)
    agree8(z8, want_z, "z in 8 bits")


# m, d, f, tiles of the gated product and of the second one
FFN = [(1500, 1032, 776, 128, 64), (3001, 1032, 518, 128, 128), (16400, 72, 2056, 256, 64)]


@pytest.mark.parametrize("precision", ["f16", "bf16"])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("m, d, f, gated, second", FFN)
def test_ffn(m, d, f, gated, second, pad, precision):
    mk, dt, kind = Maker(m + d + f, precision, pad), DT[precision], "silu" if m % 2 else "gelu"
    x, r = mk.rows(m, d), mk.rows(m, d)
    w_in, w_out, b_in, b_out = mk.rows(2 * f, d, d ** -0.5, 0), mk.rows(d, f, f ** -0.5, 0), mk.vec(2 * f), mk.vec(d)
    y, z, one = mk.out(m, d), torch.empty(m, 2 * f, dtype=x.dtype, device="cuda"), U.oidn_ckpt_bytes(m, f)
    z8, ws = bytes_(2 * one), bytes_(U.oidn_ffn_workspace_bytes(m, d, f, dt))

    def call(z, flags=0):
        U.oidn_ffn(x, x.stride(0), w_in, b_in, w_out, b_out, r, r.stride(0), y, y.stride(0), z, m, d, f, ACT[kind], dt, flags,
                   ws, ws.numel())

    assert launches(lambda: call(z)) == [("gated", min(gated, 128) if pad else gated, pad == 0), ("linear", second, f % 8 == 0)]
    call(z)
    want, want_z = ffn(wide(x), wide(w_in), wide(b_in), wide(w_out), wide(b_out), wide(r), kind, precision)
    agree(mk.intact(y, d), want, precision, "y")
    agree(z, want_z, precision, "z")
    first = y.clone()
    y.fill_(7)
    call(z8, U.OIDN_Z_CKPT8)
    assert torch.equal(y, first)
    for k in range(2):
        agree8(z8[k * one:(k + 1) * one], tuple(a[:, k * f:(k + 1) * f] for a in want_z), "z in 8 bits")
    del want, want_z
    call(None)
    assert torch.equal(y, first)


# m, k, n and the tile of both products
LINEAR_BACK = [(2051, 4104, 2056, 256), (12301, 4104, 2056, 256), (8201, 520, 1032, 128), (521, 4104, 520, 128)]


@pytest.mark.parametrize("precision", ["f16", "bf16"])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("m, k, n, tile", LINEAR_BACK)
def test_linear_backward(m, k, n, tile, pad, precision):
    """At odd pitches dw = dz^T x goes through registers, dx = dz w, whose operands lie well, as before."""
    mk, dt = Maker(m + k + n, precision, pad), DT[precision]
    x, dy, z, w = mk.rows(m, k), mk.rows(m, n), mk.rows(m, n), mk.rows(n, k, k ** -0.5, 0)
    dx, dw, db = mk.out(m, k), mk.out(n, k), torch.empty(n, device="cuda")
    ws = bytes_(U.oidn_linear_backward_workspace_bytes(m, k, n, U.OIDN_ACT_SILU, dt, 0))

    def call():
        U.oidn_linear_backward(dy, dy.stride(0), x, x.stride(0), z, z.stride(0), w, k, dx, k + pad, dw, k + pad, db, m, k, n,
                               U.OIDN_ACT_SILU, dt, 0, ws, ws.numel())

    there = [("group", tile, True)] if pad == 0 else [("group", 128, False), ("group", tile, True)]
    assert launches(call) == there
    call()
    want = linear_backward(wide(dy), wide(x), wide(z), wide(w), "silu", precision)
    agree(mk.intact(dx, k), want[0], precision, "dx")
    agree(mk.intact(dw, k), want[1], precision, "dw")
    agree(db, want[2], "f32", "dbias")


# m, d, f, tiles of dh and of the gradients' products
FFN_BACK = [(2051, 4104, 1032, 64, 256), (6150, 264, 2056, 256, 128), (16401, 72, 2056, 128, 128)]


@pytest.mark.parametrize("precision", ["f16", "bf16"])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("m, d, f, back, tile", FFN_BACK)
def test_ffn_backward(m, d, f, back, tile, eight, pad, precision):
    mk, dt, ty = Maker(m + d + f, precision, pad), DT[precision], TORCH[precision]
    x, dy, extra, z = mk.rows(m, d), mk.rows(m, d), mk.rows(m, d), mk.rows(m, 2 * f, pad=0)
    w_in, w_out = mk.rows(2 * f, d, d ** -0.5, 0), mk.rows(d, f, f ** -0.5, 0)
    dx, dw_in, dw_out = mk.out(m, d), torch.empty_like(w_in), torch.empty_like(w_out)
    db_in, db_out = torch.empty(2 * f, device="cuda"), torch.empty(d, device="cuda")
    flags, from_x, from_z, ldx = 0, x, z, x.stride(0)
    if eight:
        flags, one = U.OIDN_X_CKPT8 | U.OIDN_Z_CKPT8, U.oidn_ckpt_bytes(m, f)
        from_x, from_z, ldx = bytes_(U.oidn_ckpt_bytes(m, d)), bytes_(2 * one), 0
        U.oidn_ckpt_pack(x, x.stride(0), m, d, from_x, dt)
        for k in range(2):
            U.oidn_ckpt_pack(z[:, k * f:], 2 * f, m, f, from_z[k * one:], dt)
        z = torch.cat([kept(from_z[k * one:], m, f) for k in range(2)], 1)
        x = kept(from_x, m, d)
    ws = bytes_(U.oidn_ffn_backward_workspace_bytes(m, d, f, dt, flags))

    def call():
        U.oidn_ffn_backward(dy, dy.stride(0), from_x, ldx, from_z, w_in, w_out, extra, extra.stride(0), dx, d + pad, dw_in,
                            db_in, dw_out, db_out, m, d, f, U.OIDN_ACT_GELU, dt, flags, ws, ws.numel())

    found = launches(call)
    assert found[0] == ("gated back", min(back, 128) if pad else back, pad == 0)
    # dy and x at odd pitches go through registers, an x that came back from 8 bits and dx's operands do not
    assert ("group", tile, True) in found[1:] and ((("group", 128, False) in found[1:]) == (pad != 0))
    call()
    kept_x = stored(wide(x), precision) if eight else wide(x)
    want = ffn_backward(wide(dy), kept_x, wide(z), wide(w_in), wide(w_out), wide(extra), "gelu", precision)
    agree(mk.intact(dx, d), want[0], precision, "dx")
    agree(dw_in, want[1], precision, "dw_in")
    agree(dw_out, want[2], precision, "dw_out")
    agree(db_in, want[3], "f32", "db_in")
    agree(db_out, want[4], "f32", "db_out")


@pytest.mark.parametrize("m, n, streamed", [(529, 2048, False), (16401, 192, True), (174737, 192, False), (4113, 2048, False),
                                            (49169, 1024, True), (2048, 513, False), (2048, 512, True)])
def test_which_results_go_past_the_caches(m, n, streamed):
    """Those that the next reader is better off without in them: narrow ones of up to 18 MB, all from 96 MB on."""
    x, w, y = (torch.empty(r, c, dtype=torch.bfloat16, device="cuda") for r, c in ((m, 64), (n, 64), (m, n)))
    ws = bytes_(U.oidn_linear_workspace_bytes(m, 64, n, U.OIDN_BF16))
    called = names(lambda: U.oidn_linear(x, 64, w, 64, None, None, 0, y, n, None, 0, m, 64, n, U.OIDN_ACT_RELU, U.OIDN_BF16, 0,
                                         ws, ws.numel()))
    assert len(called) == 1 and re.search(r"CachingE([01])E", called[0])[1] == str(int(streamed))
