"""The dense operators' definitions in 64 bits, each value with a bound on how
far the kernels' result may be from it.

A value travels as a pair (v, e): v in float64, e an elementwise bound on the
absolute error of the library's value.  The bounds are the standard ones:

* a sum of L products in fp32 is off by at most (L + 2) u sum|p q|; u is taken
  as 2^-23, twice the unit roundoff, which also covers an adder that truncates;
* a value stored in a type is off by half a step, eps / 2 of it, or half the
  spacing of the subnormals;
* an fp32 activation or slope is off by a few units in the last place of its
  argument's magnitude (2^-20 relative to max(|z|, 1) covers the exponential,
  the reciprocal and the 1.5e-7 of the error function's formula), and passes
  its argument's error on times its largest slope (1.13), the slope times its
  largest derivative (0.8).
"""
import math

import torch

HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -23
ACTS = ["none", "relu", "silu", "gelu"]


def given(t):
    """Inputs are exact."""
    v = t.detach().cpu().double()
    return v, torch.zeros_like(v)


def product(q, p):
    """q p^T: (i, l) x (j, l) summed over l."""
    (qv, qe), (pv, pe) = q, p
    qa, pa = qv.abs(), pv.abs()
    span = (qa + qe) @ (pa + pe).T
    return qv @ pv.T, qa @ pe.T + qe @ pa.T + qe @ pe.T + (qv.shape[1] + 2) * U32 * span


def t(a):
    return a[0].T, a[1].T


def add(a, b):
    v = a[0] + b[0]
    return v, a[1] + b[1] + U32 * (v.abs() + a[1] + b[1])


def mul(a, b):
    v = a[0] * b[0]
    e = a[0].abs() * b[1] + a[1] * b[0].abs() + a[1] * b[1]
    return v, e + U32 * (v.abs() + e)


def stored(a, precision):
    return a[0], a[1] + HALF[precision] * (a[0].abs() + a[1]) + TINY[precision]


def total(a):
    """Column sums."""
    m = a[0].shape[0]
    return a[0].sum(0), a[1].sum(0) + (m + 2) * U32 * (a[0].abs() + a[1]).sum(0)


def act(kind, z):
    v, e = z
    if kind == "none":
        return z
    if kind == "relu":
        return v.clamp_min(0), e
    if kind == "silu":
        f = v / (1 + torch.exp(-v))
    else:
        f = v * torch.special.erfc(-v / math.sqrt(2)) / 2
    return f, 1.13 * e + 2.0 ** -20 * v.abs().clamp_min(1)


def slope(kind, z):
    v, e = z
    if kind == "none":
        return torch.ones_like(v), torch.zeros_like(v)
    if kind == "relu":
        assert not e.any()
        return (v > 0).double(), torch.zeros_like(v)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-v))
        f = p + v * p * (1 - p)
    else:
        f = torch.special.erfc(-v / math.sqrt(2)) / 2 + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    return f, 0.8 * e + 2.0 ** -20 * v.abs().clamp_min(1)


def linear(x, w, bias, residual, kind):
    z = product(x, w)
    if bias is not None:
        z = add(z, (bias[0][None, :].expand_as(z[0]), torch.zeros_like(z[0])))
    y = act(kind, z)
    return (add(y, residual) if residual is not None else y), z


def linear_backward(dy, x, z, w, kind, precision):
    dz = dy if kind == "none" else mul(dy, slope(kind, z))
    kept = dz if kind == "none" else stored(dz, precision)
    return product(kept, t(w)), product(t(kept), t(x)), total(dz)


def ffn(x, w_in, b_in, w_out, b_out, residual, kind, precision):
    f = w_out[0].shape[1]
    _, z = linear(x, w_in, b_in, None, "none")
    a, b = (z[0][:, :f], z[1][:, :f]), (z[0][:, f:], z[1][:, f:])
    h = stored(mul(act(kind, a), b), precision)
    y, _ = linear(h, w_out, b_out, residual, "none")
    return y, z


def ffn_backward(dy, x, z, w_in, w_out, extra, kind, precision):
    f = w_out[0].shape[1]
    a, b = (z[0][:, :f], z[1][:, :f]), (z[0][:, f:], z[1][:, f:])
    dh = product(dy, t(w_out))
    g = act(kind, a)
    da, db = mul(mul(dh, b), slope(kind, a)), mul(dh, g)
    dz = torch.cat([da[0], db[0]], 1), torch.cat([da[1], db[1]], 1)
    kept, h = stored(dz, precision), stored(mul(g, b), precision)
    dx = product(kept, t(w_in))
    if extra is not None:
        dx = add(dx, extra)
    return dx, product(t(kept), t(x)), product(t(dy), t(h)), total(dz), total(dy)


def check(got, want, precision, label):
    """Every element within its bound, after the output's own rounding.  A value past the type's range is stored as
    an infinity of its sign: allowed where the bound reaches the border (the largest value and half a step), asked
    for where it lies past it."""
    v, e = stored(want, precision)
    g = got.detach().cpu().double()
    assert g.shape == v.shape, (label, g.shape, v.shape)
    off = (g - v).abs()
    border = float(torch.finfo(TORCH[precision]).max) * (1 + HALF[precision] / 2)
    over = (g == torch.where(v > 0, math.inf, -math.inf)) & (v.abs() + e >= border)
    bad = ~(over | (off <= e)) | (v.abs() - e > border) & ~over
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} off, first at {at}: "
                             f"got {g[at].item():.9g}, want {v[at].item():.9g} +- {e[at].item():.3g}")
