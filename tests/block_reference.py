"""Definitions in 64 bits of what stands around a block, with bounds on how far
an fp32 computation may be from them; values are the pairs of dense_reference.

* a mean of n values is their sum over n: off by (n + 3) u times the mean magnitude
* a row's factor r = (v + eps)^-1/2 moves with its argument as the function does,
  and is formed with a few more roundings (4 u of it)
"""
import numpy as np
import torch

from dense_reference import U32, add, mul, total

NORMS = ["none", "rms", "layer"]


def philox(counter, key):
    """Philox4x32-10 of uint64 arrays: counter four words, key two."""
    low = np.uint64(0xffffffff)
    c, k = [np.asarray(v, np.uint64) for v in counter], [np.uint64(v) for v in key]
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ k[0], q & low, (p >> np.uint64(32)) ^ c[3] ^ k[1], p & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return c


def kept(m, n, p, seed, offset):
    """m x n factors: 0 or the gain of a kept element."""
    limit = round(float(np.float32(p)) * 65536)
    if limit == 0:
        return torch.ones(m, n, dtype=torch.float64)
    per = -(-n // 8)
    at = np.arange(m * per, dtype=np.uint64)
    halves = lambda v: (v & 0xffffffff, v >> 32)  # noqa: E731
    o, k = halves(offset % 2 ** 64), halves(seed % 2 ** 64)
    words = philox([at & np.uint64(0xffffffff), at >> np.uint64(32), np.full_like(at, o[0]), np.full_like(at, o[1])], k)
    bits = np.stack([v for w in words for v in (w & np.uint64(0xffff), w >> np.uint64(16))], 1)
    keep = torch.from_numpy(bits.reshape(m, per * 8)[:, :n].astype(np.int64)) >= limit
    return keep.double() * (65536 / (65536 - limit) if limit < 65536 else 0)


def mean(a):
    v, e = a
    n = v.shape[1]
    return v.mean(1, keepdim=True), (e + (n + 3) * U32 * (v.abs() + e)).mean(1, keepdim=True)


def sub(a, b):
    return add(a, (-b[0], b[1]))


def scaled(a, factor):
    """Times exact factors (a tensor that broadcasts)."""
    v = a[0] * factor
    e = a[1] * factor.abs()
    return v, e + U32 * (v.abs() + e)


def exact(v):
    return v, torch.zeros_like(v)


def normed(kind, x, eps):
    """hat and r of rows."""
    if kind == "none":
        one = torch.ones(x[0].shape[0], 1, dtype=torch.float64)
        return x, exact(one)
    d = sub(x, tuple(t.expand_as(x[0]) for t in mean(x))) if kind == "layer" else x
    v, e = mean(mul(d, d))
    v, e = v + eps, e + U32 * (v + eps)
    r = v.rsqrt()
    far = (v - e).clamp_min(0).rsqrt() - r
    r = r, far + 4 * U32 * (r + far)
    return mul(d, tuple(t.expand_as(d[0]) for t in r)), r


def pulled(kind, g, hat, r):
    """The gradient of a norm's input from that of its output."""
    if kind == "none":
        return g
    wide = lambda a: tuple(t.expand_as(g[0]) for t in a)  # noqa: E731
    d = sub(g, mul(hat, wide(mean(mul(g, hat)))))
    if kind == "layer":
        d = sub(d, wide(mean(g)))
    return mul(d, wide(r))


def affine(hat, weight, shift):
    y = scaled(hat, weight) if weight is not None else hat
    return add(y, exact(shift.expand_as(y[0]))) if shift is not None else y


def of_rows(gate, gate_rows, m):
    return gate.repeat_interleave(gate_rows, 0)[:m] if gate is not None else torch.ones(1, 1, dtype=torch.float64)


def after(o, weight, shift, gate, gate_rows, x, scale, keep, kind, eps):
    """u."""
    b = scaled(affine(normed(kind, o, eps)[0], weight, shift), keep)
    return add(scaled(x, torch.tensor(float(np.float32(scale)), dtype=torch.float64)),
               scaled(b, of_rows(gate, gate_rows, x[0].shape[0])))


def before(u, weight, shift, kind, eps):
    """v."""
    return affine(normed(kind, u, eps)[0], weight, shift)


def back(du, dv, o, u, weight, shift, gate, gate_rows, scale, keep, kind, next_weight, next_kind, eps):
    """All gradients, by name; pairs."""
    got, d = {}, du
    if next_kind != "none":
        hat, r = normed(next_kind, u, eps)
        g = scaled(dv, next_weight) if next_weight is not None else dv
        pull = pulled(next_kind, g, hat, r)
        d = add(d, pull) if d is not None else pull
        got["dnext_weight"], got["dnext_shift"] = total(mul(dv, hat)), total(dv)
    got["dx"] = scaled(d, torch.tensor(float(np.float32(scale)), dtype=torch.float64))
    if o is None:
        return got
    m = d[0].shape[0]
    hat, r = normed(kind, o, eps)
    if gate is not None:
        each = mul(d, scaled(affine(hat, weight, shift), keep))
        parts = [total((each[0][i:i + gate_rows], each[1][i:i + gate_rows])) for i in range(0, m, gate_rows)]
        got["dgate"] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    h = scaled(scaled(d, of_rows(gate, gate_rows, m)), keep)
    got["dweight"], got["dshift"] = total(mul(h, hat)), total(h)
    got["d_o"] = pulled(kind, scaled(h, weight) if weight is not None else h, hat, r)
    return got
