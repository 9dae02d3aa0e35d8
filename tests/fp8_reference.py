"""The packed 8-bit form and its products in 64 bits, with bounds; values are the
pairs of dense_reference.

* a code is exact for an exact value; one that is off by e is coded between the codes
  of v - e and v + e (coding is monotone), and where the block's largest value may
  fall on the other side of a power of two, values below 2^-6 of the scale may be a
  step of the wider scale further off (the others have the same codes in both);
* the matrix cores add eight products (neighbouring summed elements) with the last
  bit at 2^-13 of the largest one's power of two: 7 of them lose less than that each,
  and the power is at most the product of the two eights' largest values; the sums of
  eight are added in fp32.
"""
import torch

from dense_reference import U32

BLOCK, LARGEST = 128, 448.0


def power(top):
    """e of blocks from their largest finite magnitude."""
    part, e = torch.frexp(top)
    e = torch.where(part <= 0.875, e - 9, e - 8).clamp(-120, 120)
    return torch.where(top > 0, e, torch.zeros_like(e))


def rounded(v):
    """To e4m3: four significant bits, steps of 2^-9 below 2^-6; ties to even."""
    e = (torch.frexp(v).exponent - 1).clamp_min(-6)
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return torch.round(v / step) * step


def padded(v, rows, cols):
    out = torch.zeros(-(-v.shape[0] // rows) * rows, -(-v.shape[1] // cols) * cols, dtype=v.dtype)
    out[:v.shape[0], :v.shape[1]] = v
    return out


def blocks(v, square=False):
    """v in blocks: [row block][row][column block][column]."""
    r = BLOCK if square else 1
    w = padded(v, r, BLOCK)
    return w.view(w.shape[0] // r, r, w.shape[1] // BLOCK, BLOCK)


def back(b, like):
    return b.reshape(b.shape[0] * b.shape[1], -1)[:like.shape[0], :like.shape[1]]


def code(v, square=False):
    """(values, e of each row's blocks) of a matrix in float64."""
    b = blocks(v, square)
    finite = torch.where(b.isfinite(), b.abs(), torch.zeros_like(b))
    p = power(finite.amax((1, 3), keepdim=True))
    scale = torch.ldexp(torch.ones_like(b[:, :1, :, :1]), p)
    q = rounded(b / scale) * scale
    q = torch.where(b.isfinite(), q, torch.full_like(q, float("nan")))
    each = p.expand(b.shape[0], b.shape[1], b.shape[2], 1).reshape(-1, b.shape[2])[:v.shape[0]]
    return back(q, v), each


def coded(a, square=False):
    """The pair of a coded pair."""
    v, e = a
    b, be = blocks(v, square), blocks(e, square)
    p = power(b.abs().amax((1, 3), keepdim=True))
    scale = torch.ldexp(torch.ones_like(b[:, :1, :, :1]), p)
    mid, low, high = (rounded(t / scale) * scale for t in (b, b - be, b + be))
    reach = (b.abs() + be).amax((1, 3), keepdim=True), (b.abs() - be).clamp_min(0).amax((1, 3), keepdim=True)
    other = (power(reach[0]) != p) | (power(reach[1]) != p)
    extra = torch.where(other, scale * 2.0 ** -8, torch.zeros_like(scale))
    far = torch.maximum(high - mid, mid - low) + extra
    return back(mid, v), back(far, v)


def eights(v):
    """The largest magnitude of each eight neighbours."""
    w = padded(v, 1, 8)
    return w.view(w.shape[0], -1, 8).abs().amax(2)


def product(q, p):
    """q p^T of coded pairs."""
    (qv, qe), (pv, pe) = q, p
    qa, pa = qv.abs(), pv.abs()
    span = (qa + qe) @ (pa + pe).T
    cut = 7 * 2.0 ** -13 * (eights(qa + qe) @ eights(pa + pe).T)
    return qv @ pv.T, qa @ pe.T + qe @ pa.T + qe @ pe.T + cut + (qv.shape[1] / 8 + 18) * U32 * span
