"""Cases of what stands in and around a block over activation rows: the dense
layer in 8-bit floating point with a scale for every block of 128 values, the
norms before and after a block with its gate, residual scale and dropout, and
dropout by itself.

Rows are pixels (or tokens), columns are channels.  `own` selects the library's
kernels; otherwise the operators are computed in their plain form, in 32 bits,
rounded once to the storage type at the end.
"""
import math

import torch

own = False

_TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
_BLOCK = 128       # values that share a scale
_LARGEST = 448.0   # of e4m3
_EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new row through a square layer whose weights are kept in 8 bits, as in serving
        dict(name="fp8 one row", op="linear8", type="bf16", m=1, k=4096, n=4096, act="none", bias=True, residual=True,
             save=False, pad=0),
        # the 96 channels of a 1920 x 1080 frame's deepest level (120 x 68 pixels), widened; z kept for training
        dict(name="fp8 deepest level", op="linear8", type="fp16", m=8160, k=96, n=384, act="gelu", bias=True,
             residual=False, save=True, pad=0),
        # a large layer over many rows: the matrix cores' 8-bit rate
        dict(name="fp8 large", op="linear8", type="bf16", m=8192, k=4096, n=4096, act="gelu", bias=True, residual=True,
             save=False, pad=0),
        # the gradients of odd sizes, rows inside wider buffers: nothing is aligned, every block ends in a part
        dict(name="fp8 backward odd", op="linear8_backward", type="fp16", m=1021, k=515, n=771, act="silu",
             bias=True, pad=5),
        # the gradients of a large layer, its new weights taken to 8 bits: the most work of all
        dict(name="fp8 backward large", op="linear8_backward", type="bf16", m=8192, k=2048, n=4096, act="gelu",
             bias=True, pad=0),
        # one new row between two blocks: the residual sum and the next block's norm, as in serving
        dict(name="norms one row", op="norm", type="bf16", m=1, n=4096, after="none", next="rms", groups=0, p=0.0,
             scale=1.0, shift=False, pad=0),
        # a quarter-resolution frame (480 x 272 pixels) before a block: many short rows
        dict(name="norm pixels", op="norm", type="fp16", m=130560, n=32, after="off", next="layer", groups=0, p=0.0,
             scale=1.0, shift=True, pad=0),
        # between two blocks of a large network in training, a gate for each of 16 sequences
        dict(name="norms large", op="norm", type="bf16", m=16384, n=4096, after="rms", next="rms", groups=16, p=0.1,
             scale=1.0, shift=False, pad=0),
        # the gradients around a block at the deepest level, two images with a gate each, in single precision
        dict(name="norms backward deepest level", op="norm_backward", type="fp32", m=8160, n=96, after="layer",
             next="layer", groups=2, p=0.1, scale=0.8, shift=True, pad=0),
        # the same of a large network
        dict(name="norms backward large", op="norm_backward", type="bf16", m=16384, n=4096, after="rms", next="rms",
             groups=1, p=0.1, scale=1.0, shift=False, pad=0),
        # a level's activations (240 x 136 pixels, 112 channels)
        dict(name="dropout level", op="dropout", type="fp16", m=32640, n=112, p=0.2, residual=False, pad=0),
        # a large network's rows, with the residual
        dict(name="dropout large", op="dropout", type="bf16", m=16384, n=4096, p=0.1, residual=True, pad=0),
    ]


def _size(rng, low, high):
    """Spread over the logarithm; half of them multiples of 32 (where the range has one), the rest as they fall."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 32 and rng.random() < 0.5:
        v = v // 32 * 32
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["linear8", "linear8", "linear8_backward", "norm", "norm", "norm_backward", "norm_backward",
                     "dropout"])
    pad = rng.choice([0, 0, 8, 3])
    if op in ("linear8", "linear8_backward"):
        c = dict(op=op, type=rng.choice(["fp16", "bf16"]), pad=pad, m=_size(rng, 1, 8192),
                 k=_size(rng, 8, 4096 if op == "linear8" else 2048), n=_size(rng, 8, 4096),
                 act=rng.choice(["none", "relu", "silu", "gelu"]), bias=rng.random() < 0.7)
        if op == "linear8":
            c.update(residual=rng.random() < 0.5, save=rng.random() < 0.3)
        return c
    n = _size(rng, 4, 8192)
    c = dict(op=op, type=rng.choice(["fp16", "bf16", "fp16", "bf16", "fp32"]), pad=pad, n=n,
             m=_size(rng, 1, min(131072, (1 << 25) // n)), p=rng.choice([0.0, 0.1, 0.1, 0.5]))
    if op == "dropout":
        return dict(c, p=max(c["p"], 0.05), residual=rng.random() < 0.5)
    c.update(after=rng.choice(["off", "none", "rms", "layer"]), next=rng.choice(["rms", "layer"]),
             shift=rng.random() < 0.5, scale=rng.choice([1.0, 1.0, 0.7]), groups=0)
    if c["after"] == "off":
        return dict(c, p=0.0, scale=1.0)
    if rng.random() < 0.5:
        c["next"] = "none"
    if rng.random() < 0.6:
        c["groups"] = _size(rng, 1, c["m"])
    return c


# ----------------------------------------------------------------- inputs
def _rows(g, m, n, t, pad, scale=1.0):
    """m x n normal values, the rows of a buffer that is `pad` columns wider."""
    buf = torch.randn(m, n + pad, generator=g, device="cuda", dtype=torch.float32)
    return buf.mul_(scale).to(t)[:, :n]


def prepare(case, seed):
    """Activations and gradients are normal, weights normal with variance 1 / inputs, biases small, the norms' weights
    and gates around 1: what a normalised network has."""
    c, t = case, _TYPES[case["type"]]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c, "t": t, "own": {}}
    m, n, pad, op = c["m"], c["n"], c["pad"], c["op"]
    vec = lambda *shape: torch.randn(*shape, generator=g, device="cuda") * 0.1  # noqa: E731
    if op in ("linear8", "linear8_backward"):
        # some channels are far larger than others, as in activations that are hard to keep in few bits
        s["x"] = (_rows(g, m, c["k"], torch.float32, pad) * torch.exp(vec(c["k"]) * 10)).to(t)
        if pad:
            wide = torch.zeros(m, c["k"] + pad, dtype=t, device="cuda")
            wide[:, :c["k"]] = s["x"]
            s["x"] = wide[:, :c["k"]]
        s["w"] = _rows(g, n, c["k"], t, 0, c["k"] ** -0.5)
        s["bias"] = vec(n) if c["bias"] else None
        if op == "linear8":
            s["residual"] = _rows(g, m, n, t, pad) if c["residual"] else None
        else:
            # z as the forward pass saved it
            s["dy"], s["z"] = _rows(g, m, n, t, pad), _rows(g, m, n, t, 0) if c["act"] != "none" else None
        return s
    # the generator's state lives on the device: a seed, and an offset that is another for each call
    s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda", dtype=torch.int64)
    if op == "dropout":
        s["x"] = _rows(g, m, n, t, pad)
        s["residual"] = _rows(g, m, n, t, pad) if c["residual"] else None
        return s
    # x, or the sum u that the forward pass left
    s["u" if op == "norm_backward" else "x"] = _rows(g, m, n, t, pad, 2.0)
    after, following = c["after"] != "off", c["next"] != "none"
    if after:
        s["o"] = _rows(g, m, n, t, pad)
        if c["after"] != "none":
            s["weight"] = 1 + vec(n)
            s["shift"] = vec(n) if c["shift"] else None
        if c["groups"]:
            s["gate_rows"] = -(-m // c["groups"])
            s["gate"] = 1 + vec(-(-m // s["gate_rows"]), n)
    if following:
        s["next_weight"] = 1 + vec(n)
        s["next_shift"] = vec(n) if c["shift"] else None
        if op == "norm_backward":
            s["dv"] = _rows(g, m, n, t, pad)
    if op == "norm_backward":
        s["du"] = _rows(g, m, n, t, pad)
    return s


# ------------------------------------------------------------- plain form
def _act(kind, z):
    if kind == "relu":
        return z.clamp_min(0)
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    return z


def _slope(kind, z):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    return torch.ones_like(z)


def _eight(x, square=False):
    """The values that e4m3 codes and a power of two for every 128 columns (square: for every 128 x 128) stand for."""
    m, n = x.shape
    high = -(-m // _BLOCK) * _BLOCK if square else m
    wide = torch.zeros(high, -(-n // _BLOCK) * _BLOCK, device=x.device)
    wide[:m, :n] = x
    blocks = wide.view(-1, _BLOCK if square else 1, wide.shape[1] // _BLOCK, _BLOCK)
    part, power = torch.frexp(blocks.abs().amax((1, 3), keepdim=True))
    power = torch.where(part <= _LARGEST / 512, power - 9, power - 8).clamp(-120, 120)
    codes = torch.ldexp(blocks, -power).to(torch.float8_e4m3fn).float()
    return torch.ldexp(codes, power).view(high, -1)[:m, :n]


def _plain_linear8(s, c, t):
    z = _eight(s["x"].float()) @ _eight(s["w"].float(), square=True).t()
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(c["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(t), "z": z.to(t)} if c["save"] else {"y": y.to(t)}


def _plain_linear8_backward(s, c, t):
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _slope(c["act"], s["z"].float())
    out = {"dx": (_eight(dz) @ _eight(s["w"].float(), square=True)).to(t),
           "dw": (_eight(dz.t().contiguous()) @ _eight(s["x"].float().t().contiguous()).t()).to(t)}
    if c["bias"]:
        out["dbias"] = dz.sum(0)
    return out


def _keep(rng, m, n, p):
    """Philox4x32-10 of counter (row * blocks + block of eight columns, offset) and key seed; 16 bits an element."""
    low = 0xffffffff
    blocks = -(-n // 8)
    at = torch.arange(m * blocks, device="cuda", dtype=torch.int64)
    a, b = at & low, at >> 32
    seed, offset = rng[0], rng[1]
    c, d = (offset & low).expand_as(a), ((offset >> 32) & low).expand_as(a)
    k0, k1 = seed & low, (seed >> 32) & low
    for r in range(10):
        p0, p1 = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (((p1 >> 32) & low) ^ b ^ k0, p1 & low, ((p0 >> 32) & low) ^ d ^ k1, p0 & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([a, b, c, d], 1)
    bits = torch.stack([words & 0xffff, words >> 16], 2).view(m, blocks * 8)[:, :n]
    return bits >= round(p * 65536)


def _gain(p):
    return 65536 / (65536 - round(p * 65536))


def _plain_dropout(s, c, t):
    x = s["x"].float()
    y = torch.where(_keep(s["rng"], *x.shape, c["p"]), x * _gain(c["p"]), torch.zeros_like(x))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(t)}


def _hat(kind, x):
    """Normalised rows and the factor that made them so."""
    if kind == "none":
        return x, None
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + _EPS)
    return x * r, r


def _hat_back(kind, g, hat, r):
    if kind == "none":
        return g
    d = g - hat * (g * hat).mean(1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(1, keepdim=True)
    return d * r


def _affine(s, prefix, hat):
    y = hat * s[prefix + "weight"] if s.get(prefix + "weight") is not None else hat
    return y + s[prefix + "shift"] if s.get(prefix + "shift") is not None else y


def _of_rows(s, m):
    """The gate of each row."""
    return s["gate"].repeat_interleave(s["gate_rows"], 0)[:m] if "gate" in s else None


def _plain_norm(s, c, t):
    out, u = {}, s["x"].float()
    m, n = u.shape
    if c["after"] != "off":
        b = _affine(s, "", _hat(c["after"], s["o"].float())[0])
        if c["p"]:
            b = torch.where(_keep(s["rng"], m, n, c["p"]), b * _gain(c["p"]), torch.zeros_like(b))
        gate = _of_rows(s, m)
        u = c["scale"] * u + (b if gate is None else gate * b)
        out["u"] = u.to(t)
        u = out["u"].float()
    if c["next"] != "none":
        out["v"] = _affine(s, "next_", _hat(c["next"], u)[0]).to(t)
    return out


def _plain_norm_backward(s, c, t):
    out, d = {}, s["du"].float()
    m, n = d.shape
    if c["next"] != "none":
        hat, r = _hat(c["next"], s["u"].float())
        dv = s["dv"].float()
        d = d + _hat_back(c["next"], dv * s["next_weight"], hat, r)
        out["dnext_weight"] = (dv * hat).sum(0)
        if s["next_shift"] is not None:
            out["dnext_shift"] = dv.sum(0)
    if c["after"] == "off":
        out["dx"] = d.to(t)
        return out
    out["dx"] = (c["scale"] * d).to(t)
    hat, r = _hat(c["after"], s["o"].float())
    keep = _keep(s["rng"], m, n, c["p"]) if c["p"] else None
    drop = lambda b: b if keep is None else torch.where(keep, b * _gain(c["p"]), torch.zeros_like(b))  # noqa: E731
    h = d
    gate = _of_rows(s, m)
    if gate is not None:
        groups, rows = s["gate"].shape[0], s["gate_rows"]
        each = torch.zeros(groups * rows, n, device=d.device)
        each[:m] = d * drop(_affine(s, "", hat))
        out["dgate"] = each.view(groups, rows, n).sum(1)
        h = d * gate
    h = drop(h)
    if c["after"] != "none":
        out["dweight"] = (h * hat).sum(0)
        if s["shift"] is not None:
            out["dshift"] = h.sum(0)
        h = h * s["weight"]
    out["do"] = _hat_back(c["after"], h, hat, r).to(t)
    return out


_PLAIN = {"linear8": _plain_linear8, "linear8_backward": _plain_linear8_backward, "norm": _plain_norm,
          "norm_backward": _plain_norm_backward, "dropout": _plain_dropout}


# ---------------------------------------------------- the library's calls
def _codes():
    import unet_x3_convolution_amd as U
    return (U, {"fp32": U.OIDN_F32, "fp16": U.OIDN_F16, "bf16": U.OIDN_BF16},
            {"none": U.OIDN_ACT_NONE, "relu": U.OIDN_ACT_RELU, "silu": U.OIDN_ACT_SILU, "gelu": U.OIDN_ACT_GELU},
            {"none": U.OIDN_NORM_NONE, "rms": U.OIDN_NORM_RMS, "layer": U.OIDN_NORM_LAYER})


def _kept(s, make):
    """The buffers that the program allocates once for a layer and uses for every call."""
    if not s["own"]:
        s["own"].update(make())
    return s["own"]


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def _pitch(x):
    return x.stride(0) if x is not None else 0


def _own_linear8(s, c, t):
    U, types, acts, _ = _codes()
    m, k, n, dt = c["m"], c["k"], c["n"], types[c["type"]]

    def make():
        w8 = _bytes(U.oidn_fp8_bytes(n, k))       # the weights are laid out once
        U.oidn_fp8_pack(s["w"], k, n, k, w8, None, dt, U.OIDN_FP8_SQUARE)
        return {"ws": _bytes(U.oidn_linear_fp8_workspace_bytes(m, k, n, dt, 0)), "w8": w8,
                "y": torch.empty(m, n, dtype=t, device="cuda"),
                "z": torch.empty(m, n, dtype=t, device="cuda") if c["save"] else None}

    o, x, r = _kept(s, make), s["x"], s["residual"]
    U.oidn_linear_fp8(x, x.stride(0), o["w8"], s["bias"], r, _pitch(r), o["y"], n, o["z"], n, m, k, n, acts[c["act"]],
                      dt, 0, o["ws"], o["ws"].numel())
    return {"y": o["y"], "z": o["z"]} if c["save"] else {"y": o["y"]}


def _own_linear8_backward(s, c, t):
    U, types, acts, _ = _codes()
    m, k, n, dt, act = c["m"], c["k"], c["n"], types[c["type"]], acts[c["act"]]
    new = lambda *shape: torch.empty(*shape, dtype=t, device="cuda")  # noqa: E731

    def make():
        return {"ws": _bytes(U.oidn_linear_fp8_backward_workspace_bytes(m, k, n, act, dt, U.OIDN_X_FP8)),
                "w8t": _bytes(U.oidn_fp8_bytes(k, n)), "x8t": _bytes(U.oidn_fp8_bytes(k, m)),
                "dx": new(m, k), "dw": new(n, k), "dbias": torch.empty(n, device="cuda") if c["bias"] else None}

    o, x, dy = _kept(s, make), s["x"], s["dy"]
    ws = o["ws"]
    U.oidn_fp8_pack(s["w"], k, n, k, None, o["w8t"], dt, U.OIDN_FP8_SQUARE)
    U.oidn_fp8_pack(x, x.stride(0), m, k, None, o["x8t"], dt, 0)
    U.oidn_linear_fp8_backward(dy, dy.stride(0), o["x8t"], 0, s["z"], n, o["w8t"], o["dx"], k, o["dw"], k, o["dbias"],
                               m, k, n, act, dt, U.OIDN_X_FP8, ws, ws.numel())
    out = {"dx": o["dx"], "dw": o["dw"]}
    return dict(out, dbias=o["dbias"]) if c["bias"] else out


def _own_norm(s, c, t):
    U, types, _, kinds = _codes()
    m, n, dt, x = c["m"], c["n"], types[c["type"]], s["x"]
    new = lambda: torch.empty(m, n, dtype=t, device="cuda")  # noqa: E731
    o = _kept(s, lambda: {"u": new() if c["after"] != "off" else None, "v": new() if c["next"] != "none" else None})
    if c["after"] == "off":
        U.oidn_norm(x, x.stride(0), s["next_weight"], s["next_shift"], o["v"], n, m, n, kinds[c["next"]], _EPS, dt)
        return {"v": o["v"]}
    U.oidn_norm_residual(s["o"], s["o"].stride(0), s.get("weight"), s.get("shift"), s.get("gate"), n,
                         s.get("gate_rows", 0), x, x.stride(0), c["scale"], c["p"], s["rng"], o["u"], n,
                         s.get("next_weight"), s.get("next_shift"), o["v"], n, m, n, kinds[c["after"]],
                         kinds[c["next"]], _EPS, dt)
    return {"u": o["u"], "v": o["v"]} if o["v"] is not None else {"u": o["u"]}


def _own_norm_backward(s, c, t):
    U, types, _, kinds = _codes()
    m, n, dt = c["m"], c["n"], types[c["type"]]
    after, gate_rows = c["after"] != "off", s.get("gate_rows", 0)

    def make():
        new = lambda: torch.empty(m, n, dtype=t, device="cuda")  # noqa: E731
        like = lambda name: torch.empty_like(s[name]) if s.get(name) is not None else None  # noqa: E731
        ws = (U.oidn_norm_residual_backward_workspace_bytes(m, n, gate_rows, dt) if after else
              U.oidn_norm_backward_workspace_bytes(m, n, dt))
        return dict(ws=_bytes(ws), dx=new(), do=new() if after else None,
                    **{"d" + name: like(name) for name in ("gate", "weight", "shift", "next_weight", "next_shift")})

    o, du, dv, u = _kept(s, make), s["du"], s.get("dv"), s["u"]
    ws = o["ws"]
    if not after:
        U.oidn_norm_backward(dv, dv.stride(0), u, u.stride(0), s["next_weight"], du, du.stride(0), o["dx"], n,
                             o["dnext_weight"], o["dnext_shift"], m, n, kinds[c["next"]], _EPS, dt, ws, ws.numel())
    else:
        U.oidn_norm_residual_backward(
            du, du.stride(0), dv, _pitch(dv), s["o"], s["o"].stride(0), s.get("weight"), s.get("shift"), s.get("gate"),
            n, gate_rows, u, u.stride(0), c["scale"], c["p"], s["rng"], s.get("next_weight"), o["dx"], n, o["do"], n,
            o["dgate"], n, o["dweight"], o["dshift"], o["dnext_weight"], o["dnext_shift"], m, n, kinds[c["after"]],
            kinds[c["next"]], _EPS, dt, ws, ws.numel())
    names = ("dx", "do", "dgate", "dweight", "dshift", "dnext_weight", "dnext_shift")
    return {name: o[name] for name in names if o[name] is not None}


def _own_dropout(s, c, t):
    U, types, _, _ = _codes()
    m, n, x, r = c["m"], c["n"], s["x"], s["residual"]
    o = _kept(s, lambda: {"y": torch.empty(m, n, dtype=t, device="cuda")})
    U.oidn_dropout(x, x.stride(0), r, _pitch(r), o["y"], n, m, n, c["p"], s["rng"], types[c["type"]])
    return {"y": o["y"]}


_OWN = {"linear8": _own_linear8, "linear8_backward": _own_linear8_backward, "norm": _own_norm,
        "norm_backward": _own_norm_backward, "dropout": _own_dropout}


def run(state):
    c = state["case"]
    return (_OWN if own else _PLAIN)[c["op"]](state, c, state["t"])


# ------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once; scales are a byte for 128 values.  A backward pass's x8 and w8
    are made on the way: x and w are what it reads."""
    c, m, n, op = case, case["m"], case["n"], case["op"]
    e = 4 if c["type"] == "fp32" else 2
    if op == "linear8":
        k = c["k"]
        return {"bytes": e * (m * k + m * n * (1 + c["residual"] + c["save"])) + (1 + 1 / _BLOCK) * n * k +
                4 * n * c["bias"], "flops": 2 * m * k * n}
    if op == "linear8_backward":
        k = c["k"]
        return {"bytes": e * (2 * m * k + m * n * (1 + (c["act"] != "none")) + 2 * n * k) + 4 * n * c["bias"],
                "flops": 4 * m * k * n}
    if op == "dropout":
        return {"bytes": e * m * n * (2 + c["residual"]), "flops": 2 * m * n}
    after, following = c["after"] != "off", c["next"] != "none"
    affine, vectors = after and c["after"] != "none", 4 * n * (1 + c["shift"])
    gate = 4 * n * c["groups"]
    if op == "norm":        # x, o; u, v
        return {"bytes": e * m * n * (1 + 2 * after + following) + vectors * (affine + following) + gate,
                "flops": 8 * m * n}
    # du, dv and u, o; dx, do
    return {"bytes": e * m * n * (2 + 2 * following + 2 * after) + 2 * vectors * (affine + following) + 2 * gate,
            "flops": 20 * m * n}


# --------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The definitions in 64 bits, output by output."""
    c, s = case, prepare(case, seed)
    t = s["t"]
    wide = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    get = lambda k, other=zero: wide.get(k, other)  # noqa: E731
    if c["op"] in ("linear8", "linear8_backward"):
        return _exact_linear8(c, wide, get)
    m, n = c["m"], c["n"]
    kept = _exact_keep(s["rng"], m, n, c["p"])
    if c["op"] == "dropout":
        return {"y": wide["x"] * kept + get("residual")}
    one = torch.ones((), dtype=torch.float64, device="cuda")
    got, back = {}, c["op"] == "norm_backward"

    def normal(kind, x):
        center = x.mean(dim=1, keepdim=True) if kind == "layer" else zero
        spread = ((x - center).pow(2).sum(dim=1, keepdim=True) / n + _EPS).sqrt() if kind != "none" else one
        return center, spread

    if c["after"] != "off":
        center, spread = normal(c["after"], wide["o"])
        hat = (wide["o"] - center) / spread
        which = torch.arange(m, device="cuda") // s["gate_rows"] if "gate" in s else None
        gate = wide["gate"][which] if which is not None else one
        branch = (hat * get("weight", one) + get("shift")) * kept
    u = wide["u"] if back else wide["x"]
    if c["after"] != "off" and not back:
        got["u"] = c["scale"] * u + gate * branch
        u = got["u"].to(t).double()
    if c["next"] != "none":
        ucenter, uspread = normal(c["next"], u)
        uhat = (u - ucenter) / uspread
    if not back:
        if c["next"] != "none":
            got["v"] = uhat * wide["next_weight"] + get("next_shift")
        return got

    def pull(kind, g, hat, spread):
        if kind == "none":
            return g
        along = torch.einsum("ij,ij->i", g, hat)[:, None] / n
        return (g - (g.sum(dim=1, keepdim=True) / n if kind == "layer" else 0) - along * hat) / spread

    d = wide["du"]
    if c["next"] != "none":
        dv = wide["dv"]
        got["dnext_weight"] = torch.einsum("ij,ij->j", dv, uhat)
        if "next_shift" in wide:
            got["dnext_shift"] = dv.sum(dim=0)
        d = d + pull(c["next"], dv * wide["next_weight"], uhat, uspread)
    got["dx"] = c["scale"] * d
    if c["after"] == "off":
        return got
    if which is not None:
        got["dgate"] = torch.zeros_like(wide["gate"]).index_add_(0, which, d * branch)
    h = d * gate * kept
    if c["after"] != "none":
        got["dweight"] = torch.einsum("ij,ij->j", h, hat)
        if "shift" in wide:
            got["dshift"] = h.sum(dim=0)
    got["do"] = pull(c["after"], h * get("weight", one), hat, spread)
    return got


def _exact_keep(rng, m, n, p):
    """0 or the factor of a kept element; the products of 32-bit words by 16-bit halves."""
    if not p:
        return torch.ones((), dtype=torch.float64, device="cuda")
    ones = (1 << 32) - 1
    per = (n + 7) // 8
    seed, offset = (int(v) & ((1 << 64) - 1) for v in rng.tolist())
    at = torch.arange(m, device="cuda")[:, None] * per + torch.arange(per, device="cuda")
    x = [at % (1 << 32), at // (1 << 32), torch.full_like(at, offset & ones), torch.full_like(at, offset >> 32)]
    key = [seed & ones, seed >> 32]

    def times(v, factor):
        low, high = v * (factor & 0xffff), v * (factor >> 16)        # below 2^48
        carried = (low >> 16) + high
        return carried >> 16, ((carried & 0xffff) << 16) | (low & 0xffff)

    for _ in range(10):
        (h0, l0), (h1, l1) = times(x[0], 0xD2511F53), times(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) & ones, (key[1] + 0xBB67AE85) & ones]
    halves = [v for w in x for v in (w % 65536, w // 65536)]
    limit = round(p * 65536)
    return (torch.stack(halves, dim=2).reshape(m, per * 8)[:, :n] >= limit).double() * (65536 / (65536 - limit))


def _exact_linear8(c, wide, get):
    normal_cdf = lambda v: torch.special.erfc(-v / math.sqrt(2.0)) / 2  # noqa: E731
    phi = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v),
           "gelu": lambda v: v * normal_cdf(v)}[c["act"]]

    def dphi(v):
        if c["act"] == "relu":
            return torch.where(v > 0, 1.0, 0.0).double()
        if c["act"] == "silu":
            return torch.sigmoid(v) + v * torch.sigmoid(v) * torch.sigmoid(-v)
        if c["act"] == "gelu":
            return normal_cdf(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        return torch.ones_like(v)

    def code(v, top):
        """v to the step of its binade, for the least power of two that holds top."""
        power = torch.ceil(torch.log2(top / _LARGEST)).clamp(-120, 120)
        power = torch.where(top > 0, power, torch.zeros_like(power))
        # log2 may be a rounding off at a border
        lower = (top > 0) & (top <= _LARGEST * torch.exp2(power - 1))
        power = power + (top > _LARGEST * torch.exp2(power)).double() - lower.double()
        v = v * torch.exp2(-power)
        step = torch.exp2((torch.frexp(v).exponent - 1).clamp_min(-6).double() - 3)
        return torch.round(v / step) * step * torch.exp2(power)

    def rows8(v):
        cols = torch.nn.functional.pad(v, (0, -v.shape[1] % _BLOCK)).unflatten(1, (-1, _BLOCK))
        return code(cols, cols.abs().max(2, keepdim=True).values).flatten(1)[:, :v.shape[1]]

    def square8(v):
        high, across = v.shape
        cells = torch.nn.functional.pad(v, (0, -across % _BLOCK, 0, -high % _BLOCK))
        cells = cells.unflatten(1, (-1, _BLOCK)).unflatten(0, (-1, _BLOCK))
        return code(cells, cells.abs().amax(dim=(1, 3), keepdim=True)).flatten(2).flatten(0, 1)[:high, :across]

    x, w = wide["x"], square8(wide["w"])
    if c["op"] == "linear8":
        z = torch.matmul(rows8(x), w.T) + get("bias")
        y = phi(z) + get("residual")
        return {"y": y, "z": z} if c["save"] else {"y": y}
    dz = wide["dy"] * dphi(wide["z"]) if "z" in wide else wide["dy"]
    got = {"dx": torch.matmul(rows8(dz), w), "dw": torch.matmul(rows8(dz.T.contiguous()), rows8(x.T.contiguous()).T)}
    return dict(got, dbias=dz.sum(dim=0)) if c["bias"] else got
