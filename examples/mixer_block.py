"""A channel-mixing block on the network's activations, trained and served.

The features of a 3x3 convolution (NHWC, 96 channels, fp16) are a matrix with
a row for each pixel.  On it stands a block of a dense layer and a gated
feed-forward part, both residual:

    u = x + gelu(x w^T + bias)
    y = u + ffn(u)

Some steps of gradient descent fit it to a target.  What the forward pass
keeps for the backward pass is held in 8 bits: the inputs x and u, the dense
layer's and the block's pre-activations.  Then the same weights serve single
pixels, with nothing kept.

    python examples/mixer_block.py [--steps 30]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import unet_x3_convolution_amd as U  # noqa: E402

F16 = U.OIDN_F16


def buffer(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


class MixerBlock:
    """Weights (fp32 for the optimiser, fp16 for the kernels) and the buffers of m rows of d channels, f hidden."""

    def __init__(self, m, d, f, generator):
        self.m, self.d, self.f = m, d, f
        new = lambda *shape: torch.randn(*shape, generator=generator, device="cuda") * shape[-1] ** -0.5  # noqa: E731
        self.master = {"w": new(d, d), "bias": torch.zeros(d, device="cuda"), "w_in": new(2 * f, d),
                       "b_in": torch.zeros(2 * f, device="cuda"), "w_out": new(d, f) * 0.1,
                       "b_out": torch.zeros(d, device="cuda")}
        self.grad = {k: torch.empty_like(v, dtype=torch.float16 if v.dim() == 2 else torch.float32)
                     for k, v in self.master.items()}
        rows = lambda: torch.empty(m, d, dtype=torch.float16, device="cuda")  # noqa: E731
        self.u, self.y, self.du, self.dx = rows(), rows(), rows(), rows()
        ckpt = lambda n: buffer(U.oidn_ckpt_bytes(m, n))  # noqa: E731
        self.x8, self.u8, self.z8, self.ab8 = ckpt(d), ckpt(d), ckpt(d), buffer(2 * U.oidn_ckpt_bytes(m, f))
        both = U.OIDN_X_CKPT8 | U.OIDN_Z_CKPT8
        self.workspace = buffer(max(
            U.oidn_linear_workspace_bytes(m, d, d, F16), U.oidn_ffn_workspace_bytes(m, d, f, F16),
            U.oidn_linear_backward_workspace_bytes(m, d, d, U.OIDN_ACT_GELU, F16, both),
            U.oidn_ffn_backward_workspace_bytes(m, d, f, F16, both)))
        self.cast()

    def cast(self):
        self.param = {k: v.half() if v.dim() == 2 else v for k, v in self.master.items()}

    def forward(self, x, u, y, m, keep):
        """y of the first m rows of x; keep: hold what the backward pass reads, in 8 bits."""
        d, f, p, ws = self.d, self.f, self.param, self.workspace
        flag = U.OIDN_Z_CKPT8 if keep else 0
        if keep:
            U.oidn_ckpt_pack(x, d, m, d, self.x8, F16)
        U.oidn_linear(x, d, p["w"], d, p["bias"], x, d, u, d, self.z8 if keep else None, 0, m, d, d,
                      U.OIDN_ACT_GELU, F16, flag, ws, ws.numel())
        if keep:
            U.oidn_ckpt_pack(u, d, m, d, self.u8, F16)
        U.oidn_ffn(u, d, p["w_in"], p["b_in"], p["w_out"], p["b_out"], u, d, y, d, self.ab8 if keep else None, m, d, f,
                   U.OIDN_ACT_SILU, F16, flag, ws, ws.numel())

    def backward(self, dy):
        """Gradients of the weights into self.grad, of the input into self.dx."""
        m, d, f, p, g, ws = self.m, self.d, self.f, self.param, self.grad, self.workspace
        both = U.OIDN_X_CKPT8 | U.OIDN_Z_CKPT8
        U.oidn_ffn_backward(dy, d, self.u8, 0, self.ab8, p["w_in"], p["w_out"], dy, d, self.du, d, g["w_in"],
                            g["b_in"], g["w_out"], g["b_out"], m, d, f, U.OIDN_ACT_SILU, F16, both, ws, ws.numel())
        U.oidn_linear_backward(self.du, d, self.x8, 0, self.z8, 0, p["w"], d, self.dx, d, g["w"], d, g["bias"], m, d, d,
                               U.OIDN_ACT_GELU, F16, both, ws, ws.numel())
        self.dx += self.du                        # through the first residual

    def step(self, rate, scale):
        for k, v in self.master.items():
            v.add_(self.grad[k].float(), alpha=-rate / scale)
        self.cast()


def features(h, w, d, generator):
    """d channels of a 3x3 convolution with ReLU over random pixels."""
    import numpy as np
    r = np.random.default_rng(3)
    x = torch.randn(h, w, 32, generator=generator, device="cuda").half()
    weight = (r.standard_normal((d, 3, 3, 32)) * (2 / 288) ** 0.5).astype("float32")
    packed = buffer(U.oidn_conv3x3_weights_bytes(32, 0, d, F16))
    U.oidn_conv3x3_pack_weights(weight, np.zeros(d, "float32"), 32, 0, d, F16, packed)
    y = torch.empty(h, w, d, dtype=torch.float16, device="cuda")
    U.oidn_conv3x3(x, h, w, 32, packed, y, d, F16, F16, U.OIDN_RELU)
    return y.view(h * w, d)


def main(steps=30, h=68, w=120, d=96, f=256, rate=0.001, scale=1024.0):
    """Returns (losses, largest difference of a served pixel from the trained pass)."""
    torch.cuda.set_device(0)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = features(h, w, d, g)
    target = torch.tanh(x.float() @ torch.randn(d, d, generator=g, device="cuda") * d ** -0.5)
    block = MixerBlock(h * w, d, f, g)
    losses = []
    for k in range(steps):
        block.forward(x, block.u, block.y, block.m, keep=True)
        off = block.y.float() - target
        losses.append(float(off.square().mean()))
        # the loss is scaled so that small gradients survive fp16
        block.backward((off * (2 * scale / block.m)).half())
        block.step(rate, scale)
        if k % 10 == 0 or k == steps - 1:
            print(f"step {k}: loss {losses[-1]:.5f}", flush=True)
    block.forward(x, block.u, block.y, block.m, keep=False)
    u, y = torch.empty(1, d, dtype=torch.float16, device="cuda"), torch.empty(1, d, dtype=torch.float16, device="cuda")
    pixel = x.shape[0] // 2
    block.forward(x[pixel:pixel + 1], u, y, 1, keep=False)
    off = float((y[0].float() - block.y[pixel].float()).abs().max())
    print(f"one pixel served: at most {off:.2e} from the whole image's pass", flush=True)
    return losses, off


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    main(ap.parse_args().steps)
