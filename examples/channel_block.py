"""An int8 convolution followed by a residual channel block, forward and
backward, on the library's operators:

    acc = conv_fprop(image, filter)                        int32 accumulators, channels last
    h   = layer_norm(scale * acc)                          the stem's output
    n   = layer_norm(h) * gain + shift
    a   = gelu(n w1^T + b1)
    y   = a w2^T + b2 + h

and, for a loss gradient dy, the gradients of w1, b1, w2, b2, gain, shift and
h.  The convolution's int32 result is normalised as it is, the bias, GELU and
residual ride in the products' epilogues, and the skip's gradient in the layer
norm's.

    python examples/channel_block.py            # runs it, compares with a plain float32 computation, times it
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import int8_conv2d_fprop_gb300 as ic  # noqa: E402

SCALE = 2.0 ** -13  # of the quantised product image * filter


class ChannelBlock:
    """Weights of the block, and what its forward pass keeps for the backward."""

    def __init__(self, channels: int, hidden: int, device="cuda", dtype=torch.bfloat16, seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(*shape, generator=g, device=device) * scale

        self.w1 = normal(hidden, channels, scale=channels ** -0.5).to(dtype)
        self.b1 = normal(hidden, scale=0.1)
        self.w2 = normal(channels, hidden, scale=hidden ** -0.5).to(dtype)
        self.b2 = normal(channels, scale=0.1)
        self.gain = 1 + normal(channels, scale=0.1)
        self.shift = normal(channels, scale=0.1)

    def forward(self, h):
        rows = h.numel() // h.shape[-1]
        self.h = h
        self.mean = torch.empty(rows, device=h.device)
        self.rstd = torch.empty(rows, device=h.device)
        self.n = ic.conv_layer_norm(h, self.gain, self.shift, mean=self.mean, rstd=self.rstd)
        self.z = torch.empty(*h.shape[:-1], self.w1.shape[0], dtype=h.dtype, device=h.device)
        self.a = ic.conv_linear(self.n, self.w1, self.b1, activation="gelu", preact=self.z)
        return ic.conv_linear(self.a, self.w2, self.b2, residual=h)

    def backward(self, dy):
        """Gradients by name; "h" is the gradient that goes on to the stem."""
        g = {k: torch.empty_like(getattr(self, k)) for k in ("w1", "b1", "w2", "b2", "gain", "shift", "h")}
        da, dn = torch.empty_like(self.a), torch.empty_like(self.n)
        ic.conv_linear_grad(dy, self.a, self.w2, dx=da, dw=g["w2"], dbias=g["b2"])
        ic.conv_linear_grad(da, self.n, self.w1, preact=self.z, activation="gelu", dx=dn, dw=g["w1"], dbias=g["b1"])
        ic.conv_layer_norm_grad(dn, self.h, self.gain, self.mean, self.rstd, residual_grad=dy, dx=g["h"],
                                dgain=g["gain"], dshift=g["shift"])
        return g


def stem(image, weight, padding=(1, 1), dtype=torch.bfloat16):
    """int8 convolution and layer norm: [N, P, Q, K] rows of channels."""
    acc = ic.conv_fprop(image, weight, padding=padding).permute(0, 2, 3, 1)
    return ic.conv_layer_norm(acc, scale=SCALE, out=torch.empty(acc.shape, dtype=dtype, device=acc.device))


def inputs(batch, channels, size, out_channels, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def int8(*shape):
        t = torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)
        return t.contiguous(memory_format=torch.channels_last)

    dy = torch.randn(batch, size, size, out_channels, generator=g, device="cuda").to(torch.bfloat16)
    return int8(batch, channels, size, size), int8(out_channels, channels, 3, 3), dy


def plain(block, h, dy):
    """The block by float32 autograd: (y, gradients by name)."""
    p = {k: getattr(block, k).detach().float().requires_grad_() for k in ("w1", "b1", "w2", "b2", "gain", "shift")}
    p["h"] = h.detach().float().requires_grad_()
    n = torch.nn.functional.layer_norm(p["h"], (h.shape[-1],), p["gain"], p["shift"])
    a = torch.nn.functional.gelu(n @ p["w1"].t() + p["b1"])
    y = a @ p["w2"].t() + p["b2"] + p["h"]
    y.backward(dy.float())
    return y.detach(), {k: v.grad for k, v in p.items()}


def compare(batch=2, channels=64, size=14, out_channels=96, hidden=384):
    """Largest relative distance (2-norm) of the block's results from plain()'s."""
    image, weight, dy = inputs(batch, channels, size, out_channels)
    block = ChannelBlock(out_channels, hidden)
    h = stem(image, weight)
    y = block.forward(h)
    grads = block.backward(dy)
    want, want_grads = plain(block, h, dy)
    far = {"y": float((y.float() - want).norm() / want.norm())}
    far |= {k: float((grads[k].float() - v).norm() / v.norm()) for k, v in want_grads.items()}
    return far


def main():
    for name, far in compare().items():
        print(f"{name:6s} {far:.2e} from the float32 computation")
    image, weight, dy = inputs(32, 256, 56, 256)
    block = ChannelBlock(256, 1024)

    def step():
        block.forward(stem(image, weight))
        block.backward(dy)

    for _ in range(3):
        step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        step()
    end.record()
    torch.cuda.synchronize()
    print(f"32 x 256 x 56 x 56 convolution, 256 -> 1024 -> 256 block, forward and backward: {start.elapsed_time(end) / 10:.3f} ms")


if __name__ == "__main__":
    main()
