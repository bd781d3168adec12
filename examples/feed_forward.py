#!/usr/bin/env python3
"""A gated feed-forward block in BF16 behind its norm, with 8-bit activation checkpoints, trained for a step and then run for one token.

    python3 examples/feed_forward.py [--tokens T] [--width W] [--inner I] [--steps S] [--act silu]

Forward, for T tokens: n = norm(x), h = act(n W_g^T) * (n W_u^T) in one kernel, which also keeps both projections in
E4M3, y = x + h W_d^T. Backward, from the gradient of y: that of h (a product with W_d), those of both projections and h
itself again from the checkpoints, the weights' (products over the tokens, added in FP32), and through the norm that of x.
It prints how far each is from the same step in FP32, the checkpoints' size, and the time of each part.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import fp32_gemm_nn_amd as mg  # noqa: E402


class Block:
    """Weights of a norm and of a gated block (inner x width twice, width x inner), and the buffers of a step of `tokens` tokens."""

    def __init__(self, width, inner, tokens, act="silu", eps=1e-5, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.act, self.eps = act, eps
        weight = lambda rows, cols: (torch.randn(rows, cols, generator=g, device="cuda") / cols**0.5).bfloat16()  # noqa: E731
        self.wg, self.wu, self.wd = weight(inner, width), weight(inner, width), weight(width, inner)
        self.norm = 1 + 0.1 * torch.randn(width, generator=g, device="cuda")
        self.dwg, self.dwu, self.dwd = (torch.zeros(w.shape, device="cuda") for w in (self.wg, self.wu, self.wd))
        self.dnorm, self.rstd = torch.empty_like(self.norm), torch.empty(tokens, device="cuda")
        self.n, self.y, self.dn, self.dx = (torch.empty(tokens, width, dtype=torch.bfloat16, device="cuda") for _ in range(4))
        self.h, self.dh, self.dg, self.du = (torch.empty(tokens, inner, dtype=torch.bfloat16, device="cuda") for _ in range(4))
        self.g, self.gs = mg.fp8_empty(tokens, inner)
        self.u, self.us = mg.fp8_empty(tokens, inner)

    def forward(self, x):
        mg.rmsnorm(x, self.norm, self.eps, y=self.n, rstd=self.rstd)
        mg.gated(self.n, self.wg, self.wu, self.h, act=self.act, g=self.g, scale_g=self.gs, u=self.u, scale_u=self.us)
        return mg.linear("N", "T", 1.0, self.h, self.wd, 1.0, self.y, residual=x)

    def backward(self, x, dy):
        """From the gradient of y that of x. The weights' are added to those before. h is formed again: its buffer was free meanwhile."""
        mg.linear("N", "N", 1.0, dy, self.wd, 0.0, self.dh)
        mg.gated_backward(self.dh, self.g, self.u, self.dg, self.du, scale_g=self.gs, scale_u=self.us, act=self.act, h=self.h)
        mg.linear("T", "N", 1.0, dy, self.h, 1.0, self.dwd)
        mg.linear("T", "N", 1.0, self.dg, self.n, 1.0, self.dwg)
        mg.linear("T", "N", 1.0, self.du, self.n, 1.0, self.dwu)
        mg.linear("N", "N", 1.0, self.dg, self.wg, 0.0, self.dn)
        mg.linear("N", "N", 1.0, self.du, self.wu, 1.0, self.dn)
        mg.rmsnorm_backward(self.dn, x, self.norm, self.rstd, self.dx, self.dnorm, dh=dy)
        return self.dx

    def token(self, x):
        """One token, in buffers of its own."""
        n, y = torch.empty_like(x), torch.empty_like(x)
        h = torch.empty(x.shape[0], self.wg.shape[0], dtype=x.dtype, device=x.device)
        mg.rmsnorm(x, self.norm, self.eps, y=n)
        mg.gated(n, self.wg, self.wu, h, act=self.act)
        return mg.linear("N", "T", 1.0, h, self.wd, 1.0, y, residual=x)


def plain(block, x, dy):
    """The same step in FP32 by autograd: y, and the gradients of x, the three weights and the norm's."""
    leaves = [t.float().detach().requires_grad_() for t in (x, block.wg, block.wu, block.wd, block.norm)]
    x, wg, wu, wd, norm = leaves
    act = {"none": lambda z: z, "relu": torch.relu, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[block.act]
    n = x * torch.rsqrt(x.square().mean(1, keepdim=True) + block.eps) * norm
    y = x + (act(n @ wg.T) * (n @ wu.T)) @ wd.T
    y.backward(dy.float())
    return [y.detach()] + [t.grad for t in leaves]


def timed(call, steps):
    for _ in range(3):
        call()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        call()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) * 1e3 / steps


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=8192)
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--inner", type=int, default=8192)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--act", default="silu")
    args = p.parse_args(argv)
    block = Block(args.width, args.inner, args.tokens, args.act)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(args.tokens, args.width, generator=g, device="cuda").bfloat16() for _ in range(2))
    y = block.forward(x)
    dx = block.backward(x, dy)
    off = {}
    for name, got, want in zip(("y", "dx", "dwg", "dwu", "dwd", "dnorm"), (y, dx, block.dwg, block.dwu, block.dwd, block.dnorm), plain(block, x, dy)):
        off[name] = float((got.float() - want).norm() / want.norm())
        print(f"{name:6s} relative distance from FP32: {off[name]:.4f}")
    kept = sum(t.numel() * t.element_size() for t in (block.g, block.gs, block.u, block.us))
    print(f"kept of both projections: {kept / 2**20:.1f} MiB ({4 * args.tokens * args.inner / 2**20:.1f} in BF16)")
    print(f"forward  {timed(lambda: block.forward(x), args.steps):8.1f} us")
    print(f"backward {timed(lambda: block.backward(x, dy), args.steps):8.1f} us")
    print(f"token    {timed(lambda: block.token(x[:1]), args.steps):8.1f} us")
    one = block.token(x[:1]).float()
    off["token"] = float((one - y[:1].float()).norm() / y[:1].float().norm())
    print(f"one token, relative distance from its row of the batch: {off['token']:.5f}")
    return off


if __name__ == "__main__":
    main()
