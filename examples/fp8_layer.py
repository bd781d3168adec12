#!/usr/bin/env python3
"""A linear layer in 8 bits behind its norm, trained for a step and then run for one token.

    python3 examples/fp8_layer.py [--tokens T] [--inner K] [--outer N] [--steps S]

Forward, for T tokens: h = x + residual, a = norm(h) (kept in BF16, and in E4M3 with a scale for each row and 128
columns), y = a W^T with W in E4M3 (a scale for each 128 x 128 block). Backward, from the gradient of y in E5M2:
that of a (a product with W^T), that of W (a product over the tokens, added in FP32), and through the norm those of
h and of its weight. It prints how far each is from the same step in FP32, and the time of each call.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import fp32_gemm_nn_amd as mg  # noqa: E402

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


class Layer:
    """Weights of a norm and of a linear layer (outer x inner), and the buffers of a step of up to `tokens` tokens."""

    def __init__(self, inner, outer, tokens, eps=1e-5, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.eps = eps
        self.weight = torch.randn(outer, inner, generator=g, device="cuda") / inner**0.5
        self.norm = 1 + 0.1 * torch.randn(inner, generator=g, device="cuda")
        self.w, self.ws = mg.fp8_empty(outer, inner, "tile", E4M3)
        self.wt, self.wts = mg.fp8_empty(inner, outer, "tile", E4M3)
        self.dweight, self.dnorm = torch.zeros_like(self.weight), torch.empty_like(self.norm)
        self.h, self.a, self.da, self.dx = (torch.empty(tokens, inner, dtype=torch.bfloat16, device="cuda") for _ in range(4))
        self.rstd = torch.empty(tokens, device="cuda")
        self.q, self.qs = mg.fp8_empty(tokens, inner, "row", E4M3)
        self.at, self.ats = mg.fp8_empty(inner, tokens, "row", E4M3)
        self.g, self.gs = mg.fp8_empty(tokens, outer, "row", E5M2)
        self.gt, self.gts = mg.fp8_empty(outer, tokens, "row", E5M2)
        self.y = torch.empty(tokens, outer, dtype=torch.bfloat16, device="cuda")
        self.update()

    def update(self):
        """After a change of the weight: it and its transpose in 8 bits."""
        mg.fp8_quantize(self.weight, self.w, self.ws, self.wt, self.wts, block="tile")

    def forward(self, x, residual):
        mg.rmsnorm(x, self.norm, self.eps, residual=residual, h=self.h, y=self.a, q=self.q, scale=self.qs, rstd=self.rstd)
        return mg.fp8_gemm(1.0, self.q, self.qs, self.w, self.ws, 0.0, self.y)

    def backward(self, dy, dh):
        """From the gradients of y and of h (past the norm): that of x and the residual. The weights' are kept."""
        mg.fp8_quantize(dy, self.g, self.gs, self.gt, self.gts)
        mg.fp8_quantize(self.a, qt=self.at, scale_t=self.ats)
        mg.fp8_gemm(1.0, self.g, self.gs, self.wt, self.wts, 0.0, self.da)
        mg.fp8_gemm(1.0, self.gt, self.gts, self.at, self.ats, 1.0, self.dweight, block="row")
        mg.rmsnorm_backward(self.da, self.h, self.norm, self.rstd, self.dx, self.dnorm, dh=dh)
        return self.dx

    def token(self, x, residual):
        """One token: h and y alone, in buffers of their own (kept by a user's program from call to call)."""
        h, (q, s) = torch.empty_like(x), mg.fp8_empty(1, x.shape[1])
        y = torch.empty(1, self.weight.shape[0], dtype=x.dtype, device=x.device)
        mg.rmsnorm(x, self.norm, self.eps, residual=residual, h=h, q=q, scale=s)
        return h, mg.fp8_gemm(1.0, q, s, self.w, self.ws, 0.0, y)


def plain(layer, x, residual, dy, dh):
    """The same step in FP32: y, and the gradients of x, W and the norm's weight."""
    h = (x.float() + residual.float()).bfloat16().float()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + layer.eps)
    a = h * rstd * layer.norm
    da = dy.float() @ layer.weight
    g, u = da * layer.norm, h * rstd
    dx = rstd * (g - u * (g * u).mean(1, keepdim=True)) + dh.float()
    return a @ layer.weight.T.contiguous(), dx, dy.float().T.contiguous() @ a, (da * u).sum(0)


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
    p.add_argument("--inner", type=int, default=4096)
    p.add_argument("--outer", type=int, default=8192)
    p.add_argument("--steps", type=int, default=20)
    args = p.parse_args(argv)
    layer = Layer(args.inner, args.outer, args.tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual, dh = (torch.randn(args.tokens, args.inner, generator=g, device="cuda").bfloat16() for _ in range(3))
    dy = torch.randn(args.tokens, args.outer, generator=g, device="cuda").bfloat16()
    y = layer.forward(x, residual)
    dx = layer.backward(dy, dh)
    off = {}
    for name, got, want in zip(("y", "dx", "dweight", "dnorm"), (y, dx, layer.dweight, layer.dnorm),
                               plain(layer, x, residual, dy, dh)):
        off[name] = float((got.float() - want).norm() / want.norm())
        print(f"{name:8s} relative distance from FP32: {off[name]:.4f}")
    print(f"forward  {timed(lambda: layer.forward(x, residual), args.steps):8.1f} us")
    print(f"backward {timed(lambda: layer.backward(dy, dh), args.steps):8.1f} us")
    print(f"weight   {timed(layer.update, args.steps):8.1f} us")
    print(f"token    {timed(lambda: layer.token(x[:1], residual[:1]), args.steps):8.1f} us")
    one = layer.token(x[:1], residual[:1])[1].float()
    off["token"] = float((one - y[:1].float()).norm() / y[:1].float().norm())
    print(f"one token, relative distance from its row of the batch: {off['token']:.4f}")
    return off


if __name__ == "__main__":
    main()
