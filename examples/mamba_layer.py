"""A selective state space layer on the library's operators: training steps, a
prompt of packed sequences, and the same tokens one at a time.

    python examples/mamba_layer.py [--width 256] [--tokens 200] [--dtype bf16]

The layer is norm -> projection -> short convolution -> selective scan with a
gate -> projection, added to its input.  The library gives every operator's
forward and backward pass; ``Norm``, ``Conv`` and ``Scan`` hand them to torch's
autograd, the two projections are torch's.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mamba_ssd_chunked_02_amd as ssd  # noqa: E402


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, mean, rstd = ssd.ssd_norm_fwd(x, weight, bias)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        g = ssd.ssd_norm_bwd(x, weight, mean, rstd, dy.contiguous())
        return g["dx"], g["dweight"], g["dbias"]


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, cu):
        ctx.save_for_backward(x, weight, bias)
        ctx.cu = cu
        return ssd.ssd_conv_fwd(x, weight, bias, cu_seqlens=cu, final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias = ctx.saved_tensors
        g = ssd.ssd_conv_bwd(x, weight, bias, dy.contiguous(), cu_seqlens=ctx.cu)
        return g["dx"], g["dweight"], g["dbias"], None


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, raw, bias, A, B, C, D, z, cu):
        ctx.save_for_backward(x, raw, bias, A, B, C, D, z)
        ctx.cu = cu
        return ssd.ssd_selscan_fwd(x, raw, bias, A, B, C, D=D, z=z, cu_seqlens=cu,
                                   final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        x, raw, bias, A, B, C, D, z = ctx.saved_tensors
        g = ssd.ssd_selscan_bwd(x, raw, bias, A, B, C, dy.contiguous(), D=D, z=z, cu_seqlens=ctx.cu)
        return g["dx"], g["dd_raw"], g["dd_init"], g["dA"], g["dB"], g["dC"], g["dD"], g["dz"], None


class Layer:
    """One layer's parameters; weights of the projections in ``dtype``, the rest
    in float32."""

    def __init__(self, width, states=16, taps=4, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        E, rank = 2 * width, max(1, width // 16)
        self.width, self.E, self.N, self.rank, self.taps = width, E, states, rank, taps

        def normal(*shape, scale, dt=torch.float32):
            return (scale * torch.randn(shape, generator=g)).to(device=device, dtype=dt)

        step = torch.exp(torch.rand(E, generator=g) * math.log(100.0)) * 1e-3
        self.params = {
            "norm_w": torch.ones(width, device=device), "norm_b": torch.zeros(width, device=device),
            "w_in": normal(width, 2 * E, scale=width ** -0.5, dt=dtype),
            "conv_w": normal(taps, E, scale=taps ** -0.5), "conv_b": torch.zeros(E, device=device),
            "w_x": normal(E, rank + 2 * states, scale=E ** -0.5, dt=dtype),
            "w_dt": normal(rank, E, scale=rank ** -0.5, dt=dtype),
            "dt_b": (step + torch.log(-torch.expm1(-step))).to(device),
            "log_a": torch.log(torch.arange(1, states + 1).float())[:, None].repeat(1, E).to(device),
            "D": torch.ones(E, device=device),
            "w_out": normal(E, width, scale=E ** -0.5, dt=dtype),
        }

    def _scan_inputs(self, u):
        """Raw steps, B and C (views of one projection) of the convolved channels."""
        p, r, N = self.params, self.rank, self.N
        proj = u @ p["w_x"]
        B = proj[..., r:r + N].unsqueeze(-2)
        C = proj[..., r + N:].unsqueeze(-2)
        return proj[..., :r] @ p["w_dt"], B, C

    def __call__(self, x, cu=None):
        """x [b, L, width] (packed: b = 1 with cu) -> the same shape."""
        p = self.params
        xz = Norm.apply(x, p["norm_w"], p["norm_b"]) @ p["w_in"]
        u = Conv.apply(xz[..., :self.E], p["conv_w"], p["conv_b"], cu)
        raw, B, C = self._scan_inputs(u)
        y = Scan.apply(u, raw, p["dt_b"], -torch.exp(p["log_a"]), B, C, p["D"], xz[..., self.E:], cu)
        return x + y @ p["w_out"]

    def states(self, slots, dtype, device="cuda"):
        """Pools of convolution and scan states for serving."""
        return (torch.zeros((slots, self.taps - 1, self.E), dtype=dtype, device=device),
                torch.zeros((slots, self.N, self.E), device=device))

    @torch.no_grad()
    def prompt(self, x, cu, pools, slots):
        """The layer over packed prompts; their states go to the pools' rows."""
        p = self.params
        h, _, _ = ssd.ssd_norm_fwd(x, p["norm_w"], p["norm_b"])
        xz = h @ p["w_in"]
        u, conv_state = ssd.ssd_conv_fwd(xz[..., :self.E], p["conv_w"], p["conv_b"], cu_seqlens=cu)
        raw, B, C = self._scan_inputs(u)
        y, state = ssd.ssd_selscan_fwd(u, raw, p["dt_b"], -torch.exp(p["log_a"]), B, C, D=p["D"],
                                       z=xz[..., self.E:], cu_seqlens=cu)
        pools[0][slots.long()] = conv_state
        pools[1][slots.long()] = state
        return x + y @ p["w_out"]

    @torch.no_grad()
    def token(self, x, pools, slots):
        """One token x [b, width] of each sequence; the pools are updated in place."""
        p = self.params
        h, _, _ = ssd.ssd_norm_fwd(x, p["norm_w"], p["norm_b"])
        xz = h @ p["w_in"]
        u = ssd.ssd_conv_step(xz[..., :self.E], pools[0], p["conv_w"], p["conv_b"], slots=slots)
        raw, B, C = self._scan_inputs(u)
        y = ssd.ssd_selscan_step(u, raw, p["dt_b"], -torch.exp(p["log_a"]), B, C, pools[1],
                                 D=p["D"], z=xz[..., self.E:], slots=slots)
        return x + y @ p["w_out"]


def train(layer, x, target, steps=20, rate=0.02):
    """Gradient steps on a squared error; the losses."""
    losses = []
    for v in layer.params.values():
        v.requires_grad_(True)
    for _ in range(steps):
        loss = (layer(x).float() - target.float()).square().mean()
        grads = torch.autograd.grad(loss, list(layer.params.values()))
        with torch.no_grad():
            for v, g in zip(layer.params.values(), grads):
                # a step of fixed size in each parameter tensor's gradient direction
                v -= (rate * v.float().norm() / (g.float().norm() + 1e-12) * g.float()).to(v.dtype)
        losses.append(loss.item())
    for v in layer.params.values():
        v.requires_grad_(False)
    return losses


def serve(layer, lengths, new_tokens, dtype):
    """Prompts of these lengths, then new tokens one at a time; the largest
    difference to one packed pass over everything, relative to its values."""
    g = torch.Generator().manual_seed(1)
    whole = [torch.randn((n + new_tokens, layer.width), generator=g).to("cuda", dtype) for n in lengths]
    bounds = lambda ns: torch.tensor([0] + list(torch.tensor(ns).cumsum(0)), dtype=torch.int32,
                                     device="cuda")
    with torch.no_grad():
        full = layer(torch.cat(whole)[None], bounds([n + new_tokens for n in lengths]))[0]
    pools = layer.states(len(lengths) + 2, dtype)
    slots = torch.randperm(len(lengths) + 2, generator=g)[:len(lengths)].to(torch.int32).cuda()
    layer.prompt(torch.cat([w[:n] for w, n in zip(whole, lengths)])[None], bounds(lengths), pools,
                 slots)
    worst, at = 0.0, [0]
    for n in lengths:
        at.append(at[-1] + n + new_tokens)
    for t in range(new_tokens):
        y = layer.token(torch.stack([w[n + t] for w, n in zip(whole, lengths)]), pools, slots)
        ref = torch.stack([full[a + n + t] for a, n in zip(at, lengths)])
        worst = max(worst, ((y - ref).abs().max() / ref.abs().max()).item())
    return worst


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args(argv)
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[a.dtype]
    layer = Layer(a.width, dtype=dtype)
    g = torch.Generator().manual_seed(2)
    x = torch.randn((2, a.tokens, a.width), generator=g).to("cuda", dtype)
    target = x + 0.5 * torch.roll(x, 1, dims=1)
    losses = train(layer, x, target)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    worst = serve(layer, [a.tokens, 1, a.tokens // 3 + 1], 8, dtype)
    print(f"token by token against one pass: {worst:.2e} of the largest value")
    return losses, worst


if __name__ == "__main__":
    main()
