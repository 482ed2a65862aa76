"""A retention layer on the library's operators: training steps, a prompt of packed
sequences, and the same tokens one at a time.

    python examples/retention_layer.py [--width 256] [--tokens 200] [--dtype bf16]

The layer is norm -> projection -> linear attention with a decay per head -> group norm of
every head's output with a gate -> projection, added to its input.  The library gives every
operator's forward and backward pass; ``Norm``, ``Attend`` and ``GatedNorm`` hand them to
torch's autograd, the two projections are torch's.
"""
from __future__ import annotations

import argparse
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


class Attend(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, decay, scale, cu):
        ctx.save_for_backward(q, k, v, decay)
        ctx.scale, ctx.cu = scale, cu
        return ssd.ssd_linattn_fwd(q, k, v, decay, scale=scale, cu_seqlens=cu, final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        q, k, v, decay = ctx.saved_tensors
        g = ssd.ssd_linattn_bwd(q, k, v, decay, dy.contiguous(), scale=ctx.scale, cu_seqlens=ctx.cu)
        return g["dq"], g["dk"], g["dv"], None, None, None


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, weight, bias, groups):
        y, mean, rstd = ssd.ssd_groupnorm_fwd(x, groups, weight, bias, z=z)
        ctx.save_for_backward(x, z, weight, bias, mean, rstd)
        ctx.groups = groups
        return y

    @staticmethod
    def backward(ctx, dy):
        x, z, weight, bias, mean, rstd = ctx.saved_tensors
        g = ssd.ssd_groupnorm_bwd(x, ctx.groups, weight, bias, mean, rstd, dy.contiguous(), z=z)
        return g["dx"], g["dz"], g["dweight"], g["dbias"], None


class Layer:
    """One layer's parameters; weights of the projections in ``dtype``, the rest in float32.
    Keys are width / heads wide, values twice that."""

    def __init__(self, width, heads=4, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.width, self.heads, self.keys, self.values = width, heads, width // heads, 2 * width // heads
        self.scale = self.keys ** -0.5
        inner = heads * self.values
        self.parts = [width, width, inner, inner]

        def normal(*shape, scale, dt=torch.float32):
            return (scale * torch.randn(shape, generator=g)).to(device=device, dtype=dt)

        # a head keeps 1 - 2^-5, 1 - 2^-6, ... of its state each token
        self.decay = torch.log1p(-torch.exp2(-5.0 - torch.arange(heads))).to(device)
        self.params = {
            "norm_w": 1 + normal(width, scale=0.1), "norm_b": normal(width, scale=0.1),
            "w_in": normal(width, sum(self.parts), scale=width ** -0.5, dt=dtype),
            "head_w": 1 + normal(inner, scale=0.1), "head_b": normal(inner, scale=0.1),
            "w_out": normal(inner, width, scale=inner ** -0.5, dt=dtype),
        }

    def _heads(self, h):
        """q, k, v by heads and the gate z: views of one projection."""
        q, k, v, z = (h @ self.params["w_in"]).split(self.parts, dim=-1)
        H = self.heads
        return (q.unflatten(-1, (H, self.keys)), k.unflatten(-1, (H, self.keys)),
                v.unflatten(-1, (H, self.values)), z)

    def __call__(self, x, cu=None):
        """x [b, L, width] (packed: b = 1 with cu) -> the same shape."""
        p = self.params
        q, k, v, z = self._heads(Norm.apply(x, p["norm_w"], p["norm_b"]))
        y = Attend.apply(q, k, v, self.decay, self.scale, cu)
        # every token's heads on their own: tokens are the samples
        y = GatedNorm.apply(y.flatten(2).flatten(0, 1), z.flatten(0, 1), p["head_w"], p["head_b"], self.heads)
        return x + (y @ p["w_out"]).view(x.shape)

    def states(self, slots, device="cuda"):
        """A pool of states for serving."""
        return torch.zeros((slots, self.heads, self.keys, self.values), device=device)

    def _finish(self, x, y, z):
        p = self.params
        y = ssd.ssd_groupnorm_fwd(y.flatten(1), self.heads, p["head_w"], p["head_b"], z=z)[0]
        return x + y @ p["w_out"]

    @torch.no_grad()
    def prompt(self, x, cu, pool, slots):
        """The layer over packed prompts x [1, L, width]; their states go to the pool's rows."""
        p = self.params
        q, k, v, z = self._heads(ssd.ssd_norm_fwd(x, p["norm_w"], p["norm_b"])[0])
        y, state = ssd.ssd_linattn_fwd(q, k, v, self.decay, scale=self.scale, cu_seqlens=cu)
        pool[slots.long()] = state
        return self._finish(x[0], y[0], z[0])[None]

    @torch.no_grad()
    def token(self, x, pool, slots):
        """One token x [b, width] of each of b sequences."""
        p = self.params
        q, k, v, z = self._heads(ssd.ssd_norm_fwd(x, p["norm_w"], p["norm_b"])[0])
        y = ssd.ssd_linattn_step(q, k, v, self.decay, pool, scale=self.scale, slots=slots)
        return self._finish(x, y, z)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args(argv)
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(1)
    layer = Layer(a.width, dtype=dtype)

    # training: the next token's vector, on two sequences
    x = torch.randn((2, a.tokens + 1, a.width), generator=g).to("cuda", dtype)
    leaves = [t.requires_grad_() for t in layer.params.values()]
    losses = []
    for _ in range(a.steps):
        loss = (layer(x[:, :-1].contiguous()) - x[:, 1:]).float().square().mean()
        grads = torch.autograd.grad(loss, leaves)
        with torch.no_grad():
            for t, d in zip(leaves, grads):
                t -= 0.1 * d.to(t.dtype)
        losses.append(loss.item())
    print("losses", " ".join("%.4f" % v for v in losses))

    # serving: packed prompts, then their next tokens one by one, against the whole at once
    lengths = [a.tokens // 3, a.tokens - a.tokens // 3, 5]
    rest = 4
    seqs = [torch.randn((n + rest, a.width), generator=g).to("cuda", dtype) for n in lengths]

    def packed(parts):
        bounds = [0]
        for t in parts:
            bounds.append(bounds[-1] + t.shape[0])
        return torch.cat(parts)[None], torch.tensor(bounds, dtype=torch.int32, device="cuda")

    slots = torch.tensor([3, 0, 2], dtype=torch.int32, device="cuda")
    pool = layer.states(5)
    layer.prompt(*packed([t[:n] for t, n in zip(seqs, lengths)]), pool, slots)
    got = torch.stack([layer.token(torch.stack([t[n + i] for t, n in zip(seqs, lengths)]), pool, slots)
                       for i in range(rest)], 1)
    with torch.no_grad():
        whole, cu = packed(seqs)
        want = layer(whole, cu)[0]
    ends = cu[1:].tolist()
    worst = max((got[i] - want[e - rest:e]).abs().max().item() for i, e in enumerate(ends))
    size = want.abs().max().item()
    print("tokens one by one: off by %.2e of %.2f" % (worst, size))
    return losses, worst / size


if __name__ == "__main__":
    main()
