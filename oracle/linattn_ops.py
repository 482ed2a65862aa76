"""fp64 references of linear attention with a decay per head and of group norm (CPU, torch),
written from their definitions; gradients come from torch's autograd over them.  Test
infrastructure only.

Shapes as in include/ssd.h: q [b, L, H, K], k [b, L, G, K], v [b, L, G, V] (packed: b = 1 with
cu a list of sequence bounds), decay [H], states [S, H, K, V].
"""
import torch

from oracle.layer_ops import silu, spans


def linattn(q, k, v, decay, scale=1.0, init=None, cu=None, reverse=False):
    """(y [b, L, H, V], final state [S, H, K, V])"""
    b, L, H, K = q.shape
    G, V = v.shape[2:]
    k, v = (t.repeat_interleave(H // G, 2) for t in (k, v))
    rate = torch.exp(decay)[:, None, None]
    y = [[None] * L for _ in range(b)]
    final = []
    for i, (row, first, last) in enumerate(spans(q, cu)):
        h = q.new_zeros((H, K, V)) if init is None else init[i]
        for t in (reversed(range(first, last)) if reverse else range(first, last)):
            h = rate * h + k[row, t, :, :, None] * v[row, t, :, None]
            y[row][t] = scale * (q[row, t, :, :, None] * h).sum(1)
        final.append(h)
    zero = q.new_zeros((H, V))
    rows = [torch.stack([zero if u is None else u for u in r]) if r else q.new_zeros((0, H, V)) for r in y]
    return torch.stack(rows), torch.stack(final)


def linattn_grads(q, k, v, decay, dy, d_final=None, **kw):
    """Gradients of <y, dy> + <final, d_final> by autograd: dq, dk, dv, dinit_state."""
    init = kw.pop("init", None)
    b, L, H, K = q.shape
    S = len(spans(q, kw.get("cu")))
    init = q.new_zeros((S, H, K, v.shape[3])) if init is None else init
    leaves = [t.clone().requires_grad_() for t in (q, k, v, init)]
    y, final = linattn(*leaves[:3], decay, init=leaves[3], **kw)
    loss = (y * dy).sum() + (0 if d_final is None else (final * d_final).sum())
    got = torch.autograd.grad(loss, leaves, allow_unused=True)
    return dict(zip(("dq", "dk", "dv", "dinit_state"),
                    (torch.zeros_like(t) if g is None else g for g, t in zip(got, leaves))))


def groupnorm(x, groups, weight=None, bias=None, z=None, activation=None, eps=1e-5):
    """(y, mean [n, G], rstd [n, G]) of x [n, ..., C]"""
    n, C = x.shape[0], x.shape[-1]
    xg = x.reshape(n, -1, groups, C // groups)
    mean = xg.mean((1, 3))
    c = xg - mean[:, None, :, None]
    rstd = (c.square().mean((1, 3)) + eps).rsqrt()
    u = (c * rstd[:, None, :, None]).reshape(x.shape)
    if weight is not None:
        u = u * weight
    if bias is not None:
        u = u + bias
    if activation == "silu":
        u = silu(u)
    if z is not None:
        u = u * silu(z)
    return u, mean, rstd
