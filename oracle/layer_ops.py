"""fp64 references of the operators around the scan (CPU, torch), written
token by token from their definitions; gradients come from torch's autograd
over these recurrences.  Test infrastructure only.

Shapes as in include/ssd.h: x [b, L, E] (packed: b = 1 with cu a list of
sequence bounds), weights [W, E], B and C [b, L, G, N], A and states [.., N, E].
"""
import torch


def spans(x, cu=None):
    """(batch row, first, last) of every sequence."""
    b, L = x.shape[:2]
    if cu is None:
        return [(i, 0, L) for i in range(b)]
    return [(0, u, v) for u, v in zip(cu[:-1], cu[1:])]


def silu(v):
    return v / (1 + torch.exp(-v))


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def norm(x, weight, bias, eps):
    mean = x.mean(-1)
    c = x - mean[..., None]
    rstd = (c.square().mean(-1) + eps).rsqrt()
    y = c * rstd[..., None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def conv(x, weight, bias, init=None, cu=None):
    """(y [b, L, E], final state [S, W - 1, E])"""
    W, E = weight.shape
    rows, finals = {}, []
    for s, (i, u, v) in enumerate(spans(x, cu)):
        front = x.new_zeros(W - 1, E) if init is None else init[s]
        line = torch.cat([front, x[i, u:v]])
        finals.append(line[v - u:])
        for t in range(u, v):
            a = (line[t - u:t - u + W] * weight).sum(0)
            rows[i, t] = silu(a if bias is None else a + bias)
    y = [torch.stack([rows.get((i, t), x.new_zeros(E)) for t in range(x.shape[1])])
         if x.shape[1] else x.new_zeros(0, E) for i in range(x.shape[0])]
    return torch.stack(y), torch.stack(finals)


def selscan(x, raw, dinit, A, B, C, D=None, z=None, init=None, cu=None):
    """(y [b, L, E], final state [S, N, E])"""
    N, E = A.shape
    G = B.shape[2]
    rows, finals = {}, []
    for s, (i, u, v) in enumerate(spans(x, cu)):
        h = x.new_zeros(N, E) if init is None else init[s]
        for t in range(u, v):
            d = softplus(raw[i, t] + dinit)
            Bt = B[i, t].T.repeat_interleave(E // G, 1)
            Ct = C[i, t].T.repeat_interleave(E // G, 1)
            h = torch.exp(d * A) * h + Bt * (d * x[i, t])
            o = (Ct * h).sum(0)
            if D is not None:
                o = o + D * x[i, t]
            if z is not None:
                o = o * silu(z[i, t])
            rows[i, t] = o
        finals.append(h)
    y = [torch.stack([rows.get((i, t), x.new_zeros(E)) for t in range(x.shape[1])])
         if x.shape[1] else x.new_zeros(0, E) for i in range(x.shape[0])]
    return torch.stack(y), torch.stack(finals)


def ssd_token(x, raw, dinit, B, C, state):
    """One token: x [b, H, P], raw [b, H], B, C [b, G, N], state [b, H, N, P]."""
    H, G = x.shape[1], B.shape[1]
    d = softplus(raw + dinit)
    Bh, Ch = (m.repeat_interleave(H // G, 1) for m in (B, C))
    h = torch.exp(-d)[..., None, None] * state + d[..., None, None] * Bh[..., None] * x[:, :, None]
    return (Ch[..., None] * h).sum(2), h


def gradients(fn, inputs, seeds):
    """Gradients of sum over outputs of <output, seed> for every tensor of the
    dict ``inputs`` (None entries stay None); ``fn`` takes them by name."""
    leaves = {k: (None if v is None else v.detach().clone().requires_grad_(True))
              for k, v in inputs.items()}
    loss = sum((o * s).sum() for o, s in zip(fn(**leaves), seeds) if s is not None)
    named = [k for k, v in leaves.items() if v is not None]
    if not getattr(loss, "requires_grad", False):  # no token: nothing depends on the inputs
        return {k: torch.zeros_like(leaves[k]) for k in named}
    got = torch.autograd.grad(loss, [leaves[k] for k in named], allow_unused=True)
    return {k: (torch.zeros_like(leaves[k]) if g is None else g) for k, g in zip(named, got)}
