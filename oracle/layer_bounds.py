"""fp64 values of the selective scan and its gradients together with bounds on what a
float32 evaluation may be off by, entry by entry (CPU, torch).  Test infrastructure only.

Every quantity is carried as (value, size, error): ``size`` is the same expression over
absolute values, which bounds every partial result of any order of evaluation (chunks
from zero, folds of states) whatever cancels in the value; ``error`` adds up the roundings
that reach it, u = 2^-24 each, of the terms' sizes:

  d   |z| u of the sum raw + d_init, and (8 + 1.25 |z|) u of softplus: the rounded exponent
      and its factor, the hardware's exp2 and reciprocal (2 u each), four roundings
  a   |d A| (err(d) / d + 32 u) + 2 u: the rounded rate and product, and the sum of d where
      the decay of a chunk, a run or a span is formed from it, through the exponential; and
      exp2's own
  h   4 u a token: product and sum, in the chunk and where chunks are joined
  silu(z), sigmoid(z), silu'(z)   (|z| + 6) u, (|z| + 4) u, 16 (1 + |z|) u
  sums  one u of the sum's size for each addition on the longest path
"""
import torch

U = 2.0 ** -24


def selscan(x, raw, dinit, A, B, C, D, z, init, dy, d_final, spans, sums):
    """Dict of name -> (value, bound) for y, final, and the gradients by their binding
    names.  x, raw, z, dy [T, E] (z None: no gate), B, C [T, G, N], init, d_final
    [S, N, E], all float64; ``spans``: (first, last) of the sequences; ``sums``: additions
    on the longest path of a sum over channels and over tokens."""
    T, E = x.shape
    N, G = A.shape[0], B.shape[1]
    over_channels, over_tokens = sums
    B, C = (m.transpose(1, 2).repeat_interleave(E // G, 2) for m in (B, C))  # [T, N, E]
    zr = raw + dinit
    d = torch.logaddexp(zr, torch.zeros_like(zr))
    ed = (8 + 2.25 * zr.abs()) * U  # relative
    sig = torch.sigmoid(zr)
    esig = (2 * zr.abs() + 4) * U
    u, eu = d * x, ed + U
    if z is None:
        gate, egate, slope, eslope = torch.ones_like(x), torch.zeros_like(x), None, None
    else:
        sz = torch.sigmoid(z)
        gate, egate = z * sz, (z.abs() + 6) * U
        slope, eslope = sz * (1 + z * (1 - sz)), 16 * (1 + z.abs()) * U
    w, ew = dy * gate, egate + U
    a = torch.exp(d[:, None] * A)
    ea = (d[:, None] * A).abs() * (ed[:, None] + 32 * U) + 2 * U
    h = torch.zeros(T, N, E, dtype=torch.float64)     # after token t
    hs, he = torch.zeros_like(h), torch.zeros_like(h)  # sizes, errors
    p, ps, pe = (torch.zeros_like(h) for _ in range(3))  # before token t
    g, gs, ge = (torch.zeros_like(h) for _ in range(3))
    q, qs, qe = (torch.zeros_like(h) for _ in range(3))  # a g
    final, efinal, dinit_state, edinit = (torch.zeros_like(init) for _ in range(4))
    for s, (first, last) in enumerate(spans):
        v, vs, ve = init[s], init[s].abs(), torch.zeros_like(init[s])
        for t in range(first, last):
            p[t], ps[t], pe[t] = v, vs, ve
            bu = B[t] * u[t]
            ve = a[t] * ve + a[t] * vs * (ea[t] + 4 * U) + bu.abs() * (eu[t] + 4 * U)
            v, vs = a[t] * v + bu, a[t] * vs + bu.abs()
            h[t], hs[t], he[t] = v, vs, ve
        final[s], efinal[s] = v, ve
        v, vs, ve = d_final[s], d_final[s].abs(), torch.zeros_like(init[s])
        for t in range(last - 1, first - 1, -1):
            cw = C[t] * w[t]
            ve = ve + cw.abs() * (ew[t] + 2 * U) + 2 * U * (vs + cw.abs())
            v, vs = v + cw, vs + cw.abs()
            g[t], gs[t], ge[t] = v, vs, ve
            ve = a[t] * ve + a[t] * vs * (ea[t] + 4 * U)
            v, vs = a[t] * v, a[t] * vs
            q[t], qs[t], qe[t] = v, vs, ve
        dinit_state[s], edinit[s] = v, ve

    def total(value, size, error, dim, additions):
        return value.sum(dim), size.sum(dim), error.sum(dim) + additions * U * size.sum(dim)

    def per_group(v):  # [T, N, E] summed over a group's channels: [T, G, N]
        return v.unflatten(2, (G, E // G)).sum(3).transpose(1, 2)

    out, outs, oute = total(C * h, (C * hs).abs(), C.abs() * he, 1, N + 4)
    if D is not None:
        out, outs = out + D * x, outs + (D * x).abs()
        oute = oute + 4 * U * outs
    y = out * gate
    gb, gbs, gbe = total(g * B, gs * B.abs(), ge * B.abs(), 1, N + 4)
    sv, ss = q * p, qs * ps
    se = qe * ps + qs * pe + 2 * U * ss
    sa, sas, sae = total(A * sv, (A * ss).abs(), A.abs() * (se + 4 * U * ss), 1, N + 4)
    Dw = w * D if D is not None else torch.zeros_like(w)
    dx = Dw + d * gb
    dd = x * gb + sa
    edd = x.abs() * gbe + sae + 3 * U * (x.abs() * gbs + sas)
    ddr = dd * sig
    sddr = (x.abs() * gbs + sas) * sig
    eddr = edd * sig + sddr * (esig + U)
    res = {"y": (y, oute * gate.abs() + outs * gate.abs() * (egate + 2 * U)),
           "final": (final, efinal),
           "dx": (dx, Dw.abs() * (ew + 3 * U) + d * (gbe + gbs * (ed + 3 * U))),
           "dd_raw": (ddr, eddr), "dinit_state": (dinit_state, edinit)}
    if z is not None:
        res["dz"] = (dy * out * slope, dy.abs() * (oute * slope.abs() + outs * (eslope + 2 * U)))
    for name, value, size, error in (
            ("dB", g * u[:, None], gs * u[:, None].abs(), ge * u[:, None].abs() + gs * (u * eu)[:, None].abs()),
            ("dC", h * w[:, None], hs * w[:, None].abs(), he * w[:, None].abs() + hs * (w * ew)[:, None].abs())):
        res[name] = (per_group(value), per_group(error) + (over_channels + 2) * U * per_group(size))
    for name, value, size, error in (
            ("dA", d[:, None] * sv, d[:, None] * ss, d[:, None] * (se + ss * ed[:, None])),
            ("dD", w * x, (w * x).abs(), (w * x).abs() * ew), ("dd_init", ddr, sddr, eddr)):
        res[name] = (value.sum(0), error.sum(0) + (over_tokens + 2) * U * size.sum(0))
    return res
