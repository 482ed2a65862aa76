"""Group norm, channels last, with an activation, on the GPU against the fp64 definition.

Tolerances.  An output of type t is the float32 result rounded once, off by at most eps(t) / 2
of its value.  The float32 result: xh is off by its own few roundings and by the statistics',
which are sums of N terms in blocks: 16 roundings and one for every doubling of N and every
256 terms of a thread, K = 32 + N / 64, of the largest |xh|; gradients that are sums over rows
have one more for every term.  Sizes are the largest entry of the exact output, at least that
of the products that it is the sum of.
"""
import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from oracle import linattn_ops as lo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FORMS = ("plain", "silu", "gate")


def within(got, ref, K, size, name):
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    half = torch.finfo(got.dtype).eps / 2 if got.dtype == torch.bfloat16 else 0.0
    err = (got.double().cpu() - ref).abs()
    tol = half * ref.abs() * (1 + half) + K * 2.0 ** -24 * max(size, 1e-30)
    bad = ~(err <= tol)
    assert not bad.any(), (name, int(bad.sum()), err.max().item(), size * K * 2.0 ** -24)


def make(dtype, shape, form, seed=0, shift=0.0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    C = shape[-1]
    r = lambda *s: torch.randn(s, generator=g)
    t = TYPES[dtype]
    return dict(x=(r(*shape) * (0.5 + torch.rand(C, generator=g)) + shift).to(t), weight=1 + 0.3 * r(C),
                bias=0.3 * r(C), z=r(*shape).to(t) if form == "gate" else None, dy=r(*shape).to(t),
                activation="silu" if form == "silu" else None)


def up(t):
    return None if t is None else t.to(DEV)


def d(t):
    return None if t is None else t.double()


def check(s, G, view=lambda t: t, affine=True, bwd=True, eps=1e-5):
    w, b = (s["weight"], s["bias"]) if affine else (None, None)
    x = view(up(s["x"]))
    kw = dict(z=None if s["z"] is None else view(up(s["z"])), activation=s["activation"])
    y, mean, rstd = m.ssd_groupnorm_fwd(x, G, up(w), up(b), eps=eps, **kw)
    leaf = [d(s["x"]).requires_grad_(), torch.ones(s["x"].shape[-1], dtype=torch.float64) if w is None else d(w),
            torch.zeros(s["x"].shape[-1], dtype=torch.float64) if b is None else d(b)]
    leaf = [leaf[0]] + [t.requires_grad_() for t in leaf[1:]]
    z = None if s["z"] is None else d(s["z"]).requires_grad_()
    ry, rm, rr = lo.groupnorm(leaf[0], G, leaf[1], leaf[2], z, s["activation"], eps)
    n, C = s["x"].shape[0], s["x"].shape[-1]
    N = s["x"].numel() // n // G
    K = 32 + N / 64
    xabs = d(s["x"]).abs().max().item()
    top = lambda t: t.detach().abs().max().item()
    # the mean's error is of x's size: relative to the deviations it grows with |x| / std
    grow = 1 + xabs * rr.max().item()
    within(mean, rm.detach(), K, xabs, "mean")
    within(rstd / rr.detach().float().to(DEV), torch.ones_like(rr), K * grow, 1.0, "rstd")
    size = max(top(ry), 1.0) * (1 if s["z"] is None else max(1.0, top(z)))
    within(y, ry.detach(), K * grow, size, "y")
    if not bwd:
        return y, None
    g = m.ssd_groupnorm_bwd(x, G, up(w), up(b), mean, rstd, view(up(s["dy"])), **kw)
    names = ["dx", "dweight", "dbias"] + (["dz"] if z is not None else [])
    ref = dict(zip(names, torch.autograd.grad((ry * d(s["dy"])).sum(), leaf + ([z] if z is not None else []))))
    assert sorted(g) == sorted(ref)
    rows = s["x"].numel() // C
    big = 4 * top(s["dy"]) * (1 if z is None else max(1.0, top(z))) * max(1.0, top(w) if w is not None else 1.0)
    within(g["dx"], ref["dx"], K * grow, big * rr.max().item() * 4, "dx")
    if z is not None:
        within(g["dz"], ref["dz"], K * grow, big * max(1.0, top(ry)), "dz")
    within(g["dweight"], ref["dweight"], K * grow + rows, big * 4, "dweight")
    within(g["dbias"], ref["dbias"], K * grow + rows, big, "dbias")
    return y, g


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,C,G", [(1, 1, 1), (5, 24, 8), (33, 7 * 5, 5), (130, 12 * 128, 12), (64, 2 * 77, 2),
                                   (9, 3 * 513, 3), (7, 1030, 1), (6, 2047, 1), (3, 5000, 1), (1000, 64, 8),
                                   (2, 6 * 1001, 6)])
def test_rows(dtype, form, n, C, G):
    """Every row on its own (one position)."""
    check(make(dtype, (n, C), form), G)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shape,G", [((2, 3, 6), 3), ((3, 1000, 10), 5), ((1, 7, 5, 320), 32), ((2, 4096, 24), 3),
                                     ((4, 35, 35, 77), 7), ((2, 2, 5003), 1), ((1, 1, 40, 8), 2), ((1, 900, 3), 1),
                                     ((130, 2, 64), 4), ((2, 65, 2056), 8)])
def test_maps(dtype, form, shape, G):
    check(make(dtype, shape, form), G)


@pytest.mark.parametrize("dtype", TYPES)
def test_without_weights(dtype):
    check(make(dtype, (40, 96), "silu"), 4, affine=False)
    check(make(dtype, (3, 50, 96), "gate"), 4, affine=False)


@pytest.mark.parametrize("shape,G", [((50, 256), 2), ((2, 3000, 16), 2)])
def test_large_mean(shape, G):
    """Values of 1000 +- 1: the deviations keep their bits."""
    check(make("f32", shape, "plain", shift=1000.0), G)


@pytest.mark.parametrize("shape", [(6, 32), (2, 70, 32)])
def test_constant_groups(shape):
    """No deviations: xh is 0 and rstd is 1 / sqrt(eps)."""
    x = torch.full(shape, 3.25, device=DEV)
    bias = torch.linspace(-1, 1, 32, device=DEV)
    y, mean, rstd = m.ssd_groupnorm_fwd(x, 4, None, bias, eps=1e-4)
    assert torch.equal(y, bias.expand(shape)) and (mean == 3.25).all()
    assert (rstd - 100).abs().max() < 100 * 4 * 2.0 ** -24


@pytest.mark.parametrize("shape", [(6, 40), (3, 70, 40)])
def test_nan_stays_in_its_group(shape):
    s = make("f32", shape, "plain")
    x = up(s["x"])
    clean, m0, _ = m.ssd_groupnorm_fwd(x, 4)
    x[1, ..., 10:12] = float("nan")
    x[2, ..., 30] = float("inf")
    y, mean, _ = m.ssd_groupnorm_fwd(x, 4)
    assert y[1, ..., 10:20].isnan().all() and mean[1, 1].isnan()
    y[1, ..., 10:20] = clean[1, ..., 10:20]
    assert not y[2, ..., 30:40].isfinite().any() or shape[0] == 0
    y[2, ..., 30:40] = clean[2, ..., 30:40]
    assert torch.equal(y, clean)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,G", [((20, 3 * 21), 3), ((2, 50, 3 * 21), 3), ((2, 6, 7, 2 * 32), 2)])
def test_views(dtype, shape, G):
    """Channels of a wider tensor, one element in; in place."""
    s = make(dtype, shape, "gate")

    def odd(t):
        wide = torch.full(shape[:-1] + (shape[-1] + 5,), 9.0, dtype=t.dtype, device=DEV)
        wide[..., 1:-4] = t
        return wide[..., 1:-4]

    y, g = check(s, G, view=odd)
    y0, g0 = check(s, G)
    assert torch.equal(y, y0) and all(torch.equal(g[k], g0[k]) for k in g)
    x = odd(up(s["x"]))
    y1, _, _ = m.ssd_groupnorm_fwd(x, G, up(s["weight"]), up(s["bias"]), z=up(s["z"]), y=x)
    assert y1 is x and torch.equal(x, y0)


def test_nothing():
    y, mean, _ = m.ssd_groupnorm_fwd(torch.zeros(0, 5, 8, device=DEV), 2)
    assert y.shape == (0, 5, 8) and mean.shape == (0, 2)
    g = m.ssd_groupnorm_bwd(y, 2, None, None, mean, mean, y)
    assert not g["dweight"].any() and not g["dbias"].any()


def test_gradients_against_differences():
    for shape, form in (((6, 30), "gate"), ((2, 9, 30), "silu")):
        s = make("f32", shape, form, seed=4)
        y, mean, rstd = m.ssd_groupnorm_fwd(up(s["x"]), 3, up(s["weight"]), up(s["bias"]), z=up(s["z"]),
                                            activation=s["activation"])
        g = m.ssd_groupnorm_bwd(up(s["x"]), 3, up(s["weight"]), up(s["bias"]), mean, rstd, up(s["dy"]),
                                z=up(s["z"]), activation=s["activation"])
        at = {n: d(s[n]) for n in ("x", "weight", "bias", "z") if s[n] is not None}

        def loss(v):
            o = lo.groupnorm(v["x"], 3, v["weight"], v["bias"], v.get("z"), s["activation"])[0]
            return (o * d(s["dy"])).sum().item()

        gen = torch.Generator().manual_seed(8)
        for n in at:
            way = torch.randn(at[n].shape, generator=gen, dtype=torch.float64)
            h = 1e-5
            diff = (loss(at | {n: at[n] + h * way}) - loss(at | {n: at[n] - h * way})) / (2 * h)
            terms = g["d" + n].double().cpu() * way
            # the difference is off by h^2 times a third derivative (1e-10 of a few hundred)
            assert abs(diff - terms.sum().item()) <= 64 * 2.0 ** -24 * terms.abs().sum().item() + 1e-6, n


def test_streams_and_graphs():
    for shape in ((300, 512), (3, 500, 64)):
        s = make("bf16", shape, "gate")
        x, z, dy, w, b = (up(s[n]) for n in ("x", "z", "dy", "weight", "bias"))

        def both():
            y, mean, rstd = m.ssd_groupnorm_fwd(x, 8, w, b, z=z)
            return [y, mean, rstd, *m.ssd_groupnorm_bwd(x, 8, w, b, mean, rstd, dy, z=z).values()]

        first = both()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            second = both()
        side.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(first, second))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = both()
        for i in range(3):
            x.copy_(up(s["x"]) * (i + 1))
            graph.replay()
            again = both()
            torch.cuda.synchronize()
            assert all(torch.equal(a, c) for a, c in zip(held, again))
