"""Values of the operators around the scan where they are easily lost: rates that are
NaN or -inf.  Tolerances as test_gpu_layer's."""
import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from oracle import layer_ops as lo
from test_gpu_layer import DEV, TYPES, Source, dd, scan_call, scan_problem, up, within

pytestmark = pytest.mark.gpu

GRADS = {"x": "dx", "raw": "dd_raw", "dinit": "dd_init", "A": "dA", "B": "dB", "C": "dC",
         "D": "dD", "z": "dz", "init": "dinit_state"}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", [(2, 77, 20, 16, 1, None), (1, 2600, 20, 16, 1, None),
                                  (1, 90, 40, 40, 2, [0, 40, 41, 90])], ids=str)
def test_selscan_nan_rate_gives_nan(dtype, case):
    """A rate that has become NaN shows: everything that the definition forms of it is
    NaN, and nothing else is."""
    b, L, E, N, G, cu = case
    p, (dy, df), _ = scan_problem(dtype, case)
    n, e = 3, 7
    p["A"][n, e] = float("nan")
    args, kw = scan_call(p, cu)
    y, f = m.ssd_selscan_fwd(*args, **kw)
    g = m.ssd_selscan_bwd(*args, up(dy), **kw, d_final=up(df))
    ins = {k: dd(v) for k, v in p.items()}
    fn = lambda **k: lo.selscan(**k, cu=cu)
    ry, rf = fn(**ins)
    rg = lo.gradients(fn, ins, [dd(dy), dd(df)])
    assert ry[..., e].isnan().all() and not ry[..., e + 1:].isnan().any()
    for got, ref, name in [(y, ry, "y"), (f, rf, "final")] + [(g[GRADS[k]], r, k) for k, r in rg.items()]:
        assert torch.equal(got.isnan().cpu(), ref.isnan()), name
    assert torch.equal(g["dA"].isnan().nonzero().cpu(), torch.tensor([[n, e]]))
    pool = kw["init_state"][:1].repeat(b, 1, 1)
    at = lambda t: t[:, 0]
    yt = m.ssd_selscan_step(*map(at, args[:2]), args[2], args[3], *map(at, args[4:]), pool, D=kw["D"],
                            z=at(kw["z"]))
    for t in (yt, pool):
        want = torch.zeros(t.shape, dtype=torch.bool)
        want[(slice(None), e) if t is yt else (slice(None), n, e)] = True
        assert torch.equal(t.isnan().cpu(), want)


@pytest.mark.parametrize("dtype", TYPES)
def test_selscan_rates_of_minus_infinity_backward(dtype):
    """Entries that forget at once: gradients finite, and those of a rate so large that
    its decay is 0."""
    case = (1, 75, 20, 16, 1, [0, 40, 41, 75])
    p, (dy, df), cu = scan_problem(dtype, case)
    p["A"][1] = -float("inf")
    p["A"][4, 3:9] = -float("inf")
    args, kw = scan_call(p, cu)
    g = m.ssd_selscan_bwd(*args, up(dy), **kw, d_final=up(df))
    ins = {k: dd(v) for k, v in p.items()}
    ins["A"] = ins["A"].clamp(min=-1e30)
    rg = lo.gradients(lambda **k: lo.selscan(**k, cu=cu), ins, [dd(dy), dd(df)])
    for k, ref in rg.items():
        within(g[GRADS[k]], ref, 4 * (64 + 4 * 75) + (4 * 20 if k in "BC" else 0), k)


def steps_and_values():
    """Raw steps over the range that layers use and its ends, and softplus of them."""
    z = torch.cat([torch.linspace(-4.2, -2, 3200), torch.linspace(-30, 30, 896)]).float()
    return z, torch.log1p(torch.exp(-z.double().abs())) + z.double().clamp(min=0)


def steps_right(got, z, exact):
    """d = max(z, 0) + log(1 + v) with v = e^-|z|.  In units of 2^-24: |z| for the rounded
    exponent and 0.25 |z| for its rounded factor log2(e), 2 each for the hardware's exp2
    and reciprocal, and 4 more roundings."""
    err = (got.double().cpu().flatten() / exact - 1).abs()
    units = 8 + 1.25 * z.double().abs()
    assert (err <= units * 2.0 ** -24).all(), (err / units * 2 ** 24).max().item()


@pytest.mark.parametrize("form", ["scan", "gradient", "token", "ssd_token"])
def test_step_sizes_keep_their_low_bits(form):
    """With rates of 0 and ones for the rest one token's output is the step itself."""
    z, exact = steps_and_values()
    E = len(z)
    one = lambda *s: torch.ones(s, device=DEV)
    A, dinit = torch.zeros(1, E, device=DEV), torch.zeros(E, device=DEV)
    if form == "ssd_token":
        B = torch.zeros(64, 1, 16, device=DEV)
        B[..., 0] = 1
        y = m.ssd_step(one(64, E // 64, 16), up(z.view(64, -1)), 0.0, B, B,
                       torch.zeros(64, E // 64, 16, 16, device=DEV))
        assert (y == y[..., :1]).all()
        got = y[..., 0]
    elif form == "token":
        got = m.ssd_selscan_step(one(1, E), up(z[None]), dinit, A, one(1, 1, 1), one(1, 1, 1),
                                 torch.zeros(1, 1, E, device=DEV))
    else:
        args = (one(1, 1, E), up(z[None, None]), dinit, A, one(1, 1, 1, 1), one(1, 1, 1, 1))
        got = m.ssd_selscan_fwd(*args)[0] if form == "scan" else m.ssd_selscan_bwd(
            *args, one(1, 1, E))["dx"]
    steps_right(got, z, exact)
