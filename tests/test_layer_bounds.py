"""oracle/layer_bounds.py (CPU): its values against autograd over the recurrence, its bounds
against a plain float32 evaluation, and mistakes far smaller than the largest entry, which
the bounds must show."""
import pytest
import torch

from oracle import layer_bounds as lb
from oracle import layer_ops as lo

CASES = [(1, 37, 12, 5, 1, None, True), (1, 60, 12, 16, 2, [0, 1, 1, 20, 60], True),
         (1, 200, 6, 16, 1, None, False)]


def problem(case, seed=0, dtype=torch.float32):
    b, L, E, N, G, cu, gated = case
    S = len(cu) - 1 if cu else 1
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, shift=0.0: (shift + torch.randn(s, generator=g)).to(dtype).double()
    p = {"x": r(1, L, E), "raw": r(1, L, E), "dinit": r(E, shift=-2.0), "A": -r(N, E).exp(),
         "B": r(1, L, G, N), "C": r(1, L, G, N), "D": r(E) if gated else None,
         "z": r(1, L, E) if gated else None, "init": r(S, N, E)}
    return p, (r(1, L, E), r(S, N, E)), cu or [0, L]


def bounds(p, seeds, cu, sums=(40, 200)):
    first = lambda t: None if t is None else t[0]
    return lb.selscan(*(first(p[k]) for k in ("x", "raw")), p["dinit"], p["A"], first(p["B"]),
                      first(p["C"]), p["D"], first(p["z"]), p["init"], first(seeds[0]), seeds[1],
                      list(zip(cu[:-1], cu[1:])), sums)


NAMES = {"x": "dx", "raw": "dd_raw", "dinit": "dd_init", "A": "dA", "B": "dB", "C": "dC",
         "D": "dD", "z": "dz", "init": "dinit_state"}


def evaluate(p, seeds, cu, dtype):
    cast = {k: None if v is None else v.to(dtype) for k, v in p.items()}
    fn = lambda **k: lo.selscan(**k, cu=cu)
    y, f = fn(**cast)
    g = lo.gradients(fn, cast, [s.to(dtype) for s in seeds])
    got = {"y": y[0], "final": f}
    for k, v in g.items():
        got[NAMES[k]] = v[0] if k in ("x", "raw", "z", "B", "C") else v
    return got


@pytest.mark.parametrize("case", CASES, ids=str)
def test_values_and_bounds(case):
    p, seeds, cu = problem(case)
    res = bounds(p, seeds, cu)
    exact, single = (evaluate(p, seeds, cu, t) for t in (torch.float64, torch.float32))
    for k, (value, bound) in res.items():
        if k not in exact:
            continue
        assert (value - exact[k]).abs().max() <= 1e-11 * value.abs().max().clamp(min=1), k
        assert ((single[k].double() - value).abs() <= bound + 1e-30).all(), k
        # tight enough to show much; dd_init sums every token's signed terms
        assert bound.median() <= (4e-3 if k == "dd_init" else 1e-4) * value.abs().max(), k


def test_bounds_show_small_mistakes():
    """A term of a thousandth left out of y, dx and dz; decays off by a ten-thousandth."""
    p, seeds, cu = problem(CASES[2])
    p["D"], p["z"] = torch.full((6,), 1e-3, dtype=torch.float64), torch.randn(1, 200, 6).double()
    res = bounds(p, seeds, cu)
    wrong = evaluate(p | {"D": torch.zeros(6).double()}, seeds, cu, torch.float64)
    for k in ("y", "dx", "dz"):
        value, bound = res[k]
        assert ((wrong[k] - value).abs() > bound).double().mean() > 0.5, k
    wrong = evaluate(p | {"A": p["A"] * (1 + 1e-4)}, seeds, cu, torch.float64)
    for k in ("final", "dA", "dinit_state"):
        value, bound = res[k]
        assert ((wrong[k] - value).abs() > bound).any(), k
