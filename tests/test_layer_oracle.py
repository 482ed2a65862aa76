"""Pins of the fp64 references of the operators around the scan (CPU): values
worked out by hand, equivalences between the forms, finite differences of the
gradients, and mistakes planted in the oracle that the comparisons catch."""
import math

import pytest
import torch

from oracle import layer_ops as lo


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + 31 * sum(shape))
    return scale * torch.randn(shape, generator=g, dtype=torch.float64)


def test_conv_by_hand():
    x = torch.tensor([[[1.0], [2.0], [4.0]]], dtype=torch.float64)
    w = torch.tensor([[0.5], [1.0]], dtype=torch.float64)
    b = torch.tensor([0.25], dtype=torch.float64)
    init = torch.tensor([[[8.0]]], dtype=torch.float64)
    y, f = lo.conv(x, w, b, init)
    for got, v in zip(y[0, :, 0].tolist(), [5.25, 2.75, 5.25]):
        assert got == pytest.approx(v / (1 + math.exp(-v)), rel=1e-14)
    assert f.tolist() == [[[4.0]]]


def test_selscan_by_hand():
    one = lambda *s: torch.ones(s, dtype=torch.float64)
    d = math.log1p(math.exp(0.5))
    y, f = lo.selscan(one(1, 2, 1) * 3, one(1, 2, 1) * 0.2, one(1) * 0.3, -one(1, 1) * 2,
                      one(1, 2, 1, 1) * 0.5, one(1, 2, 1, 1) * 4, one(1) * 0.1)
    h1 = d * 0.5 * 3
    h2 = math.exp(-2 * d) * h1 + h1
    assert y[0, :, 0].tolist() == pytest.approx([4 * h1 + 0.3, 4 * h2 + 0.3], rel=1e-14)
    assert f.item() == pytest.approx(h2, rel=1e-14)


def test_empty_sequences_keep_their_state():
    x = randn(1, 3, 2)
    init = randn(3, 2, 2)
    _, f = lo.conv(x, randn(3, 2), None, init, [0, 0, 3, 3])
    assert torch.equal(f[0], init[0]) and torch.equal(f[2], init[2])
    assert torch.equal(f[1], x[0, 1:])


def problem():
    return dict(x=randn(2, 5, 4), raw=randn(2, 5, 4, seed=1), dinit=randn(4, seed=2),
                A=-randn(3, 4, seed=3).exp(), B=randn(2, 5, 2, 3, seed=4),
                C=randn(2, 5, 2, 3, seed=5), D=randn(4, seed=6), z=randn(2, 5, 4, seed=7),
                init=randn(2, 3, 4, seed=8))


def conv_problem():
    return dict(x=randn(2, 5, 4), weight=randn(3, 4, seed=1), bias=randn(4, seed=2),
                init=randn(2, 2, 4, seed=3))


@pytest.mark.parametrize("fn,inputs", [(lo.selscan, problem()), (lo.conv, conv_problem())])
def test_gradients_are_the_differences(fn, inputs):
    seeds = [randn(*o.shape, seed=11) for o in fn(**inputs)]
    got = lo.gradients(fn, inputs, seeds)
    loss = lambda p: sum((o * s).sum() for o, s in zip(fn(**p), seeds)).item()
    for k, v in inputs.items():
        for at in range(0, v.numel(), max(1, v.numel() // 5)):
            step = torch.zeros_like(v).view(-1)
            step[at] = 1e-5
            step = step.view(v.shape)
            diff = (loss(inputs | {k: v + step}) - loss(inputs | {k: v - step})) / 2e-5
            # central differences: h^2 f''' / 6 and rounding 2^-53 |f| / h
            assert got[k].view(-1)[at].item() == pytest.approx(diff, rel=1e-6, abs=1e-7), (k, at)


def test_selscan_with_one_decay_is_the_ssd_recurrence():
    """A = -1 in every entry and equal steps: h decays as e^-d, as in ssd_fwd."""
    p = problem()
    p["A"] = -torch.ones_like(p["A"])
    p["B"], p["C"] = p["B"][:, :, :1], p["C"][:, :, :1]
    p["raw"] = p["raw"][..., :1].expand(-1, -1, 4).contiguous()
    p["dinit"] = torch.full((4,), 0.3, dtype=torch.float64)
    y, f = lo.selscan(**{**p, "D": None, "z": None})
    h = p["init"]  # [b, N, E]: one head of four columns
    for t in range(5):
        yt, h2 = lo.ssd_token(p["x"][:, t, None], p["raw"][:, t, :1], 0.3, p["B"][:, t],
                              p["C"][:, t], h[:, None])
        h = h2[:, 0]
        assert torch.allclose(yt[:, 0], y[:, t], rtol=1e-13, atol=1e-13)
    assert torch.allclose(h, f, rtol=1e-13, atol=1e-13)


def test_planted_mistakes_show():
    """A decay one token late, a state not reset, a tap order reversed: each
    changes the result by far more than any comparison's tolerance."""
    p = problem()
    y, _ = lo.selscan(**p)
    late = dict(p, raw=torch.roll(p["raw"], 1, 1))
    assert (lo.selscan(**late)[0] - y).abs().max() > 0.05
    x = p["x"].reshape(1, 10, 4)
    w = randn(3, 4, seed=1)
    assert (lo.conv(x, w, None, None, [0, 5, 10])[0] - lo.conv(x, w, None)[0]).abs().max() > 0.05
    assert (lo.conv(x, w.flip(0), None)[0] - lo.conv(x, w, None)[0]).abs().max() > 0.05


def test_norm_matches_the_formula():
    x, w, b = randn(3, 7), randn(7, seed=1), randn(7, seed=2)
    y, mean, rstd = lo.norm(x, w, b, 1e-5)
    for i in range(3):
        m = sum(x[i].tolist()) / 7
        v = sum((q - m) ** 2 for q in x[i].tolist()) / 7
        assert mean[i].item() == pytest.approx(m, abs=1e-15)
        assert rstd[i].item() == pytest.approx((v + 1e-5) ** -0.5, rel=1e-14)
        assert y[i, 3].item() == pytest.approx(
            (x[i, 3].item() - m) * (v + 1e-5) ** -0.5 * w[3].item() + b[3].item(), rel=1e-13)
