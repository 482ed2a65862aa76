"""Linear attention on bfloat16 inputs keeps what a float32 evaluation keeps, up to the rounding of
its outputs.

Tolerance.  |.| is the same expression of the inputs' absolute values.  A score, and a state entry
that a query meets, is the sum of two bfloat16 values: the first leaves at most half a step,
2^-8 of it, and the second half a step of that: 2^-16 |.|.  float32 sums: one 2^-24 |.| for each
product and each addition in a row, at most K + V (scores, or the state's keys), 32 (the tokens of a
chunk), L (the state), 4 (shared heads) and 16 (weights, scales, the three parts of what is added).
Then the output is rounded once, by half a step of its value.
"""
import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from oracle import linattn_ops as lo
from test_gpu_linattn import a, cu_of, d, make, up

pytestmark = pytest.mark.gpu


def once_rounded(got, ref, size, steps, name):
    assert got.shape == ref.shape, name
    err = (got.double().cpu() - ref).abs()
    tol = (2.0 ** -16 + steps * 2.0 ** -24) * size + 1e-37
    tol = tol + (2.0 ** -8 * (ref.abs() + tol) if got.dtype == torch.bfloat16 else 0.0)
    assert (err <= tol).all(), (name, int((~(err <= tol)).sum()), (err / tol).max().item())


def check(b, L, H, G, K, V, cu=None, reverse=False, decay=None):
    s = make("bf16", b, L, H, G, K, V, cu=cu, decay=decay)
    kw = dict(scale=0.37, reverse=reverse)
    args = [up(s[n]) for n in ("q", "k", "v", "decay")]
    own = dict(init_state=up(s["init"]), cu_seqlens=cu_of(cu), **kw)
    y, final = m.ssd_linattn_fwd(*args, **own)
    got = {"y": y, "final": final} | m.ssd_linattn_bwd(*args, up(s["dy"]), d_final=up(s["d_final"]), **own)

    def oracle(f):
        y, final = lo.linattn(f(s["q"]), f(s["k"]), f(s["v"]), d(s["decay"]), init=f(s["init"]), cu=cu, **kw)
        return {"y": y, "final": final} | lo.linattn_grads(
            f(s["q"]), f(s["k"]), f(s["v"]), d(s["decay"]), f(s["dy"]), f(s["d_final"]), init=f(s["init"]), cu=cu,
            **kw)

    ref, size = oracle(d), oracle(a)
    for n in ref:
        once_rounded(got[n], ref[n], size[n], K + V + 32 + L + 4 + 16, n)


@pytest.mark.parametrize("K,V", [(16, 16), (40, 56), (64, 64), (64, 128), (77, 33), (128, 64), (128, 128),
                                 (130, 200), (256, 64), (256, 256)])
@pytest.mark.parametrize("reverse", [False, True])
def test_head_sizes(K, V, reverse):
    check(2, 150, 2, 2, K, V, reverse=reverse)


@pytest.mark.parametrize("H,G", [(4, 2), (3, 1)])
@pytest.mark.parametrize("L,cu", [(70, None), (400, [0, 0, 5, 70, 134, 135, 400])])
def test_shared_heads(H, G, L, cu):
    check(1, L, H, G, 24, 40, cu=cu)


@pytest.mark.parametrize("K,V", [(32, 24), (128, 72)])
def test_spans(K, V):
    check(1, 1300, 2, 1, K, V)


def test_state_alone():
    """One token that meets a state: y = q S + (q . k) v."""
    check(3, 1, 4, 4, 128, 128, decay=torch.tensor([0.0, -0.01, -1.0, -5.0]))


@pytest.mark.parametrize("K,V,L", [(64, 128, 300), (128, 128, 1000), (256, 100, 200)])
def test_float32_over_many_entries(K, V, L):
    """The root of the mean square, where roundings of either sign average out: a score, a state and
    an output are each sums of at most 2^8 terms in a row, whose roundings of at most 2^-24 add up
    like sqrt(2^8): 16 2^-24 for each of the three, of the terms' sizes."""
    s = make("f32", 1, L, 2, 2, K, V)
    args = [up(s[n]) for n in ("q", "k", "v", "decay")]
    y, _ = m.ssd_linattn_fwd(*args, init_state=up(s["init"]))
    f = lambda t: lo.linattn(t(s["q"]), t(s["k"]), t(s["v"]), d(s["decay"]), init=t(s["init"]))[0]
    ref, size = f(d), f(a)
    assert (y.double().cpu() - ref).square().mean().sqrt() <= 48 * 2.0 ** -24 * size.square().mean().sqrt()
