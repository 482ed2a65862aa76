"""Group norm's statistics where single positions or whole runs lie far from the rest.

Tolerances, in u = 2^-24 of the variance.  Blocks of 8 positions: their squares are of distances
from one of them, at most 8 times their deviations, with at most 8 roundings: 64.  Blocks, threads,
runs and channels are joined one after the other, each addition one rounding of what is there:
`adds`, counted at each case.  The mean's own error, of a few u of the first block's, enters by its square.
rstd has half the variance's relative error, and 4 u of its own.  y = (x - mean) rstd takes both, the
mean's error being at most (adds + 64) u of the deviation.
"""
import pytest
import torch

import mamba_ssd_chunked_02_amd as m

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def check(x, G, adds, samples=1, name=""):
    """x [P, C], the same for every sample: a view.  The reference is formed on the CPU."""
    P, C = x.shape
    wide = x.to(DEV)[None].expand(samples, -1, -1)
    y, mean, rstd = m.ssd_groupnorm_fwd(wide, G, eps=0.0)
    assert torch.equal(mean, mean[:1].expand_as(mean)) and torch.equal(rstd, rstd[:1].expand_as(rstd))
    y, mean, rstd = y[[0, -1]].cpu(), mean.cpu(), rstd.cpu()
    xd = x.double().view(P, G, C // G)
    rm = xd.mean((0, 2))
    c = xd - rm[:, None]
    rv = c.square().mean((0, 2))
    K = adds + 64
    off = (1 / (rstd[0].double() ** 2 * rv) - 1).abs().max().item()
    assert off <= (K + 8) * U, (name, "variance", off / U, K + 8)
    off = ((mean[0].double() - rm).abs() / rv.sqrt()).max().item()
    assert off <= K * U, (name, "mean", off / U, K)
    ref = (c / rv.sqrt()[:, None]).view(P, C)
    half = torch.finfo(y.dtype).eps / 2
    tol = half * ref.abs() + 2 * K * U * (1 + ref.abs())
    assert ((y.double() - ref).abs() <= tol).all(), name


def normal(P, C, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + P + C)
    return torch.randn((P, C), generator=g).to(TYPES[dtype])


# samples, positions, channels, groups, and the additions in a row: blocks of 8 rows of a
# thread, threads of a column, channels a lane, lanes, runs a lane
CASES = [(512, 16384, 64, 4, 128 + 16 + 1 + 6 + 1),  # 1024 rows a thread (f32), one run
         (512, 4096, 320, 32, 171 + 3 + 3 + 3 + 1),
         (512, 3001, 8, 2, 3 + 128 + 1 + 6 + 1),
         (1, 16384, 320, 1, 2 + 6 + 5 + 6 + 16)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("first", [30.0, 1000.0])
def test_first_position_far_from_the_rest(dtype, case, first):
    samples, P, C, G, adds = case
    x = normal(P, C, dtype)
    x[0] = first
    check(x, G, adds, samples)


@pytest.mark.parametrize("where", [0, 1, 7, 8, 100, 4095])
def test_any_position_far_from_the_rest(where):
    x = normal(4096, 64, "f32", 3)
    x[where] = 1e4
    check(x, 2, 32 + 16 + 1 + 6 + 1, 512)


def test_first_run_far_from_the_rest():
    """512 runs of 64 positions, the first 64 at 1000: 8 runs a lane."""
    x = normal(32768, 320, "f32")
    x[:64] += 1000.0
    check(x, 1, 2 + 6 + 5 + 6 + 8 + 6)


def test_channels_far_from_each_other():
    x = normal(5000, 64, "f32") + torch.tensor([0.0, 50.0]).repeat(32)
    check(x, 4, 128 + 16 + 1 + 6 + 8)


@pytest.mark.parametrize("size", [1e16, 1e-15])
def test_sizes_near_the_ends(size):
    """48000 squares of 1e16 add up to 5e36, which float32 holds (its sums end at 3.4e38); a mean
    of 1e20 has no squares."""
    x = normal(3000, 32, "f32")
    check(x * size, 2, 128)
    if size > 1:
        y, mean, rstd = m.ssd_groupnorm_fwd(torch.full((2, 300, 32), 1e20, device=DEV), 2)
        assert (mean == 1e20).all() and not y.any()
