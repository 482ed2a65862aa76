"""The operators around the scan on the GPU at the sizes that take each kernel variant over
several segments, tiles or runs, entry by entry within the bounds of their roundings:
oracle/layer_bounds.py for the selective scan; for the convolution, in units u = 2^-24,
V = |bias| + sum |w x| and v within 6 u V of it:

  silu(v)   16 u (1 + V): the error of v, the hardware's exp2 and reciprocal
  silu'(v)  16 u (1 + V), the slope of silu' being at most 1/2
  sums      one u of the sum of sizes for each addition on the longest path

A bf16 output is rounded once more, by half a step of its value.
"""
import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from oracle import layer_bounds as lb
from oracle import layer_ops as lo
from test_gpu_layer import TYPES, Source, dd, scan_call, scan_problem, up

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def close(got, value, bound, name):
    assert got.shape == value.shape, (name, got.shape, value.shape)
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    tol = bound + half * (value.abs() + bound) + 1e-30
    err = (got.double().cpu() - value).abs()
    assert (err <= tol).all(), (name, (err / tol).max().item(), int((err > tol).sum()))


# ---- selective scan ------------------------------------------------------------------------

SCAN = [  # b, L, E, N, G, cu
    (2, 77, 203, 16, 1, None), (1, 300, 33, 8, 1, None), (2, 70, 34, 32, 2, None),
    (1, 90, 10, 33, 1, None), (1, 40, 18, 64, 1, None), (1, 2600, 20, 16, 1, None),
    (2, 1500, 9, 8, 1, None), (1, 900, 34, 32, 2, None),
    (1, 300, 24, 16, 1, [0, 0, 2, 19, 275, 300, 300]),
    (1, 2300, 18, 16, 1, [0, 0, 700, 701, 2300, 2300])]
WIDE = [  # workgroups of half, a quarter and an eighth of the waves, over several segments
    (1, 300, 8320, 16, 1, None), (1, 300, 16480, 16, 1, None), (1, 300, 16480, 8, 1, None),
    (1, 70, 16480, 32, 1, None), (1, 40, 16480, 64, 1, None),
    (1, 700, 8320, 16, 1, [0, 3, 300, 300, 700])]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("case", SCAN + WIDE, ids=str)
def test_selscan_within_its_roundings(dtype, gated, case):
    b, L, E, N, G, cu = case
    p, (dy, df), _ = scan_problem(dtype, case, gated, True, seed=3)
    args, kw = scan_call(p, cu)
    y, f = m.ssd_selscan_fwd(*args, **kw)
    got = {"y": y, "final": f, **m.ssd_selscan_bwd(*args, up(dy), **kw, d_final=up(df))}
    # channels do not meet but in dB and dC: of many a few are checked
    e = slice(0, E) if case in SCAN else torch.tensor([0, 15, 16, 1000, E // 2, E - 17, E - 1])
    T, S = b * L, b if cu is None else len(cu) - 1
    flat = lambda t: None if t is None else dd(t).flatten(0, 1)
    cut = lambda t: None if t is None else t[..., e]
    spans = [(i * L, (i + 1) * L) for i in range(b)] if cu is None else list(zip(cu[:-1], cu[1:]))
    res = lb.selscan(cut(flat(p["x"])), cut(flat(p["raw"])), dd(cut(p["dinit"])), dd(cut(p["A"])),
                     flat(p["B"]), flat(p["C"]), dd(cut(p["D"])), cut(flat(p["z"])),
                     dd(cut(p["init"])), cut(flat(dy)), dd(cut(df)), spans,
                     (8 + E // G // 16, 104 + (T // 64 + S) // 16))
    for k, (value, bound) in res.items():
        g = got[k]
        if k in ("y", "dx", "dd_raw", "dz", "dB", "dC"):
            g = g.flatten(0, 1)
        if k in ("dB", "dC"):
            if case in WIDE:
                continue
        else:
            g = cut(g)
        if k == "dD" and not gated:
            continue  # there is no D
        close(g, value, bound, k)


# ---- convolution ---------------------------------------------------------------------------

def bounds_of(L, tile, seed):
    """Sequences that end inside a tile, just before and just behind its end and on it,
    short and empty ones, and long ones between them."""
    g = torch.Generator().manual_seed(seed)
    at, cu = 0, [0]
    lengths = [1, 2, 3, 0, 5, tile, tile - 1, 1, 2 * tile, tile - 3, 0, 3 * tile + 2]
    while at < L:
        n = lengths[(len(cu) - 1) % len(lengths)] if len(cu) % 3 else int(torch.randint(1, 9 * tile, (), generator=g))
        at = min(L, at + n)
        cu.append(at)
    return cu + [L]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,E,W,kind", [
    (9001, 520, 4, "packed"), (25003, 520, 4, "packed"), (25003, 520, 2, "packed"), (26000, 525, 3, "packed"),
    (4200, 2050, 4, "one"), (25003, 520, 3, "batch"),
    # several tiles a wave in the gradients
    (65536, 1030, 4, "long"), (65600, 1794, 4, "packed"), (66001, 1028, 4, "one")])
def test_conv_large_tiles(dtype, L, E, W, kind):
    """Forward runs of 16 tokens and gradient runs of 16 by 4 channels, several to a wave,
    with states, sequence ends anywhere in a run, and one or many sequences."""
    s = Source(L + E + W, dtype)
    b = 3 if kind == "batch" else 1
    L //= b
    cu = {"packed": bounds_of(L, 16, L), "long": [0, L // 3 + 5, L - 7, L]}.get(kind)
    S = b if cu is None else len(cu) - 1
    x, dy, init, df = s(b, L, E), s(b, L, E), s(S, W - 1, E), s(S, W - 1, E)
    w, bias = s.f32(W, E, scale=0.5), s.f32(E)
    cug = up(None if cu is None else torch.tensor(cu, dtype=torch.int32))
    y, f = m.ssd_conv_fwd(up(x), up(w), up(bias), init_state=up(init), cu_seqlens=cug)
    g = m.ssd_conv_bwd(up(x), up(w), up(bias), up(dy), init_state=up(init), cu_seqlens=cug, d_final=up(df))
    e = torch.tensor([0, 1, 3, 4, 255, 256, E // 2 + 1, E - 3, E - 1])
    X, DY, I, DF, w, bias = (dd(t[..., e]) for t in (x, dy, init, df, w, bias))
    got = {"y": y, "f": f, **g}
    got = {k: t[..., e.to(t.device)] for k, t in got.items()}
    Y, bY, DX, bDX = (torch.zeros_like(X) for _ in range(4))
    F, DI, bDI = (torch.zeros_like(I) for _ in range(3))
    DW, sW = torch.zeros_like(w), torch.zeros_like(w)
    DB, sB = torch.zeros_like(bias), torch.zeros_like(bias)
    for q, (i, u, v) in enumerate(lo.spans(X, cu)):
        n = v - u
        line = torch.cat([I[q], X[i, u:v]])
        F[q] = line[n:]
        a = bias + sum(line[k:k + n] * w[k] for k in range(W))
        size = 1 + bias.abs() + sum((line[k:k + n] * w[k]).abs() for k in range(W))
        sg = torch.sigmoid(a)
        Y[i, u:v], bY[i, u:v] = a * sg, 16 * U * size
        dv = DY[i, u:v] * sg * (1 + a * (1 - sg))
        sv = DY[i, u:v].abs() * size  # of dv's error: 18 u of it, its product counted
        dl, bl = torch.zeros_like(line), torch.zeros_like(line)
        for k in range(W):
            dl[k:k + n] += dv * w[k]
            bl[k:k + n] += (18 + W + 2) * U * sv * w[k].abs()
            DW[k] += (dv * line[k:k + n]).sum(0)
            sW[k] += (sv * line[k:k + n].abs()).sum(0)
        dl[n:] += DF[q]
        bl[n:] += 2 * U * DF[q].abs()
        DI[q], bDI[q] = dl[:W - 1], bl[:W - 1]
        DX[i, u:v], bDX[i, u:v] = dl[W - 1:], bl[W - 1:]
        DB += dv.sum(0)
        sB += sv.sum(0)
    # a thread's sum runs over at most 8 tiles of 16 tokens, four waves are joined, and the
    # column sum adds every sixteenth of at most T / 64 + 1 rows and then sixteen
    depth = 18 + 128 + 4 + (b * L // 64 + 1) // 16 + 18
    close(got["y"], Y, bY, "y")
    assert torch.equal(got["f"].double().cpu(), F)
    close(got["dx"], DX, bDX, "dx")
    close(got["dinit_state"], DI, bDI, "dinit_state")
    close(got["dweight"], DW, depth * U * sW, "dweight")
    close(got["dbias"], DB, depth * U * sB, "dbias")
