"""Linear attention at head sizes that are 4, 2 or 1 past a multiple of 8, where a lane's run of
neighbours ends inside the row: every output, entry by entry against the fp64 recurrence, into
buffers and from workspaces that hold NaN, so that an entry nobody writes fails.

Tolerances are test_gpu_linattn's (`near`).
"""
import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from mamba_ssd_chunked_02_amd import _layer as ly
from oracle import linattn_ops as lo
from test_gpu_linattn import DEV, TYPES, a, check_fwd, cu_of, d, make, near, up

pytestmark = pytest.mark.gpu
NAN = float("nan")


def spoilt(name, dims):
    """A workspace of the size that the library names, full of NaN."""
    need = ly._entry(name)(dims)
    return torch.full((need // 4,), NAN, device=DEV) if need else None


def bwd_into_nan(s, cu=None, reverse=False, scale=0.37, in_place=False):
    """ssd_linattn_bwd through the C ABI; outputs and workspace hold NaN before it.  in_place:
    dinit_state is d_final's buffer."""
    q, k, v, dec, dy, init, df = (up(s[n]) for n in ("q", "k", "v", "decay", "dy", "init", "d_final"))
    dims, lay, c, _, state = ly._linattn_arguments(q, k, v, dec, scale, cu_of(cu), None, dy)
    g = {"dq": torch.full_like(q, NAN), "dk": torch.full_like(k, NAN), "dv": torch.full_like(v, NAN),
         "dinit_state": df if in_place else torch.full(state, NAN, device=DEV)}
    ws = spoilt("ssd_linattn_bwd_workspace_bytes", dims)
    at = ly._at
    ly._launch("ssd_linattn_bwd", q, dims, lay, at(q), at(k), at(v), at(dec), at(init), at(c), int(reverse),
               at(dy), at(df), *(at(g[n]) for n in ("dq", "dk", "dv", "dinit_state")), at(ws),
               0 if ws is None else ws.nbytes)
    return g


def oracle_bwd(s, cu=None, reverse=False, scale=0.37):
    kw = dict(scale=scale, cu=cu, reverse=reverse)
    f = lambda t: lo.linattn_grads(t(s["q"]), t(s["k"]), t(s["v"]), d(s["decay"]), t(s["dy"]), t(s["d_final"]),
                                   init=t(s["init"]), **kw)
    return f(d), f(a)


def check_all(s, cu=None, reverse=False, in_place=False):
    q, k, v, dec = (up(s[n]) for n in ("q", "k", "v", "decay"))
    b, L, H, K = q.shape
    G, V = v.shape[2:]
    code = {torch.float32: 0, torch.bfloat16: 1}[q.dtype]
    dims = m.SsdLinattnDims(b, L, H, G, K, V, 0 if cu is None else len(cu) - 1, code, 0.37, 0)
    y = torch.full((b, L, H, V), NAN, dtype=q.dtype, device=DEV)
    ws = spoilt("ssd_linattn_fwd_workspace_bytes", dims)
    _, final = m.ssd_linattn_fwd(q, k, v, dec, scale=0.37, init_state=up(s["init"]), cu_seqlens=cu_of(cu),
                                 reverse=reverse, y=y, workspace=ws)
    kw = dict(scale=0.37, cu=cu, reverse=reverse)
    ry, rf = lo.linattn(d(s["q"]), d(s["k"]), d(s["v"]), d(s["decay"]), init=d(s["init"]), **kw)
    ay, af = lo.linattn(a(s["q"]), a(s["k"]), a(s["v"]), d(s["decay"]), init=a(s["init"]), **kw)
    near(y, ry, ay, L, "y")
    near(final, rf, af, L, "final_state")
    got = bwd_into_nan(s, cu, reverse, in_place=in_place)
    ref, size = oracle_bwd(s, cu, reverse)
    for n in ref:
        near(got[n], ref[n], size[n], L, n)


WIDTHS = [(64, 68), (68, 64), (24, 76), (76, 24), (100, 100), (128, 132), (132, 128), (4, 92), (66, 70),
          (65, 129), (36, 12), (252, 244)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,G", [(2, 2), (4, 2)])
@pytest.mark.parametrize("K,V", WIDTHS)
def test_every_column_is_written(dtype, H, G, K, V):
    check_all(make(dtype, 2, 70, H, G, K, V), reverse=H == 4)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,G", [(2, 2), (4, 2)])
@pytest.mark.parametrize("K,V", [(100, 68), (68, 132)])
def test_every_column_is_written_in_spans(dtype, H, G, K, V):
    cu = [0, 0, 450, 451, 900]
    check_all(make(dtype, 1, 900, H, G, K, V, cu=cu), cu)


@pytest.mark.parametrize("K", range(60, 78))
def test_every_width_around_a_tile(K):
    """Keys from 60 to 77 wide, values from 76 to 59, and y's neighbours stay."""
    s = make("f32", 1, 40, 1, 1, K, 136 - K)
    check_all(s)
    wide = torch.full((1, 40, 1, 138 - K), 3.0, device=DEV)
    m.ssd_linattn_fwd(up(s["q"]), up(s["k"]), up(s["v"]), up(s["decay"]), y=wide[..., 1:-1])
    assert (wide[..., 0] == 3).all() and (wide[..., -1] == 3).all() and not (wide[..., 1:-1] == 3).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b,L,H,G,K,V", [(40, 70, 16, 16, 24, 28), (1, 900, 4, 2, 24, 100)])
def test_gradient_of_the_state_in_place_is_right(dtype, b, L, H, G, K, V):
    """dinit_state over d_final: against the oracle, not another call."""
    check_all(make(dtype, b, L, H, G, K, V), in_place=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_views_of_odd_widths(dtype):
    s = make(dtype, 2, 50, 3, 3, 68, 84)

    def odd(t):
        b, L, H, D = t.shape
        wide = torch.full((b, L, H * (D + 3) + 1), 7.0, dtype=t.dtype, device=DEV)
        view = wide[..., 1:].unflatten(-1, (H, D + 3))[..., :D]
        view.copy_(t)
        return view

    check_fwd(s, view=odd)
