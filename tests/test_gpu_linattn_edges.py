"""Linear attention where a table, a bound or a buffer ends: powers of the decay below the
normal numbers of float32.

Tolerances.  |.| is the same expression of the inputs' absolute values.  A float32 result is off
by one 2^-24 |.| for each product and each addition in a row: at most K (a score, or the keys of
a state), 32 (the tokens of a chunk), L (the state), and 16 for weights and scales.
"""
import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from test_gpu_linattn import DEV, a, d, make, up
from oracle import linattn_ops as lo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def close(got, ref, size, steps, name):
    err = (got.double().cpu() - ref).abs()
    tol = steps * U * size + 1e-37
    assert (err <= tol).all(), (name, int((~(err <= tol)).sum()), (err / tol).max().item())


@pytest.mark.parametrize("L", [96, 140, 2500])
@pytest.mark.parametrize("reverse", [False, True])
def test_powers_below_the_normal_numbers(L, reverse):
    """exp(32 decay) of a chunk, and of the spans' 64 to 1250 tokens, between 2^-126 and 0: 1 over
    it is no float32.  The first rates are those of a chunk, the rest of a span (2500 tokens)."""
    decay = torch.tensor([-2.75, -2.8, -3.0, -3.2, -3.22, -1.37, -1.45, -1.5, -1.61, -0.7, -0.46, -0.3, -0.1])
    s = make("f32", 1, L, len(decay), len(decay), 16, 24, decay=decay)
    args = [up(s[n]) for n in ("q", "k", "v", "decay")]
    kw = dict(reverse=reverse, init_state=up(s["init"]))
    y, final = m.ssd_linattn_fwd(*args, **kw)
    g = m.ssd_linattn_bwd(*args, up(s["dy"]), d_final=up(s["d_final"]), **kw)
    fwd = lambda t: lo.linattn(t(s["q"]), t(s["k"]), t(s["v"]), d(s["decay"]), init=t(s["init"]), reverse=reverse)
    (ry, rf), (ay, af) = fwd(d), fwd(a)
    steps = 24 + 32 + L + 16
    close(y, ry, ay, steps, "y")
    close(final, rf, af, steps, "final_state")
    bwd = lambda t: lo.linattn_grads(t(s["q"]), t(s["k"]), t(s["v"]), d(s["decay"]), t(s["dy"]), t(s["d_final"]),
                                     init=t(s["init"]), reverse=reverse)
    ref, size = bwd(d), bwd(a)
    for n in ref:
        close(g[n], ref[n], size[n], steps, n)


@pytest.mark.parametrize("tokens", [64, 128, 320])
def test_span_powers_below_the_normal_numbers(tokens):
    """Spans of `tokens`: rates whose power over one lies between 2^-149 and 2^-126."""
    H, L = 8, 10 * tokens
    decay = -torch.linspace(87.5, 103.0, H) / tokens
    g = torch.Generator().manual_seed(tokens)
    q, k, v = (torch.randn((1, L, H, 8), generator=g) for _ in range(3))
    for n in (1, 2, 4, 8, 16):  # sequences of a batch: fewer spans each
        x = [t.expand(n, -1, -1, -1).contiguous().to(DEV) for t in (q, k, v)]
        y, final = m.ssd_linattn_fwd(*x, decay.to(DEV))
        assert y.isfinite().all() and final.isfinite().all()
        if n == 1:
            (ry, rf), (ay, af) = (lo.linattn(*(f(t) for t in (q, k, v)), d(decay)) for f in (d, a))
        steps = 8 + 32 + L + 16
        close(y[-1:], ry, ay, steps, "y")
        close(final[-1:], rf, af, steps, "final_state")


BAD_CU = [[0, 4096, 0, 4096], [4096, 0, 4096, 0], [4000, 10, 4096, 4096], [-5, 5000, -9, 4096],
          [0, 2000, 1000, 4096], [1 << 30, -(1 << 30), 1 << 30, 0]]


@pytest.mark.parametrize("cu", BAD_CU)
def test_bounds_out_of_order_stay_in_the_buffers(cu):
    """Results are unspecified, but nothing behind a buffer is touched."""
    T, H, K, V = 4096, 2, 16, 24
    g = torch.Generator().manual_seed(1)
    q, k, v, dy = (torch.randn((1, T, H, n), generator=g).to(DEV) for n in (K, K, V, V))
    dec = torch.tensor([-0.1, -0.01], device=DEV)
    bounds = torch.tensor(cu, dtype=torch.int32, device=DEV)
    ly = m._layer
    dims = m.SsdLinattnDims(1, T, H, H, K, V, 3, 0, 1.0, 0)
    for name in ("fwd", "bwd"):
        need = ly._entry(f"ssd_linattn_{name}_workspace_bytes")(dims)
        buf = torch.full((2 * need + (8 << 20),), 7, dtype=torch.uint8, device=DEV)
        ws = dict(cu_seqlens=bounds, workspace=buf[:need])
        if name == "fwd":
            wide = torch.full((3, T, H, V), 5.0, device=DEV)
            states = torch.full((5, H, K, V), 5.0, device=DEV)
            m.ssd_linattn_fwd(q, k, v, dec, y=wide[1:2], final_state=states[1:4], **ws)
            assert (wide[[0, 2]] == 5).all() and (states[[0, 4]] == 5).all()
        else:
            m.ssd_linattn_bwd(q, k, v, dec, dy, **ws)
        assert (buf[need:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G", [(2, 2), (4, 2), (3, 1)])
@pytest.mark.parametrize("cu", [[0, 0, 70, 100], [20, 30, 100, 100], [0, 0, 0, 0], [0, 900, 905, 950]])
def test_tokens_outside_the_sequences_stay(dtype, H, G, cu):
    """The gradients' rows before the first and behind the last sequence, heads shared or not."""
    L, K, V = (130, 16, 24) if cu[-1] < 900 else (1000, 16, 24)
    s = make(dtype, 1, L, H, G, K, V, cu=cu)
    q, k, v, dec, dy, init, df = (up(s[n]) for n in ("q", "k", "v", "decay", "dy", "init", "d_final"))
    bounds = torch.tensor(cu, dtype=torch.int32, device=DEV)
    ly = m._layer
    dims, lay, c, _, state = ly._linattn_arguments(q, k, v, dec, 0.5, bounds, None, dy)
    need = ly._entry("ssd_linattn_bwd_workspace_bytes")(dims)
    ws = torch.full((need // 4 + 1,), float("nan"), device=DEV)
    g = {n: torch.full_like(t, 5.0) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    ly._launch("ssd_linattn_bwd", q, dims, lay, *(t.data_ptr() for t in (q, k, v, dec, init, c)), 0,
               dy.data_ptr(), df.data_ptr(), *(t.data_ptr() for t in g.values()),
               torch.empty(state, device=DEV).data_ptr(), ws.data_ptr(), need)
    want = m.ssd_linattn_bwd(q, k, v, dec, dy, scale=0.5, init_state=init, cu_seqlens=bounds, d_final=df)
    for n in g:
        assert (g[n][0, :cu[0]] == 5).all() and (g[n][0, cu[-1]:] == 5).all(), n
        inside = g[n][0, cu[0]:cu[-1]]
        assert inside.isfinite().all() and torch.equal(inside, want[n][0, cu[0]:cu[-1]]), n
