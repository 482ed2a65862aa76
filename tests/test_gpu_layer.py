"""The operators around the scan on the GPU against the fp64 references of
oracle/layer_ops.py.

Tolerances.  An output of type t is the float32 result rounded once: off by at
most eps(t) / 2 relative to the value.  The float32 result is off by at most
K 2^-24 of the size of what is summed, with K the number of roundings on the
way: a few for each factor, plus one per term of a sum.  For sums that run
over L tokens K = 16 + 4 L; sizes are taken as the largest entry of the exact
output (`within`), or of the row where a row is summed on its own.
"""
import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from oracle import layer_ops as lo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def within(got, ref, K, name=""):
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not ref.numel():
        return
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    err = (got.double().cpu() - ref).abs()
    tol = half * ref.abs() * (1 + 2 ** -8) + K * 2.0 ** -24 * max(ref.abs().max().item(), 1e-30)
    bad = ~(err <= tol)
    assert not bad.any(), (name, int(bad.sum()), err.max().item(), tol.max().item())


class Source:
    """Seeded inputs, rounded to their type: .gpu is what the kernels read, and
    d(t) its value in float64."""

    def __init__(self, seed, dtype):
        self.g = torch.Generator().manual_seed(seed)
        self.dtype = TYPES[dtype]

    def __call__(self, *shape, scale=1.0, shift=0.0, dtype=None):
        t = shift + scale * torch.randn(shape, generator=self.g)
        return t.to(dtype or self.dtype)

    def f32(self, *shape, **kw):
        return self(*shape, dtype=torch.float32, **kw)


def up(v):
    return v.to(DEV) if isinstance(v, torch.Tensor) else v


def dd(v):
    return None if v is None else v.double()


def strided(t, pad=3):
    """The same values as a view whose rows lie `pad` elements further apart and
    start one element in: nothing is 16-byte aligned."""
    wide = torch.zeros(t.shape[:-1] + (t.shape[-1] + pad,), dtype=t.dtype, device=DEV)
    view = wide[..., 1:1 + t.shape[-1]]
    view.copy_(t)
    return view


# ---- layer norm ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (5, 64), (2, 203), (257, 768), (9, 1025),
                                        (4, 2560), (1200, 100), (3, 5119), (2, 16384), (0, 32)])
def test_norm(dtype, rows, width):
    s = Source(rows + width, dtype)
    x, w, b = s(rows, width, scale=2.0, shift=0.7), s.f32(width), s.f32(width)
    dy = s(rows, width)
    y, mean, rstd = m.ssd_norm_fwd(up(x), up(w), up(b), eps=1e-5)
    ry, rm, rr = lo.norm(dd(x), dd(w), dd(b), 1e-5)
    K = 16 + 2 * width ** 0.5 + 8  # sums of a row run as trees of at most 64 + log2 terms
    within(mean, rm, 4 * K, "mean")
    within(rstd, rr, 4 * K, "rstd")
    within(y, ry, 4 * K, "y")
    g = m.ssd_norm_bwd(up(x), up(w), mean, rstd, up(dy))
    ref = lo.gradients(lambda x, weight, bias: lo.norm(x, weight, bias, 1e-5),
                       {"x": dd(x), "weight": dd(w), "bias": dd(b)}, [dd(dy)])
    if width > 1:  # of one element dx is 0 up to the rounding of its terms
        within(g["dx"], ref["x"], 8 * K, "dx")
    within(g["dweight"], ref["weight"], 16 + 8 * rows, "dweight")
    within(g["dbias"], ref["bias"], 16 + 4 * rows, "dbias")


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_views_and_options(dtype):
    s = Source(5, dtype)
    x, dy = s(6, 4, 77), s(6, 4, 77)
    xv, dyv = strided(x), strided(dy, 5)
    y, mean, rstd = m.ssd_norm_fwd(xv)
    ry, rm, _ = lo.norm(dd(x), None, None, 1e-5)
    within(y, ry, 100, "y")
    assert mean.shape == (6, 4)
    g = m.ssd_norm_bwd(xv, None, mean, rstd, dyv)
    assert g["dx"].stride() == xv.stride()
    ref = lo.gradients(lambda x: lo.norm(x, None, None, 1e-5), {"x": dd(x)}, [dd(dy)])
    within(g["dx"], ref["x"], 200, "dx")
    # in place
    z = up(x)
    assert m.ssd_norm_fwd(z, y=z)[0] is z
    assert torch.equal(z, y)


# ---- convolution ---------------------------------------------------------------------------

CONV = [  # b, L, E, W, cu
    (1, 1, 1, 2, None), (2, 3, 5, 4, None), (3, 17, 33, 3, None), (2, 40, 203, 4, None),
    (1, 130, 64, 2, None), (1, 65, 1030, 4, None),
    (1, 9, 6, 4, [0, 1, 1, 3, 9]), (1, 50, 37, 4, [0, 0, 2, 3, 19, 50, 50]),
    (1, 64, 96, 3, [0, 16, 32, 64]), (1, 0, 8, 4, [0, 0, 0]), (2, 0, 8, 4, None)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv(dtype, carry, case):
    b, L, E, W, cu = case
    S = b if cu is None else len(cu) - 1
    s = Source(L * E + W, dtype)
    x, w, bias = s(b, L, E), s.f32(W, E), s.f32(E)
    dy = s(b, L, E)
    init = s(S, W - 1, E) if carry else None
    df = s(S, W - 1, E) if carry else None
    cug = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    xv = strided(x)
    y, f = m.ssd_conv_fwd(xv, up(w), up(bias), init_state=up(init), cu_seqlens=cug)
    ref = lambda x, weight, bias, init=None: lo.conv(x, weight, bias, init, cu)
    ins = {"x": dd(x), "weight": dd(w), "bias": dd(bias),
           "init": dd(init) if carry else torch.zeros(S, W - 1, E, dtype=torch.float64)}
    ry, rf = ref(**ins)
    within(y, ry, 40, "y")
    assert torch.equal(f.double().cpu(), rf)
    g = m.ssd_conv_bwd(xv, up(w), up(bias), strided(dy, 2), init_state=up(init), cu_seqlens=cug,
                       d_final=up(df))
    rg = lo.gradients(ref, ins, [dd(dy), dd(df)])
    within(g["dx"], rg["x"], 60, "dx")
    within(g["dweight"], rg["weight"], 40 + 4 * b * L, "dweight")
    within(g["dbias"], rg["bias"], 40 + 4 * b * L, "dbias")
    within(g["dinit_state"], rg["init"], 60, "dinit_state")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [9000, 25000])
def test_conv_long_runs(dtype, L):
    """Enough tokens that every tile and partial sum size is taken, against the
    same call in two shards chained through the state, and a sampled reference."""
    s = Source(3, dtype)
    E, W = 520, 4
    x, w, bias, dy = s(1, L, E), s.f32(W, E, scale=0.5), s.f32(E), s(1, L, E)
    y, f = m.ssd_conv_fwd(up(x), up(w), up(bias))
    cut = 4097
    y0, f0 = m.ssd_conv_fwd(up(x[:, :cut].contiguous()), up(w), up(bias))
    y1, f1 = m.ssd_conv_fwd(up(x[:, cut:].contiguous()), up(w), up(bias), init_state=f0)
    assert torch.equal(torch.cat([y0, y1], 1), y) and torch.equal(f1, f)
    e = slice(250, 262)
    line = torch.cat([torch.zeros(1, W - 1, 12, dtype=torch.float64), dd(x[..., e])], 1)
    v = sum(line[:, k:k + L] * dd(w[k, e]) for k in range(W)) + dd(bias[e])
    within(y[..., e], lo.silu(v), 40, "y")
    g = m.ssd_conv_bwd(up(x), up(w), up(bias), up(dy))
    sg = torch.sigmoid(v)
    dv = dd(dy[..., e]) * sg * (1 + v * (1 - sg))
    pad = torch.cat([dv, torch.zeros(1, W - 1, 12, dtype=torch.float64)], 1)
    within(g["dx"][..., e], sum(pad[:, j:j + L] * dd(w[W - 1 - j, e]) for j in range(W)), 60, "dx")
    within(g["dweight"][:, e],
           torch.stack([(dv * line[:, k:k + L]).sum((0, 1)) for k in range(W)]), 4 * L, "dweight")
    within(g["dbias"][e], dv.sum((0, 1)), 4 * L, "dbias")


# ---- single tokens -------------------------------------------------------------------------

def pool(s, b, spare, *row, dtype=None, scale=1.0):
    """A pool of b + spare rows and the batch's slots in some order."""
    slots = torch.randperm(b + spare, generator=s.g)[:b].to(torch.int32)
    return s(b + spare, *row, dtype=dtype, scale=scale), slots


def check_pool(new, ref_rows, slots, before, K, name):
    """Written rows against the reference, the others untouched."""
    within(new[slots.long()], ref_rows, K, name)
    rest = torch.ones(len(new), dtype=torch.bool)
    rest[slots.long()] = False
    assert torch.equal(new.cpu()[rest], before[rest])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b,E,W", [(1, 1, 2), (3, 33, 4), (64, 203, 3), (7, 5376, 4)])
def test_conv_step(dtype, b, E, W):
    s = Source(b + E, dtype)
    state, slots = pool(s, b, 3, W - 1, E)
    x, w, bias = s(b, E), s.f32(W, E), s.f32(E)
    new = torch.full_like(state, 9.0)
    ng = up(new.clone())
    y = m.ssd_conv_step(strided(x), up(state), up(w), up(bias), slots=up(slots), new_state=ng)
    ry, rf = lo.conv(dd(x)[:, None], dd(w), dd(bias), dd(state)[slots.long()])
    within(y, ry[:, 0], 40, "y")
    check_pool(ng, rf, slots, new, 0, "state")
    sg = up(state)
    y2 = m.ssd_conv_step(up(x), sg, up(w), up(bias), slots=up(slots))  # in place
    assert torch.equal(y, y2) and torch.equal(sg[slots.long()], ng[slots.long()])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b,E,N,G", [(1, 1, 1, 1), (3, 66, 8, 2), (5, 203, 16, 1), (2, 40, 33, 1),
                                     (64, 4098, 16, 2), (33, 9000, 16, 1)])
@pytest.mark.parametrize("gated", [False, True])
def test_selscan_step(dtype, b, E, N, G, gated):
    s = Source(b + E + N, dtype)
    state, slots = pool(s, b, 2, N, E, dtype=torch.float32)
    x, raw, dinit, A = s(b, E), s(b, E), s.f32(E), -s.f32(N, E).exp()
    B, C = s(b, G, N), s(b, G, N)
    D, z = (s.f32(E), s(b, E)) if gated else (None, None)
    ng = up(torch.zeros_like(state))
    y = m.ssd_selscan_step(strided(x), strided(raw), up(dinit), up(A), strided(B), strided(C),
                           up(state), D=up(D), z=None if z is None else strided(z),
                           slots=up(slots), new_state=ng)
    one = lambda t: None if t is None else dd(t)[:, None]
    ry, rf = lo.selscan(one(x), one(raw), dd(dinit), dd(A), one(B), one(C), dd(D), one(z),
                        dd(state)[slots.long()])
    within(y, ry[:, 0], 40 + 4 * N, "y")
    check_pool(ng, rf, slots, torch.zeros_like(state), 40, "state")
    sg = up(state)
    y2 = m.ssd_selscan_step(up(x), up(raw), up(dinit), up(A), up(B), up(C), sg, D=up(D), z=up(z),
                            slots=up(slots))
    assert torch.equal(y, y2) and torch.equal(sg[slots.long()], ng[slots.long()])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b,H,P,N,G", [(1, 1, 16, 16, 1), (1, 24, 64, 128, 1), (5, 6, 48, 32, 2),
                                       (3, 4, 128, 64, 4), (64, 8, 80, 16, 1), (2, 3, 512, 256, 1)])
def test_ssd_step(dtype, b, H, P, N, G):
    s = Source(b + H + P + N, dtype)
    state, slots = pool(s, b, 2, H, N, P, dtype=torch.float32)
    x, raw, B, C = s(b, H, P), s(b, H), s(b, G, N), s(b, G, N)
    ng = up(torch.zeros_like(state))
    y = m.ssd_step(strided(x), strided(raw), -1.5, strided(B), strided(C), up(state),
                   slots=up(slots), new_state=ng)
    ry, rf = lo.ssd_token(dd(x), dd(raw), -1.5, dd(B), dd(C), dd(state)[slots.long()])
    within(y, ry, 40 + 4 * N, "y")
    check_pool(ng, rf, slots, torch.zeros_like(state), 40, "state")
    sg = up(state)
    y2 = m.ssd_step(up(x), up(raw), -1.5, up(B), up(C), sg, slots=up(slots))
    assert torch.equal(y, y2) and torch.equal(sg[slots.long()], ng[slots.long()])


def test_steps_leave_padding_rows_alone():
    """Slots outside the pool: y is 0 and no state changes."""
    s = Source(1, "bf16")
    slots = torch.tensor([-1, 2, 5, 1 << 30], dtype=torch.int32, device=DEV)
    st = up(s(4, 3, 40))
    y = m.ssd_conv_step(up(s(4, 40)), st, up(s.f32(4, 40)), slots=slots, new_state=(n := st.clone()))
    assert not y[[0, 2, 3]].any() and y[1].any()
    assert torch.equal(n[[0, 1, 3]], st[[0, 1, 3]]) and not torch.equal(n[2], st[2])
    st = up(s.f32(4, 16, 40))
    y = m.ssd_selscan_step(up(s(4, 40)), up(s(4, 40)), up(s.f32(40)), up(-s.f32(16, 40).exp()),
                           up(s(4, 1, 16)), up(s(4, 1, 16)), st, slots=slots, new_state=(n := st.clone()))
    assert not y[[0, 2, 3]].any() and y[1].any()
    assert torch.equal(n[[0, 1, 3]], st[[0, 1, 3]]) and not torch.equal(n[2], st[2])
    st = up(s.f32(4, 2, 16, 32))
    y = m.ssd_step(up(s(4, 2, 32)), up(s(4, 2)), -1.0, up(s(4, 1, 16)), up(s(4, 1, 16)), st,
                   slots=slots, new_state=(n := st.clone()))
    assert not y[[0, 2, 3]].any() and y[1].any()
    assert torch.equal(n[[0, 1, 3]], st[[0, 1, 3]]) and not torch.equal(n[2], st[2])


# ---- selective scan ------------------------------------------------------------------------

SCAN = [  # b, L, E, N, G, cu
    (1, 1, 1, 1, 1, None), (2, 2, 17, 3, 1, None), (1, 15, 16, 16, 1, None),
    (2, 17, 40, 16, 2, None), (3, 77, 203, 16, 1, None), (1, 257, 20, 16, 1, None),
    (1, 300, 33, 8, 1, None), (2, 70, 34, 32, 2, None), (1, 90, 10, 33, 1, None),
    (1, 40, 18, 64, 1, None), (1, 520, 5, 7, 1, None),
    (1, 9, 6, 16, 1, [0, 1, 1, 3, 9]), (1, 300, 24, 16, 1, [0, 0, 2, 19, 275, 300, 300]),
    (1, 140, 12, 8, 2, [0, 128, 140]),
    # long with few channels: cut into spans
    (1, 2600, 20, 16, 1, None), (2, 1500, 9, 8, 1, None), (1, 700, 6, 40, 1, None),
    (1, 900, 34, 32, 2, None), (1, 2300, 18, 16, 1, [0, 0, 700, 701, 2300, 2300]),
    # the fewest waves a workgroup: few tokens, many sequences
    (2, 7, 10, 33, 1, None), (2, 9, 10, 20, 1, None), (2, 20, 10, 16, 1, None),
    (1, 1300, 8, 16, 1, list(range(0, 900)) + [1000, 1040, 1300] + [1300] * 200),
    # many channels: workgroups of half and a quarter of the waves
    (1, 100, 8320, 16, 1, None), (1, 70, 16480, 16, 1, None),
    (1, 0, 8, 16, 1, [0, 0, 0]), (2, 0, 8, 16, 1, None)]


def scan_id(case):
    return str(case if case[5] is None or len(case[5]) < 20 else case[:5] + ("many",))


def scan_problem(dtype, case, gated=True, carry=True, seed=0):
    b, L, E, N, G, cu = case
    S = b if cu is None else len(cu) - 1
    s = Source(L * E + N + seed, dtype)
    p = {"x": s(b, L, E), "raw": s(b, L, E), "dinit": s.f32(E, shift=-2.0), "A": -s.f32(N, E).exp(),
         "B": s(b, L, G, N), "C": s(b, L, G, N),
         "D": s.f32(E) if gated else None, "z": s(b, L, E) if gated else None,
         "init": s.f32(S, N, E) if carry else None}
    seeds = (s(b, L, E), s.f32(S, N, E) if carry else None)
    return p, seeds, cu


def scan_call(p, cu, view=up):
    v = lambda k: None if p[k] is None else view(p[k])
    cug = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    args = (v("x"), v("raw"), up(p["dinit"]), up(p["A"]), v("B"), v("C"))
    return args, dict(D=up(p["D"]), z=v("z"), init_state=up(p["init"]), cu_seqlens=cug)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gated,carry", [(True, True), (False, False)])
@pytest.mark.parametrize("case", SCAN, ids=scan_id)
def test_selscan(dtype, gated, carry, case):
    p, (dy, df), cu = scan_problem(dtype, case, gated, carry)
    b, L, E, N, G, _ = case
    args, kw = scan_call(p, cu, strided)
    y, f = m.ssd_selscan_fwd(*args, **kw)
    ins = {k: dd(v) for k, v in p.items()}
    if not carry:
        ins["init"] = torch.zeros(len(f), N, E, dtype=torch.float64)
    fn = lambda **k: lo.selscan(**k, cu=cu)
    ry, rf = fn(**ins)
    within(y, ry, 64 + 4 * L, "y")
    within(f, rf, 64 + 4 * L, "final_state")
    g = m.ssd_selscan_bwd(*args, strided(dy, 2), **kw, d_final=up(df))
    rg = lo.gradients(fn, ins, [dd(dy), dd(df)])
    names = {"x": "dx", "raw": "dd_raw", "dinit": "dd_init", "A": "dA", "B": "dB", "C": "dC",
             "D": "dD", "z": "dz", "init": "dinit_state"}
    for k, ref in rg.items():
        # sums over tokens, channels or entries on top of the states' own errors
        within(g[names[k]], ref, 4 * (64 + 4 * b * L) + 4 * E, names[k])
    if not gated:
        assert "dz" not in g


@pytest.mark.parametrize("dtype", TYPES)
def test_selscan_chains(dtype):
    """One call equals two through the state, and single tokens through the pool."""
    case = (2, 330, 48, 16, 1, None)
    p, _, _ = scan_problem(dtype, case)
    args, kw = scan_call(p, None)
    y, f = m.ssd_selscan_fwd(*args, **kw)
    cut = lambda t, a, b: t if t is None or t.dim() < 3 or t.shape[1] != 330 else t[:, a:b].contiguous()
    st, parts = kw["init_state"], []
    for a, b in ((0, 1), (1, 129), (129, 330)):
        o, st = m.ssd_selscan_fwd(*(cut(t, a, b) for t in args), D=kw["D"], z=cut(kw["z"], a, b),
                                  init_state=st)
        parts.append(o)
    within(torch.cat(parts, 1), dd(y.cpu()), 64 + 4 * 330 + 2 ** 17 * (dtype == "bf16"), "y")
    within(st, dd(f.cpu()), 64 + 4 * 330, "state")
    pool_, tokens = kw["init_state"].clone(), []
    for t in range(40):
        at = lambda q: q if q is None or q.dim() < 3 else q[:, t]
        tokens.append(m.ssd_selscan_step(args[0][:, t], args[1][:, t], args[2], args[3], args[4][:, t],
                                         args[5][:, t], pool_, D=kw["D"], z=kw["z"][:, t]))
    within(torch.stack(tokens, 1), dd(y[:, :40].cpu()), 64 + 4 * 40 + 2 ** 17 * (dtype == "bf16"), "tokens")


def test_ssd_step_continues_ssd_fwd():
    """Tokens after a prompt: ssd_fwd's final state goes on in the pool."""
    s = Source(9, "f32")
    b, L, H, P, N = 2, 100, 4, 32, 16
    x, raw, B, C = s(b, L, H, P), s(b, L, H), s(b, L, 1, N), s(b, L, 1, N)
    y, f = m.ssd_fwd(up(x), up(raw), -1.0, up(B), up(C))
    cut = 90
    y0, st = m.ssd_fwd(*(up(t[:, :cut].contiguous()) for t in (x, raw)), -1.0,
                       *(up(t[:, :cut].contiguous()) for t in (B, C)))
    for t in range(cut, L):
        yt = m.ssd_step(up(x[:, t]), up(raw[:, t]), -1.0, up(B[:, t]), up(C[:, t]), st)
        assert (yt - y[:, t]).abs().max().item() <= 1e-4 * y.abs().max().item()
    assert (st - f).abs().max().item() <= 1e-4 * f.abs().max().item()


def test_selscan_extremes():
    """Decays of 0 and -inf, steps that vanish, gates that close: no NaN, and the
    values of the definition."""
    p, _, _ = scan_problem("f32", (1, 40, 20, 16, 1, None))
    p["A"][0], p["A"][1] = 0.0, -float("inf")
    p["raw"][0, :, 3] = -1e4
    p["z"][0, :, 4] = -200.0
    args, kw = scan_call(p, None)
    y, f = m.ssd_selscan_fwd(*args, **kw)
    ins = {k: dd(v) for k, v in p.items()}
    ins["A"][1] = -1e300
    ry, rf = lo.selscan(**ins)
    within(y, ry, 64 + 160, "y")
    within(f, rf, 64 + 160, "final")
    at = lambda t: t[:, 0]
    st = kw["init_state"].clone()
    y1 = m.ssd_selscan_step(*map(at, args[:2]), args[2], args[3], *map(at, args[4:]), st, D=kw["D"],
                            z=at(kw["z"]))
    within(y1, ry[:, 0], 64, "token")
    assert torch.isfinite(st).all()


def test_masked_places_do_not_spread():
    """NaN in one sequence, in rows behind the sequences' and in padding rows'
    states stays there."""
    case = (1, 90, 20, 16, 1, [0, 40, 41, 90])
    p, (dy, df), cu = scan_problem("f32", case)
    args, kw = scan_call(p, cu)
    g0 = m.ssd_selscan_bwd(*args, up(dy), **kw, d_final=up(df))
    y0, f0 = m.ssd_selscan_fwd(*args, **kw)
    w = up(torch.randn(4, 20))
    c0, _ = m.ssd_conv_fwd(args[0], w, cu_seqlens=kw["cu_seqlens"])
    args[0][0, 40] = float("nan")  # the sequence of one token
    y, f = m.ssd_selscan_fwd(*args, **kw)
    c, _ = m.ssd_conv_fwd(args[0], w, cu_seqlens=kw["cu_seqlens"])
    g = m.ssd_selscan_bwd(*args, up(dy), **kw, d_final=up(df))
    keep = [t for t in range(90) if t != 40]
    assert torch.equal(y[0, keep], y0[0, keep]) and torch.equal(f[[0, 2]], f0[[0, 2]])
    assert torch.equal(c[0, keep], c0[0, keep])
    for k in ("dx", "dd_raw", "dz", "dB", "dC"):
        assert torch.equal(g[k][0, keep], g0[k][0, keep]), k
    assert torch.equal(g["dinit_state"][[0, 2]], g0["dinit_state"][[0, 2]])


def test_offsets_past_32_bits():
    """Pools and token strides whose far ends lie beyond 2^31 elements and 2^32
    bytes: the same results as near ones."""
    s = Source(21, "bf16")
    H, N, P, far = 4, 128, 64, 66000
    pool_ = torch.zeros((far, H, N, P), device=DEV)
    near = up(s.f32(1, H, N, P))
    pool_[far - 1] = near[0]
    x, raw, B = up(s(1, H, P)), up(s(1, H)), up(s(1, 1, N))
    slots = torch.tensor([far - 1], dtype=torch.int32, device=DEV)
    y = m.ssd_step(x, raw, -1.0, B, B, pool_, slots=slots)
    assert torch.equal(y, m.ssd_step(x, raw, -1.0, B, B, near)) and torch.equal(pool_[far - 1], near[0])
    flat = pool_.view(far, 16, 2048)
    a, x, d = up(-s.f32(16, 2048).exp()), up(s(1, 2048)), up(s.f32(2048))
    near = flat[far - 1:].clone()
    B = up(s(1, 1, 16))
    y = m.ssd_selscan_step(x, x, d, a, B, B, flat, slots=slots)
    assert torch.equal(y, m.ssd_selscan_step(x, x, d, a, B, B, near)) and torch.equal(flat[far - 1], near[0])
    del pool_, flat
    L, E, stride = 300, 40, (1 << 23) + 1
    wide = torch.empty((1, L, stride), dtype=torch.bfloat16, device=DEV)
    x = up(s(1, L, E))
    xv = wide[..., 5:5 + E]
    xv.copy_(x)
    w, a, d = up(s.f32(4, E)), up(-s.f32(16, E).exp()), up(s.f32(E))
    B = up(s(1, L, 1, 16))
    assert torch.equal(m.ssd_conv_fwd(xv, w)[0], m.ssd_conv_fwd(x, w)[0])
    assert torch.equal(m.ssd_norm_fwd(xv)[0], m.ssd_norm_fwd(x)[0])
    assert torch.equal(m.ssd_selscan_fwd(xv, xv, d, a, B, B, z=xv)[0], m.ssd_selscan_fwd(x, x, d, a, B, B, z=x)[0])
    dx = m.ssd_conv_bwd(xv, w, None, xv)["dx"]
    assert torch.equal(dx, m.ssd_conv_bwd(x, w, None, x)["dx"])
    del dx
    g = m.ssd_selscan_bwd(xv, x, d, a, B, B, xv)
    g0 = m.ssd_selscan_bwd(x, x, d, a, B, B, x)
    assert all(torch.equal(g[k], g0[k]) for k in g)


# ---- how calls run -------------------------------------------------------------------------

def calls():
    """One small call of every operator as a function of nothing."""
    s = Source(77, "bf16")
    p, (dy, df), _ = scan_problem("bf16", (2, 150, 40, 16, 1, None))
    args, kw = scan_call(p, None)
    w, bias = up(s.f32(4, 40)), up(s.f32(40))
    dyg, dfg = up(dy), up(df)
    _, mean, rstd = m.ssd_norm_fwd(args[0], bias, bias)
    st, cst = kw["init_state"], up(s(2, 3, 40))
    hx, hraw, hB, hst = up(s(2, 4, 16)), up(s(2, 4)), up(s(2, 1, 16)), up(s.f32(2, 4, 16, 16))
    tok = [t[:, 0].contiguous() for t in (args[0], args[1], args[4], args[5])]
    return {
        "norm_fwd": lambda: m.ssd_norm_fwd(args[0], bias, bias),
        "norm_bwd": lambda: m.ssd_norm_bwd(args[0], bias, mean, rstd, dyg),
        "conv_fwd": lambda: m.ssd_conv_fwd(args[0], w, bias),
        "conv_bwd": lambda: m.ssd_conv_bwd(args[0], w, bias, dyg),
        "conv_step": lambda: m.ssd_conv_step(tok[0], cst, w, bias, new_state=torch.empty_like(cst)),
        "selscan_fwd": lambda: m.ssd_selscan_fwd(*args, **kw),
        "selscan_bwd": lambda: m.ssd_selscan_bwd(*args, dyg, **kw, d_final=dfg),
        "selscan_step": lambda: m.ssd_selscan_step(tok[0], tok[1], args[2], args[3], tok[2], tok[3],
                                                   st, new_state=torch.empty_like(st)),
        "ssd_step": lambda: m.ssd_step(hx, hraw, -1.0, hB, hB, hst, new_state=torch.empty_like(hst)),
    }


def tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    out = out.values() if isinstance(out, dict) else out
    return [t for t in out if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("name", ["norm_fwd", "norm_bwd", "conv_fwd", "conv_bwd", "conv_step",
                                  "selscan_fwd", "selscan_bwd", "selscan_step", "ssd_step"])
def test_same_bits_on_a_stream_and_in_a_graph(name):
    """A call gives the same bits again, on another stream, and when captured
    and replayed with eager work between the replays."""
    f = calls()[name]
    want = [t.clone() for t in tensors(f())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [t.clone() for t in tensors(f())]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = tensors(f())
    for _ in range(3):
        for t in held:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held))
        assert all(torch.equal(a, b) for a, b in zip(want, tensors(f())))


def test_checked_cu_seqlens(monkeypatch):
    """With SSD_CHECK=1 bounds that are not 0..L in order are an error, before
    anything is launched."""
    monkeypatch.setenv("SSD_CHECK", "1")
    p, (dy, df), _ = scan_problem("bf16", (1, 60, 24, 16, 1, [0, 20, 60]))
    w = torch.ones(4, 24, device=DEV)
    for cu, ok in (([0, 20, 60], True), ([0, 70, 60], False), ([1, 20, 60], False),
                   ([0, 20, 59], False)):
        args, kw = scan_call(p, cu)
        for f in (lambda: m.ssd_selscan_fwd(*args, **kw),
                  lambda: m.ssd_selscan_bwd(*args, up(dy), **kw, d_final=up(df)),
                  lambda: m.ssd_conv_fwd(args[0], w, cu_seqlens=kw["cu_seqlens"]),
                  lambda: m.ssd_conv_bwd(args[0], w, None, up(dy), cu_seqlens=kw["cu_seqlens"])):
            if ok:
                f()
            else:
                with pytest.raises(m.SsdError) as e:
                    f()
                assert e.value.status == -8
