"""Linear attention with a decay per head on the GPU against the fp64 recurrence.

Tolerances.  With |.| for the same expression of the inputs' absolute values
(every product and every weight is then positive, so it bounds the sum of the
terms' sizes): an output in float32 is off by at most K 2^-24 |.|, K = 16 + 4 L
roundings on the way; a bfloat16 output is also rounded once itself (half a
step of its value), and before that every score and every state entry that a
query meets was rounded once (half a step of each term, so of |.|).  States are
never rounded below 24 bits.
"""
import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from oracle import linattn_ops as lo

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def near(got, ref, size, L, name):
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    err = (got.double().cpu() - ref).abs()
    tol = (16 + 4 * L) * 2.0 ** -24 * size + 1e-37
    if got.dtype == torch.bfloat16:
        half = torch.finfo(got.dtype).eps / 2
        tol = tol + half * (ref.abs() + size) * (1 + 2 * half)
    bad = ~(err <= tol)
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:4].tolist(), err.max().item())


def make(dtype, b, L, H, G, K, V, cu=None, carry=True, seed=0, decay=None):
    g = torch.Generator().manual_seed(seed + 1000 * K + V + L)
    r = lambda *s, dt=TYPES[dtype], c=1.0: (c * torch.randn(s, generator=g)).to(dt)
    S = b if cu is None else len(cu) - 1
    if decay is None:
        decay = -torch.exp(torch.linspace(0.5, -7.0, H))
    f = torch.float32
    return dict(q=r(b, L, H, K), k=r(b, L, G, K), v=r(b, L, G, V), decay=decay, dy=r(b, L, H, V),
                init=r(S, H, K, V, dt=f) if carry else None,
                d_final=r(S, H, K, V, dt=f, c=0.3) if carry else None)


def up(t):
    return None if t is None else t.to(DEV)


def cu_of(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)


def d(t):
    return None if t is None else t.double()


def a(t):
    return None if t is None else t.double().abs()


def check_fwd(s, cu=None, reverse=False, scale=0.37, view=lambda t: t):
    y, final = m.ssd_linattn_fwd(view(up(s["q"])), view(up(s["k"])), view(up(s["v"])), up(s["decay"]),
                                 scale=scale, init_state=up(s["init"]), cu_seqlens=cu_of(cu),
                                 reverse=reverse)
    kw = dict(scale=scale, cu=cu, reverse=reverse)
    ry, rf = lo.linattn(d(s["q"]), d(s["k"]), d(s["v"]), d(s["decay"]), init=d(s["init"]), **kw)
    ay, af = lo.linattn(a(s["q"]), a(s["k"]), a(s["v"]), d(s["decay"]), init=a(s["init"]), **kw)
    L = s["q"].shape[1]
    near(y, ry, ay, L, "y")
    near(final, rf, af, L, "final_state")
    return y, final


def check_bwd(s, cu=None, reverse=False, scale=0.37, view=lambda t: t):
    g = m.ssd_linattn_bwd(view(up(s["q"])), view(up(s["k"])), view(up(s["v"])), up(s["decay"]),
                          view(up(s["dy"])), scale=scale, init_state=up(s["init"]),
                          cu_seqlens=cu_of(cu), reverse=reverse, d_final=up(s["d_final"]))
    kw = dict(scale=scale, cu=cu, reverse=reverse)
    ref = lo.linattn_grads(d(s["q"]), d(s["k"]), d(s["v"]), d(s["decay"]), d(s["dy"]), d(s["d_final"]),
                           init=d(s["init"]), **kw)
    size = lo.linattn_grads(a(s["q"]), a(s["k"]), a(s["v"]), d(s["decay"]), a(s["dy"]), a(s["d_final"]),
                            init=a(s["init"]), **kw)
    assert sorted(g) == sorted(ref)
    for n in ref:
        near(g[n], ref[n], size[n], s["q"].shape[1], n)
    return g


DIMS = [(1, 1), (16, 16), (40, 56), (64, 128), (77, 33), (128, 64), (128, 128), (130, 200), (256, 256)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K,V", DIMS)
def test_head_sizes(dtype, K, V):
    s = make(dtype, 2, 150, 2, 2, K, V)
    check_fwd(s)
    check_bwd(s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 193])
def test_lengths(dtype, L):
    s = make(dtype, 3, L, 2, 1, 48, 72)
    check_fwd(s, reverse=L % 2 == 0)
    check_bwd(s, reverse=L % 3 == 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,G", [(4, 4), (4, 2), (6, 1)])
@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("reverse", [False, True])
def test_packed(dtype, H, G, carry, reverse):
    cu = [0, 0, 5, 5, 70, 134, 135, 400, 400]
    s = make(dtype, 1, 400, H, G, 24, 40, cu=cu, carry=carry)
    check_fwd(s, cu, reverse)
    check_bwd(s, cu, reverse)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b,L,cu", [(1, 2500, None), (2, 900, None),
                                    (1, 2100, [0, 0, 1, 130, 1000, 1000, 2099, 2100])])
def test_long_sequences_in_spans(dtype, b, L, cu):
    """Few heads: sequences are cut, their states joined."""
    s = make(dtype, b, L, 2, 1, 32, 20, cu=cu)
    assert m._layer._entry("ssd_linattn_fwd_workspace_bytes")(
        m.SsdLinattnDims(b, L, 2, 1, 32, 20, 0 if cu is None else len(cu) - 1, 0, 1.0, 0)) > 0
    check_fwd(s, cu)
    check_bwd(s, cu, reverse=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (200, 90)])
@pytest.mark.parametrize("reverse", [False, True])
def test_whole_numbers_are_exact(dtype, K, V, reverse):
    """No decay and few small whole numbers: scores and states stay whole and below 257, so
    nothing is rounded but the result."""
    g = torch.Generator().manual_seed(K)
    L, H = 333, 3
    pick = lambda *s: ((torch.rand(s, generator=g) < 0.1).double() * torch.randint(-1, 2, s, generator=g)).to(TYPES[dtype])
    q, k, v, dy = pick(1, L, H, K), pick(1, L, H, K), pick(1, L, H, V), pick(1, L, H, V)
    decay = torch.zeros(H)
    y, final = m.ssd_linattn_fwd(up(q), up(k), up(v), up(decay), reverse=reverse)
    ry, rf = lo.linattn(d(q), d(k), d(v), d(decay), reverse=reverse)
    assert rf.abs().max() < 257
    assert torch.equal(y.cpu(), ry.to(y.dtype)) and torch.equal(final.cpu(), rf.float())
    got = m.ssd_linattn_bwd(up(q), up(k), up(v), up(decay), up(dy), reverse=reverse)
    for n, r in lo.linattn_grads(d(q), d(k), d(v), d(decay), d(dy), reverse=reverse).items():
        assert torch.equal(got[n].cpu(), r.to(got[n].dtype)), n


@pytest.mark.parametrize("dtype", TYPES)
def test_views_and_alignment(dtype):
    """Rows of one projection, at any element alignment and in reverse order of the heads."""
    s = make(dtype, 2, 100, 3, 3, 24, 40)

    def odd(t):
        if t is None:
            return None
        b, L, H, D = t.shape
        wide = torch.full((b, L, H * (D + 3) + 1), 7.0, dtype=t.dtype, device=DEV)
        view = wide[..., 1:].unflatten(-1, (H, D + 3))[..., :D]
        view.copy_(t)
        return view

    y, final = check_fwd(s, view=odd)
    y0, f0 = check_fwd(s)
    assert torch.equal(y, y0) and torch.equal(final, f0)
    g, g0 = check_bwd(s, view=odd), check_bwd(s)
    assert all(torch.equal(g[n], g0[n]) for n in g)
    # one key head for all, as an expanded view
    k = up(s["k"][:, :, :1]).expand(-1, -1, 3, -1)
    v = up(s["v"][:, :, :1]).expand(-1, -1, 3, -1)
    y1, _ = m.ssd_linattn_fwd(up(s["q"]), k, v, up(s["decay"]))
    y2, _ = m.ssd_linattn_fwd(up(s["q"]), k[:, :, :1], v[:, :, :1], up(s["decay"]))
    assert torch.equal(y1, y2)
    # into a strided y
    into = torch.zeros(2, 100, 3, 80, dtype=TYPES[dtype], device=DEV)
    m.ssd_linattn_fwd(up(s["q"]), up(s["k"]), up(s["v"]), up(s["decay"]), scale=0.37,
                      init_state=up(s["init"]), y=into[..., 20:60])
    assert torch.equal(into[..., 20:60], y0) and not into[..., :20].any() and not into[..., 60:].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_rates_at_the_ends(dtype):
    """No decay, almost none, strong, and nothing kept at all."""
    decay = torch.tensor([0.0, -1e-6, -30.0, float("-inf")])
    s = make(dtype, 2, 140, 4, 4, 16, 24, decay=decay)
    check_fwd(s)
    check_bwd(s)


def test_slow_decay_over_many_chunks():
    """Ones are the geometric series.  A sum of n equal terms is rounded alike every time: the
    state takes 4 tokens a matrix instruction (float32), each a rounding of at most 2^-24 of
    the state then, which the result exceeds, and one more every 32 tokens for its rate: n / 4
    + n / 32, and 16 for the output's own products."""
    decay = torch.tensor([-1e-5, -3e-7])
    L = 20000
    q = torch.ones(64, L // 64 * 64, 2, 1)[:, :L // 4]
    q = q.to(DEV)
    y, final = m.ssd_linattn_fwd(q, q, q, decay.to(DEV))
    n = torch.arange(1, L // 4 + 1, dtype=torch.float64)[:, None]
    dd = decay.double()
    ref = torch.expm1(n * dd) / torch.expm1(dd)
    assert ((y[0, :, :, 0].double().cpu() - ref).abs() / ref <= (16 + n / 4 + n / 32) * 2.0 ** -24).all()


def test_rate_over_many_chunks():
    """A state that nothing is added to, over 1000 chunks: its entries' own roundings differ
    and average out (1000 roundings of +-2^-24 at most, uniform, over 4096 entries a head: a mean
    of 0.28 2^-24 deviation), an error of the rate would not (half a step of it 1000 times)."""
    L, decay = 32000, torch.tensor([-1.7e-6, -3.1e-5, -1.3e-6, -7.7e-6])
    z = torch.zeros(1, L, 4, 64, device=DEV)
    init = 1 + torch.rand((1, 4, 64, 64), generator=torch.Generator().manual_seed(1))
    span = torch.full((64, L // 64, 4, 64), 0.0, device=DEV)
    for x, first in ((z, init), (span, init.expand(64, -1, -1, -1).contiguous())):
        final = m.ssd_linattn_fwd(x, x, x, decay.to(DEV), init_state=first.to(DEV))[1]
        ref = first.double() * torch.exp(x.shape[1] * decay.double())[:, None, None]
        assert ((final.double().cpu() / ref - 1).mean((0, 2, 3)).abs() < 4 * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_nan_stays_in_its_sequence_and_other_rows_stay(dtype):
    cu = [0, 70, 100, 300]
    s = make(dtype, 1, 330, 2, 2, 16, 16, cu=cu)
    clean, cf = m.ssd_linattn_fwd(up(s["q"]), up(s["k"]), up(s["v"]), up(s["decay"]), cu_seqlens=cu_of(cu))
    for n in ("q", "k", "v", "dy"):
        s[n][0, 70:100] = float("nan")
        s[n][0, 300:] = float("nan")  # behind the last sequence
    y = torch.full((1, 330, 2, 16), 5.0, dtype=TYPES[dtype], device=DEV)
    _, final = m.ssd_linattn_fwd(up(s["q"]), up(s["k"]), up(s["v"]), up(s["decay"]), cu_seqlens=cu_of(cu), y=y)
    assert torch.equal(y[0, :70], clean[0, :70]) and torch.equal(y[0, 100:300], clean[0, 100:300])
    assert y[0, 70:100].isnan().all() and (y[0, 300:] == 5).all()
    assert torch.equal(final[[0, 2]], cf[[0, 2]])
    g = m.ssd_linattn_bwd(up(s["q"]), up(s["k"]), up(s["v"]), up(s["decay"]), up(s["dy"]), cu_seqlens=cu_of(cu))
    for n in ("dq", "dk", "dv"):
        assert not g[n][0, :70].isnan().any() and not g[n][0, 100:300].isnan().any(), n
    assert not g["dinit_state"][[0, 2]].isnan().any()


def test_no_tokens():
    init = torch.randn(3, 2, 8, 8, device=DEV)
    q = torch.zeros(3, 0, 2, 8, device=DEV)
    decay = torch.tensor([-1.0, -2.0], device=DEV)
    y, final = m.ssd_linattn_fwd(q, q, q, decay, init_state=init)
    assert y.shape == (3, 0, 2, 8) and torch.equal(final, init)
    g = m.ssd_linattn_bwd(q, q, q, decay, y, d_final=init)
    assert torch.equal(g["dinit_state"], init)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b,L,H", [(40, 100, 16), (1, 3000, 2)])
def test_states_in_place(dtype, b, L, H):
    """init_state's buffer as final_state, d_final's as dinit_state (C ABI), whole and in spans."""
    s = make(dtype, b, L, H, H, 16, 16)
    q, k, v, dec, dy = (up(s[n]) for n in ("q", "k", "v", "decay", "dy"))
    y, final = m.ssd_linattn_fwd(q, k, v, dec, init_state=up(s["init"]))
    state = up(s["init"])
    y1, f1 = m.ssd_linattn_fwd(q, k, v, dec, init_state=state, final_state=state)
    assert f1 is state and torch.equal(y, y1) and torch.equal(final, state)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b,H,G,K,V", [(1, 1, 1, 1, 1), (3, 4, 2, 77, 33), (5, 3, 3, 64, 128),
                                       (2, 2, 1, 256, 256), (64, 8, 8, 40, 70), (4, 2, 2, 5, 3)])
def test_single_tokens(dtype, b, H, G, K, V):
    s = make(dtype, b, 1, H, G, K, V)
    q, k, v = (s[n][:, 0] for n in ("q", "k", "v"))
    g = torch.Generator().manual_seed(3)
    pool = torch.randn((b + 3, H, K, V), generator=g)
    slots = torch.randperm(b + 3, generator=g)[:b].to(torch.int32)
    ref, state = lo.linattn(d(s["q"]), d(s["k"]), d(s["v"]), d(s["decay"]), 0.37, init=d(pool)[slots.long()])
    size, asize = lo.linattn(a(s["q"]), a(s["k"]), a(s["v"]), d(s["decay"]), 0.37, init=a(pool)[slots.long()])
    half = torch.finfo(TYPES[dtype]).eps / 2 if dtype == "bf16" else 0.0
    for place in ("same", "other"):
        old = pool.to(DEV)
        new = old if place == "same" else torch.full_like(old, 9.0)
        y = m.ssd_linattn_step(up(q), up(k), up(v), up(s["decay"]), old, scale=0.37, slots=up(slots),
                               new_state=None if place == "same" else new)
        err = (y.double().cpu() - ref[:, 0]).abs()
        # all sums in float32: K terms, and one rounding of the result
        assert (err <= half * ref[:, 0].abs() * (1 + half) + (16 + 4 * K) * 2.0 ** -24 * size[:, 0] + 1e-37).all()
        got = new.cpu()
        assert ((got[slots.long()].double() - state).abs() <= 8 * 2.0 ** -24 * asize + 1e-37).all()
        others = [i for i in range(b + 3) if i not in slots.tolist()]
        assert torch.equal(got[others], pool[others] if place == "same" else torch.full_like(got[others], 9.0))


def test_single_tokens_padding_rows_and_views():
    s = make("f32", 4, 1, 2, 2, 24, 20)
    wide = torch.randn(4, 2, 100, device=DEV)
    q, k, v = wide[..., 1:25], wide[..., 30:54], wide[..., 55:75]
    pool = torch.randn(5, 2, 24, 20, device=DEV)
    keep = pool.clone()
    slots = torch.tensor([3, -1, 5, 0], dtype=torch.int32, device=DEV)
    y = m.ssd_linattn_step(q, k, v, up(s["decay"]), pool, slots=slots)
    assert not y[1].any() and not y[2].any() and torch.equal(pool[[1, 2, 4]], keep[[1, 2, 4]])
    p2 = keep.clone()
    y2 = m.ssd_linattn_step(q.contiguous(), k.contiguous(), v.contiguous(), up(s["decay"]), p2, slots=slots)
    assert torch.equal(y, y2) and torch.equal(pool, p2)
    assert not torch.equal(pool[3], keep[3])


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_then_tokens(dtype):
    """A prompt and its tokens one by one give what the whole gives."""
    s = make(dtype, 2, 90, 4, 2, 32, 48, carry=False)
    q, k, v, dec = (up(s[n]) for n in ("q", "k", "v", "decay"))
    state = m.ssd_linattn_fwd(*(t[:, :77].contiguous() for t in (q, k, v)), dec, scale=0.2)[1]
    ys = [m.ssd_linattn_step(q[:, t], k[:, t], v[:, t], dec, state, scale=0.2) for t in range(77, 90)]
    ry, rf = lo.linattn(d(s["q"]), d(s["k"]), d(s["v"]), d(s["decay"]), 0.2)
    ay, af = lo.linattn(a(s["q"]), a(s["k"]), a(s["v"]), d(s["decay"]), 0.2)
    near(torch.stack(ys, 1), ry[:, 77:], ay[:, 77:], 90, "y")
    near(state, rf, af, 90, "state")


def test_gradients_against_differences():
    """A step along a random direction changes the fp64 loss by the gradients' products."""
    s = make("f32", 1, 80, 2, 1, 12, 20)
    g = m.ssd_linattn_bwd(up(s["q"]), up(s["k"]), up(s["v"]), up(s["decay"]), up(s["dy"]), scale=0.5,
                          init_state=up(s["init"]), d_final=up(s["d_final"]))

    def loss(x):
        y, f = lo.linattn(x["q"], x["k"], x["v"], d(s["decay"]), 0.5, init=x["init"])
        return ((y * d(s["dy"])).sum() + (f * d(s["d_final"])).sum()).item()

    gen = torch.Generator().manual_seed(5)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("init", "dinit_state")):
        x = {n: d(s[n]) for n in ("q", "k", "v", "init")}
        way = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-4
        # the loss is linear in each input alone: the difference has no error but rounding
        diff = (loss(x | {name: x[name] + h * way}) - loss(x | {name: x[name] - h * way})) / (2 * h)
        want = (g[grad].double().cpu() * way).sum().item()
        size = (g[grad].double().cpu() * way).abs().sum().item()
        assert abs(diff - want) <= (16 + 4 * 80) * 2.0 ** -24 * size + 1e-7 * abs(diff) + 1e-6, name


def test_streams_graphs_and_workspaces():
    s = make("bf16", 1, 2000, 2, 2, 64, 64)
    q, k, v, dec, dy = (up(s[n]) for n in ("q", "k", "v", "decay", "dy"))
    init = up(s["init"])
    y0, f0 = m.ssd_linattn_fwd(q, k, v, dec, init_state=init)
    g0 = m.ssd_linattn_bwd(q, k, v, dec, dy, init_state=init)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1, f1 = m.ssd_linattn_fwd(q, k, v, dec, init_state=init)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(f0, f1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, f2 = m.ssd_linattn_fwd(q, k, v, dec, init_state=init)
        g2 = m.ssd_linattn_bwd(q, k, v, dec, dy, init_state=init)
    for i in range(3):
        q.copy_(up(s["q"]) * (i + 1))
        graph.replay()
        y3, _ = m.ssd_linattn_fwd(q, k, v, dec, init_state=init)
        g3 = m.ssd_linattn_bwd(q, k, v, dec, dy, init_state=init)
        torch.cuda.synchronize()
        assert torch.equal(y2, y3) and all(torch.equal(g2[n], g3[n]) for n in g3)
        if i == 0:
            assert torch.equal(y2, y0) and torch.equal(f2, f0) and all(torch.equal(g2[n], g0[n]) for n in g0)


def test_offsets_past_32_bits():
    """Tokens 2^21 elements apart: 2200 of them span 4.6e9 elements; in and against the order of
    memory, and a pool of 4.4e9 entries."""
    L, stride = 2200, 1 << 21
    wide = torch.empty((1, L, stride), dtype=torch.bfloat16, device=DEV)
    s = make("bf16", 1, L, 2, 2, 16, 24)
    at, views = 0, []
    for n in ("q", "k", "v"):
        w = s[n].shape[2] * s[n].shape[3]
        view = wide[..., at:at + w].unflatten(-1, s[n].shape[2:])
        view.copy_(up(s[n]))
        views.append(view)
        at += w
    y = wide[..., at:at + 48].unflatten(-1, (2, 24))
    dec = up(s["decay"])
    for reverse in (False, True):
        m.ssd_linattn_fwd(*views, dec, reverse=reverse, y=y)
        want = m.ssd_linattn_fwd(up(s["q"]), up(s["k"]), up(s["v"]), dec, reverse=reverse)[0]
        assert torch.equal(y, want)
    del wide, views, view, y
    nslots = (1 << 32) // (2 * 128 * 128) + 1000
    pool = torch.empty((nslots, 2, 128, 128), dtype=torch.float32, device=DEV)
    rows = torch.tensor([nslots - 1, 0], dtype=torch.int32, device=DEV)
    s = make("f32", 2, 1, 2, 1, 128, 128)
    pool[rows.long()] = up(s["init"])
    small = up(s["init"]).clone()
    q, k, v = (up(s[n])[:, 0] for n in ("q", "k", "v"))
    a_ = m.ssd_linattn_step(q, k, v, up(s["decay"]), pool, slots=rows)
    b_ = m.ssd_linattn_step(q, k, v, up(s["decay"]), small)
    assert torch.equal(a_, b_) and torch.equal(pool[rows.long()], small)


@pytest.mark.parametrize("dtype", TYPES)
def test_tokens_closer_than_their_rows(dtype):
    """Views whose tokens overlap, or are one and the same, are read as they are."""
    g = torch.Generator().manual_seed(9)
    line = torch.randn(4000, generator=g).to(TYPES[dtype]).to(DEV)
    dec = torch.tensor([-0.1, -0.01], device=DEV)
    for token in (0, 8, 24):
        q, k, v = (torch.as_strided(line, (1, 45, 2, d), (45 * token, token, 900, 1), o)
                   for d, o in ((48, 0), (48, 30), (24, 100)))
        y, f = m.ssd_linattn_fwd(q, k, v, dec)
        y2, f2 = m.ssd_linattn_fwd(q.contiguous(), k.contiguous(), v.contiguous(), dec)
        assert torch.equal(y, y2) and torch.equal(f, f2)


def test_bfloat16_rows_of_one_token_keep_their_precision():
    """One token, no state: y is (q . k) v, rounded once, which is half a step: eps / 2 = 2^-8 of
    the value.  A score in two parts is off by half a step of its remainder, 2^-8 2^-8, before
    that (a score rounded once would be off by another 2^-8)."""
    s = make("bf16", 300, 1, 2, 2, 64, 64, carry=False)
    y, _ = m.ssd_linattn_fwd(up(s["q"]), up(s["k"]), up(s["v"]), up(s["decay"]))
    ref, _ = lo.linattn(d(s["q"]), d(s["k"]), d(s["v"]), d(s["decay"]))
    size, _ = lo.linattn(a(s["q"]), a(s["k"]), a(s["v"]), d(s["decay"]))
    err = (y.double().cpu() - ref).abs()
    # q . k itself is a float32 sum of 64 terms: 80 2^-24 of their sizes
    assert (err <= (2.0 ** -8 + 2.0 ** -15) * ref.abs() + 80 * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b,L,H,G,K,V", [(40, 70, 16, 16, 24, 24), (1, 900, 2, 2, 40, 40), (1, 900, 4, 2, 24, 100)])
def test_gradient_of_the_state_in_place(dtype, b, L, H, G, K, V):
    """dinit_state written over d_final, in whole sequences and spans, passes together and apart."""
    s = make(dtype, b, L, H, G, K, V)
    q, k, v, dec, dy, init = (up(s[n]) for n in ("q", "k", "v", "decay", "dy", "init"))
    want = m.ssd_linattn_bwd(q, k, v, dec, dy, scale=0.5, init_state=init, d_final=up(s["d_final"]))
    state = up(s["d_final"])
    ly = m._layer
    dims, lay, _, _, _ = ly._linattn_arguments(q, k, v, dec, 0.5, None, None, dy)
    got = {n: torch.empty_like(t) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    keep, *ws = ly._workspace("ssd_linattn_bwd_workspace_bytes", dims, q, None)
    ly._launch("ssd_linattn_bwd", q, dims, lay, q.data_ptr(), k.data_ptr(), v.data_ptr(), dec.data_ptr(),
               init.data_ptr(), None, 0, dy.data_ptr(), state.data_ptr(), got["dq"].data_ptr(),
               got["dk"].data_ptr(), got["dv"].data_ptr(), state.data_ptr(), *ws)
    got["dinit_state"] = state
    assert all(torch.equal(got[n], want[n]) for n in want)
