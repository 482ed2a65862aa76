"""Host-side checks of linear attention and group norm (no GPU): the status of every refused
call, the workspaces, and the binding's argument checks.  Made-up pointers are only passed to
calls that must be refused, and only where no GPU exists."""
import ctypes

import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from mamba_ssd_chunked_02_amd import _layer as ly
from oracle import linattn_ops as lo

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                                  reason="made-up pointers are only passed where no GPU exists")
FAKE = 1 << 20
NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE, OVERLAP = -1, -2, -3, -4, -5, -6, -9


def lin_dims(**kw):
    return m.SsdLinattnDims(**(dict(batch=2, seqlen=8, nheads=4, ngroups=2, keydim=16, valuedim=24, nseq=0,
                                    dtype=1, scale=1.0, reserved=0) | kw))


def gn_dims(**kw):
    return m.SsdGroupnormDims(**(dict(samples=4, positions=5, x_sample=320, x_row=64, y_sample=320, y_row=64,
                                      z_sample=320, z_row=64, dy_sample=320, dy_row=64, channels=64, groups=4,
                                      dtype=1, activation=2, eps=1e-5, reserved=0) | kw))


ARGS = {
    "ssd_linattn_fwd": "layout q k v decay init cu reverse y final ws wsb",
    "ssd_linattn_bwd": "layout q k v decay init cu reverse dy d_final dq dk dv dinit ws wsb",
    "ssd_linattn_step": "layout q k v decay state slots nslots y new_state",
    "ssd_groupnorm_fwd": "x weight bias z y mean rstd ws wsb",
    "ssd_groupnorm_bwd": "x weight bias z mean rstd dy dx dz dweight dbias ws wsb",
}
ABSENT = {"layout": None, "init": None, "cu": None, "d_final": None, "slots": None, "nslots": 4,
          "reverse": 0, "wsb": 1 << 40}


def call(name, dims, **kw):
    args = []
    for i, a in enumerate(ARGS[name].split()):
        args.append(kw.pop(a) if a in kw else ABSENT.get(a, FAKE + (i << 24)))
    assert not kw, kw
    return ly._entry(name)(dims, *args, None)


def lay(**kw):
    dense = dict(q_token=64, q_head=16, k_token=32, k_group=16, v_token=48, v_group=24, y_token=96, y_head=24,
                 dy_token=96, dy_head=24, dq_token=64, dq_head=16, dk_token=32, dk_group=16, dv_token=48,
                 dv_group=24)
    return m.SsdLinattnLayout(**(dense | kw))


@needs_no_gpu
def test_linattn_refusals():
    for f in ("ssd_linattn_fwd", "ssd_linattn_bwd"):
        assert call(f, None) == NULL
        assert call(f, lin_dims(dtype=2)) == DTYPE
        for bad in (dict(batch=0), dict(seqlen=-1), dict(nheads=0), dict(ngroups=0), dict(ngroups=3),
                    dict(keydim=0), dict(valuedim=0), dict(reserved=1), dict(nseq=-1), dict(nseq=2),
                    dict(scale=float("nan")), dict(batch=4, seqlen=1 << 30),
                    dict(batch=1 << 20, nheads=4, ngroups=4)):
            assert call(f, lin_dims(**bad)) == SHAPE, bad
        assert call(f, lin_dims(keydim=257)) == UNSUPPORTED
        assert call(f, lin_dims(valuedim=257)) == UNSUPPORTED
        assert call(f, lin_dims(batch=1, nseq=2)) == NULL        # without cu_seqlens
        assert call(f, lin_dims(batch=1), cu=FAKE) == SHAPE      # cu_seqlens without nseq
        for n in ("q_token", "k_group", "v_token", "y_head", "dy_token", "dq_head"):
            assert call(f, lin_dims(), layout=lay(**{n: -1})) == SHAPE
            assert call(f, lin_dims(), layout=lay(**{n: (1 << 24) + 1})) == SHAPE
        for a in ("q", "k", "v", "decay"):
            assert call(f, lin_dims(), **{a: None}) == NULL
        for a in ("q", "k", "v"):
            assert call(f, lin_dims(), **{a: FAKE + 1}) == ALIGN
        assert call(f, lin_dims(), decay=FAKE + 2) == ALIGN
        assert call(f, lin_dims(), init=FAKE + 2) == ALIGN
        assert call(f, lin_dims(), ws=FAKE + 16) == ALIGN
    assert call("ssd_linattn_fwd", lin_dims(), y=None) == NULL
    assert call("ssd_linattn_fwd", lin_dims(), layout=lay(y_head=23)) == SHAPE      # rows that share elements
    assert call("ssd_linattn_fwd", lin_dims(), layout=lay(y_token=0)) == SHAPE
    assert call("ssd_linattn_fwd", lin_dims(), init=FAKE, final=FAKE + 4) == OVERLAP
    for a in ("dy", "dq", "dk", "dv"):
        assert call("ssd_linattn_bwd", lin_dims(), **{a: None}) == NULL
    for n in ("dq_token", "dk_group", "dv_token"):
        assert call("ssd_linattn_bwd", lin_dims(), layout=lay(**{n: 8})) == SHAPE
    assert call("ssd_linattn_bwd", lin_dims(), d_final=FAKE, dinit=FAKE + 4) == OVERLAP
    assert call("ssd_linattn_bwd", lin_dims(), init=FAKE, dinit=FAKE) == OVERLAP
    assert call("ssd_linattn_bwd", lin_dims(), ws=None) == WORKSPACE                # shared heads
    long = lin_dims(batch=1, seqlen=65536)
    assert call("ssd_linattn_fwd", long, ws=None) == WORKSPACE
    assert call("ssd_linattn_fwd", long, wsb=256) == WORKSPACE


@needs_no_gpu
def test_linattn_step_refusals():
    step = lambda **kw: lin_dims(**({"batch": 4, "seqlen": 1} | kw))
    f = "ssd_linattn_step"
    assert call(f, None) == NULL
    assert call(f, step(dtype=7)) == DTYPE
    for bad in (dict(seqlen=2), dict(nseq=1), dict(batch=-1), dict(ngroups=3), dict(keydim=0),
                dict(scale=float("nan")), dict(reserved=1)):
        assert call(f, step(**bad)) == SHAPE, bad
    assert call(f, step(keydim=257)) == UNSUPPORTED
    assert call(f, step(), nslots=3) == SHAPE
    assert call(f, step(), nslots=-1, slots=FAKE) == SHAPE
    assert call(f, step(), layout=lay(y_head=23)) == SHAPE
    for a in ("q", "k", "v", "decay", "y", "state", "new_state"):
        assert call(f, step(), **{a: None}) == NULL
    assert call(f, step(), v=FAKE + 1) == ALIGN
    assert call(f, step(), state=FAKE, new_state=FAKE + 4) == OVERLAP
    assert call(f, step(batch=0), nslots=0, q=None) == 0


@needs_no_gpu
def test_groupnorm_refusals():
    for f in ("ssd_groupnorm_fwd", "ssd_groupnorm_bwd"):
        assert call(f, None) == NULL
        assert call(f, gn_dims(dtype=3)) == DTYPE
        for bad in (dict(samples=-1), dict(positions=0), dict(groups=0), dict(groups=5), dict(channels=0),
                    dict(eps=-1.0), dict(eps=float("nan")), dict(x_row=63), dict(z_row=0), dict(dy_row=1 << 25),
                    dict(x_sample=-1), dict(samples=1 << 30, positions=4), dict(y_sample=64), dict(y_sample=0)):
            assert call(f, gn_dims(**bad)) == SHAPE, bad
        for a in (-1, 3):
            assert call(f, gn_dims(activation=a)) == UNSUPPORTED
        assert call(f, gn_dims(), x=None) == NULL
        assert call(f, gn_dims(), z=None) == NULL
        for a in ("x", "z"):
            assert call(f, gn_dims(), **{a: FAKE + 1}) == ALIGN
        for a in ("weight", "bias", "mean", "rstd"):
            assert call(f, gn_dims(), **{a: FAKE + 2}) == ALIGN
        assert call(f, gn_dims(), ws=FAKE + 8) == ALIGN
        assert call(f, gn_dims(), ws=None) == WORKSPACE
        assert call(f, gn_dims(), wsb=64) == WORKSPACE
    assert call("ssd_groupnorm_fwd", gn_dims(), y=None) == NULL
    for a in ("mean", "rstd", "dy", "dx", "dz"):
        assert call("ssd_groupnorm_bwd", gn_dims(), **{a: None}) == NULL
    assert call("ssd_groupnorm_bwd", gn_dims(z_sample=0)) == SHAPE   # dz is laid out like z
    assert call("ssd_groupnorm_fwd", gn_dims(samples=0), x=None, y=None) == 0


def test_workspaces():
    need = lambda name, dims: ly._entry(name)(ctypes.byref(dims))
    fwd, bwd = "ssd_linattn_fwd_workspace_bytes", "ssd_linattn_bwd_workspace_bytes"
    assert need(fwd, lin_dims(batch=64, nheads=16)) == 0                      # whole sequences fill the chip
    assert need(fwd, lin_dims(batch=1, seqlen=100)) == 0                      # one span
    assert need(fwd, lin_dims(batch=1, seqlen=0)) == 0
    assert need(fwd, lin_dims(batch=1, seqlen=65536)) % 256 == 0
    assert 0 < need(fwd, lin_dims(batch=1, seqlen=65536)) < 1 << 27
    assert need(fwd, lin_dims(batch=1, seqlen=65536, nseq=5)) >= need(fwd, lin_dims(batch=1, seqlen=65536))
    assert need(fwd, lin_dims(keydim=300)) == 0 and need(bwd, lin_dims(dtype=4)) == 0
    assert need(bwd, lin_dims()) >= 2 * 8 * 4 * 24 * 4                        # shares of the heads
    assert need(bwd, lin_dims(batch=64, nheads=16, ngroups=16)) == 0
    gf, gb = "ssd_groupnorm_fwd_workspace_bytes", "ssd_groupnorm_bwd_workspace_bytes"
    assert need(gf, gn_dims(positions=1)) == 0 and need(gb, gn_dims(positions=1)) > 0
    assert need(gf, gn_dims()) > 0 and need(gb, gn_dims()) > 0 and need(gf, gn_dims(groups=3)) == 0
    assert need(gf, gn_dims(samples=0)) > 0 and need(gb, gn_dims(samples=0, positions=1)) > 0


def test_binding_refuses_mismatches():
    z = torch.zeros
    q, k, v, dec = z(2, 8, 4, 16), z(2, 8, 2, 16), z(2, 8, 2, 24), z(4)
    x, i32 = z(3, 5, 12), torch.int32
    cases = [
        lambda: m.ssd_linattn_fwd(q[0], k, v, dec),
        lambda: m.ssd_linattn_fwd(q, k, v, z(3)),
        lambda: m.ssd_linattn_fwd(q, k, v, dec.double()),
        lambda: m.ssd_linattn_fwd(q, z(2, 8, 2, 15), v, dec),
        lambda: m.ssd_linattn_fwd(q, z(2, 8, 3, 16), z(2, 8, 3, 24), dec),
        lambda: m.ssd_linattn_fwd(q, k, v.bfloat16(), dec),
        lambda: m.ssd_linattn_fwd(q, k, v, dec, init_state=z(2, 4, 16, 23)),
        lambda: m.ssd_linattn_fwd(q, k, v, dec, final_state=z(3, 4, 16, 24)),
        lambda: m.ssd_linattn_fwd(q, k, v, dec, y=z(2, 8, 4, 16)),
        lambda: m.ssd_linattn_fwd(q, k, v, dec, cu_seqlens=z(3, dtype=i32)),          # b is 2
        lambda: m.ssd_linattn_fwd(q.transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1), dec),
        lambda: m.ssd_linattn_fwd(q.transpose(2, 3), k, v, dec),
        lambda: m.ssd_linattn_bwd(q, k, v, dec, z(2, 8, 4, 16)),
        lambda: m.ssd_linattn_bwd(q, k, v, dec, z(2, 8, 4, 24), d_final=z(2, 4, 24, 16)),
        lambda: m.ssd_linattn_step(q[:, 0], k[:, 0], v[:, 0], dec, z(1, 4, 16, 24)),  # 2 rows
        lambda: m.ssd_linattn_step(q[:, 0], k[:, 0], v[:, 0], dec, z(2, 4, 24, 16)),
        lambda: m.ssd_linattn_step(q[:, 0], k[:, 0], v[:, 0], dec, z(2, 4, 16, 24), slots=z(2)),
        lambda: m.ssd_groupnorm_fwd(x, 5),
        lambda: m.ssd_groupnorm_fwd(x, 0),
        lambda: m.ssd_groupnorm_fwd(x[0, 0], 3),
        lambda: m.ssd_groupnorm_fwd(x, 3, weight=z(11)),
        lambda: m.ssd_groupnorm_fwd(x, 3, activation="gelu"),
        lambda: m.ssd_groupnorm_fwd(x, 3, activation="silu", z=x),
        lambda: m.ssd_groupnorm_fwd(x, 3, z=x[:2]),
        lambda: m.ssd_groupnorm_fwd(x, 3, y=x.bfloat16()),
        lambda: m.ssd_groupnorm_fwd(x.transpose(1, 2), 5),
        lambda: m.ssd_groupnorm_bwd(x, 3, None, None, z(3, 4), z(3, 3), x),
        lambda: m.ssd_groupnorm_bwd(x, 3, None, None, z(3, 3), z(3, 3), x[:, :4]),
    ]
    for i, c in enumerate(cases):
        with pytest.raises((ValueError, RuntimeError)):
            print(i, c())
    with pytest.raises(TypeError):
        m.ssd_groupnorm_fwd(x.double(), 3)
    with pytest.raises(TypeError):
        m.ssd_linattn_fwd(q.double(), k.double(), v.double(), dec)
    for c in (lambda: m.ssd_linattn_fwd(q, k, v, dec), lambda: m.ssd_groupnorm_fwd(x, 3)):
        with pytest.raises(ValueError, match="GPU"):
            c()


def test_oracle_quadratic_form():
    """The recurrence against the sum over all pairs of tokens, forward and reversed."""
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    q, k, v, dec = r(1, 9, 2, 3), r(1, 9, 1, 3), r(1, 9, 1, 4), -torch.rand(2, generator=g, dtype=torch.float64)
    init = r(2, 2, 3, 4)
    cu = [0, 4, 9]
    for reverse in (False, True):
        y, final = lo.linattn(q, k, v, dec, 0.7, init, cu, reverse)
        for i, (a, b) in enumerate(((0, 4), (4, 9))):
            order = list(range(a, b))[::-1] if reverse else list(range(a, b))
            for h in range(2):
                for n, t in enumerate(order):
                    want = torch.exp((n + 1) * dec[h]) * q[0, t, h] @ init[i, h]
                    for p, u in enumerate(order[:n + 1]):
                        want = want + torch.exp((n - p) * dec[h]) * (q[0, t, h] @ k[0, u, 0]) * v[0, u, 0]
                    assert torch.allclose(y[0, t, h], 0.7 * want, rtol=1e-12)
                want = torch.exp((b - a) * dec[h]) * init[i, h]
                for p, u in enumerate(order):
                    want = want + torch.exp((b - a - 1 - p) * dec[h]) * torch.outer(k[0, u, 0], v[0, u, 0])
                assert torch.allclose(final[i, h], want, rtol=1e-12)


def test_oracle_groupnorm_is_torchs():
    x = torch.randn(3, 5, 7, 12, dtype=torch.float64)
    w, b = torch.randn(2, 12, dtype=torch.float64)
    y, _, _ = lo.groupnorm(x, 4, w, b)
    want = torch.nn.functional.group_norm(x.movedim(-1, 1), 4, w, b).movedim(1, -1)
    assert torch.allclose(y, want, rtol=1e-10)
