"""Host-side checks of the operators around the scan (no GPU): the status of
every refused call, planning of the workspaces, and the binding's argument
checks.  Made-up pointers are only passed to calls that must be refused, and
only where no GPU exists."""
import ctypes

import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from mamba_ssd_chunked_02_amd import _layer as ly

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                                  reason="made-up pointers are only passed where no GPU exists")
FAKE = 1 << 20
NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, WORKSPACE, OVERLAP = -1, -2, -3, -4, -5, -6, -9


def norm_dims(**kw):
    a = dict(rows=8, x_row=64, y_row=64, dy_row=64, width=64, dtype=1, eps=1e-5, reserved=0) | kw
    return m.SsdNormDims(**a)


def conv_dims(**kw):
    return m.SsdConvDims(**(dict(batch=2, seqlen=8, channels=64, width=4, nseq=0, dtype=1) | kw))


def scan_dims(**kw):
    return m.SsdSelscanDims(**(dict(batch=2, seqlen=8, channels=64, d_state=16, ngroups=1, nseq=0,
                                    dtype=1, reserved=0) | kw))


ARGS = {
    "ssd_norm_fwd": "x weight bias y mean rstd",
    "ssd_norm_bwd": "x weight mean rstd dy dx dweight dbias ws wsb",
    "ssd_conv_fwd": "layout x weight bias init cu y final",
    "ssd_conv_bwd": "layout x weight bias init cu dy d_final dx dweight dbias dinit ws wsb",
    "ssd_conv_step": "layout x weight bias state slots nslots y new_state",
    "ssd_selscan_fwd": "layout x d_raw d_init A B C D z init cu y final ws wsb",
    "ssd_selscan_bwd": "layout x d_raw d_init A B C D z init cu dy d_final dx dd_raw dB dC dz dA dD "
                       "dd_init dinit ws wsb",
    "ssd_selscan_step": "layout x d_raw d_init A B C D z state slots nslots y new_state",
    "ssd_step": "layout x d_raw d_init B C state slots nslots y new_state",
}
ABSENT = {"layout": None, "init": None, "cu": None, "d_final": None, "slots": None, "nslots": 4,
          "wsb": 1 << 40}


def call(name, dims, **kw):
    """Every pointer made up and apart, unless given."""
    args = []
    for i, a in enumerate(ARGS[name].split()):
        v = kw.pop(a) if a in kw else ABSENT.get(a, FAKE + (i << 24))
        if name == "ssd_step" and a == "d_init":
            v = -4.6
        args.append(v)
    assert not kw, kw
    return ly._entry(name)(dims, *args, None)


@needs_no_gpu
def test_norm_refusals():
    for f in ("ssd_norm_fwd", "ssd_norm_bwd"):
        assert call(f, None) == NULL
        assert call(f, norm_dims(dtype=2)) == DTYPE
        assert call(f, norm_dims(rows=-1)) == SHAPE
        assert call(f, norm_dims(rows=1 << 31)) == SHAPE
        assert call(f, norm_dims(width=0)) == SHAPE
        assert call(f, norm_dims(x_row=63)) == SHAPE
        assert call(f, norm_dims(x_row=(1 << 24) + 1)) == SHAPE
        assert call(f, norm_dims(eps=-1.0)) == SHAPE
        assert call(f, norm_dims(eps=float("nan"))) == SHAPE
        w = 16385
        assert call(f, norm_dims(width=w, x_row=w, y_row=w, dy_row=w)) == UNSUPPORTED
        assert call(f, norm_dims(), x=None) == NULL
        assert call(f, norm_dims(), x=FAKE + 1) == ALIGN
        assert call(f, norm_dims(), weight=FAKE + 2) == ALIGN
    assert call("ssd_norm_fwd", norm_dims(), y=None) == NULL
    for a in ("mean", "rstd", "dy", "dx"):
        assert call("ssd_norm_bwd", norm_dims(), **{a: None}) == NULL
    assert call("ssd_norm_bwd", norm_dims(), ws=None) == WORKSPACE
    assert call("ssd_norm_bwd", norm_dims(), wsb=64) == WORKSPACE
    assert call("ssd_norm_bwd", norm_dims(), ws=FAKE + 16) == ALIGN
    assert call("ssd_norm_fwd", norm_dims(rows=0), x=None, y=None) == 0  # nothing to do


@needs_no_gpu
def test_conv_refusals():
    for f in ("ssd_conv_fwd", "ssd_conv_bwd"):
        assert call(f, None) == NULL
        assert call(f, conv_dims(dtype=-1)) == DTYPE
        assert call(f, conv_dims(batch=0)) == SHAPE
        assert call(f, conv_dims(seqlen=-1)) == SHAPE
        assert call(f, conv_dims(batch=4, seqlen=1 << 30)) == SHAPE
        assert call(f, conv_dims(channels=0)) == SHAPE
        assert call(f, conv_dims(nseq=2)) == SHAPE               # packed needs batch 1
        assert call(f, conv_dims(batch=1, nseq=2)) == NULL       # without cu_seqlens
        assert call(f, conv_dims(batch=1), cu=FAKE) == SHAPE     # cu_seqlens without nseq
        for w in (0, 1, 5):
            assert call(f, conv_dims(width=w)) == UNSUPPORTED
        assert call(f, conv_dims(), layout=m.SsdConvLayout(63, 64, 64)) == SHAPE
        assert call(f, conv_dims(), layout=m.SsdConvLayout((1 << 24) + 1, 64, 64)) == SHAPE
        assert call(f, conv_dims(), x=None) == NULL
        assert call(f, conv_dims(), weight=None) == NULL
        assert call(f, conv_dims(), x=FAKE + 1) == ALIGN
        assert call(f, conv_dims(), bias=FAKE + 2) == ALIGN
    assert call("ssd_conv_fwd", conv_dims(), layout=m.SsdConvLayout(64, 63, 64)) == SHAPE
    assert call("ssd_conv_bwd", conv_dims(), layout=m.SsdConvLayout(64, 64, 63)) == SHAPE
    assert call("ssd_conv_fwd", conv_dims(), init=FAKE, final=FAKE) == OVERLAP
    assert call("ssd_conv_fwd", conv_dims(), init=FAKE, final=FAKE + 2) == OVERLAP
    assert call("ssd_conv_bwd", conv_dims(), d_final=FAKE, dinit=FAKE + 128) == OVERLAP
    assert call("ssd_conv_bwd", conv_dims(), ws=None) == WORKSPACE
    assert call("ssd_conv_bwd", conv_dims(), wsb=16) == WORKSPACE
    step = lambda **kw: conv_dims(**({"batch": 4, "seqlen": 1} | kw))
    assert call("ssd_conv_step", step(seqlen=2)) == SHAPE
    assert call("ssd_conv_step", step(), nslots=3) == SHAPE      # no slots: a row for each
    assert call("ssd_conv_step", step(), nslots=-1, slots=FAKE) == SHAPE
    assert call("ssd_conv_step", step(width=5)) == UNSUPPORTED
    assert call("ssd_conv_step", step(), state=None) == NULL
    assert call("ssd_conv_step", step(), state=FAKE, new_state=FAKE + 64) == OVERLAP


@needs_no_gpu
def test_selscan_refusals():
    for f in ("ssd_selscan_fwd", "ssd_selscan_bwd"):
        assert call(f, None) == NULL
        assert call(f, scan_dims(dtype=3)) == DTYPE
        assert call(f, scan_dims(channels=63, ngroups=2)) == SHAPE
        assert call(f, scan_dims(channels=(1 << 20) + 1)) == SHAPE
        assert call(f, scan_dims(d_state=0)) == SHAPE
        assert call(f, scan_dims(d_state=65)) == UNSUPPORTED
        assert call(f, scan_dims(nseq=1)) == SHAPE
        assert call(f, scan_dims(batch=1, nseq=1)) == NULL
        assert call(f, scan_dims(batch=1), cu=FAKE) == SHAPE
        lay = [64, 64, 64, 16, 16, 16, 16, 64, 64]
        for i in (0, 1, 2):
            assert call(f, scan_dims(), layout=m.SsdSelscanLayout(*lay[:i], 63, *lay[i + 1:])) == SHAPE
        for i in (3, 4, 5, 6):
            assert call(f, scan_dims(), layout=m.SsdSelscanLayout(*lay[:i], -1, *lay[i + 1:])) == SHAPE
        for a in ("x", "d_raw", "d_init", "A", "B", "C"):
            assert call(f, scan_dims(), **{a: None}) == NULL
        for a in ("x", "d_raw", "B", "C", "z"):
            assert call(f, scan_dims(), **{a: FAKE + 1}) == ALIGN
        for a in ("d_init", "A", "D", "init"):
            assert call(f, scan_dims(), **{a: FAKE + 2}) == ALIGN
    assert call("ssd_selscan_fwd", scan_dims(), y=None) == NULL
    assert call("ssd_selscan_fwd", scan_dims(), init=FAKE, final=FAKE + 4) == OVERLAP
    for a in ("dy", "dx", "dd_raw", "dB", "dC", "dz"):
        assert call("ssd_selscan_bwd", scan_dims(), **{a: None}) == NULL
    assert call("ssd_selscan_bwd", scan_dims(), d_final=FAKE, dinit=FAKE) == OVERLAP
    assert call("ssd_selscan_bwd", scan_dims(), ws=None) == WORKSPACE
    assert call("ssd_selscan_bwd", scan_dims(), wsb=256) == WORKSPACE
    step = lambda **kw: scan_dims(**({"batch": 4, "seqlen": 1} | kw))
    assert call("ssd_selscan_step", step(seqlen=2)) == SHAPE
    assert call("ssd_selscan_step", step(), nslots=3) == SHAPE
    assert call("ssd_selscan_step", step(d_state=65)) == UNSUPPORTED
    assert call("ssd_selscan_step", step(), A=None) == NULL
    assert call("ssd_selscan_step", step(), state=FAKE, new_state=FAKE + 4) == OVERLAP


@needs_no_gpu
def test_ssd_step_refusals():
    d = lambda *a, **kw: m.make_dims(*(a or (4, 1, 8, 64, 128)), **kw)
    assert call("ssd_step", None) == NULL
    assert call("ssd_step", d(dtype=5)) == DTYPE
    assert call("ssd_step", d(4, 2, 8, 64, 128)) == SHAPE
    assert call("ssd_step", d(4, 1, 8, 24, 128)) == SHAPE
    assert call("ssd_step", d(4, 1, 8, 528, 128)) == SHAPE
    assert call("ssd_step", d(4, 1, 8, 64, 128, ngroups=3)) == SHAPE
    assert call("ssd_step", d(4, 1, 8, 64, 48)) == UNSUPPORTED
    assert call("ssd_step", d(), nslots=3) == SHAPE
    assert call("ssd_step", d(), x=None) == NULL
    assert call("ssd_step", d(), new_state=None) == NULL
    assert call("ssd_step", d(), B=FAKE + 1) == ALIGN
    assert call("ssd_step", d(), state=FAKE, new_state=FAKE + 4) == OVERLAP
    lay = m.SsdLayout()
    lay.x_token = -1
    assert call("ssd_step", d(), layout=lay) == SHAPE


def test_workspaces_are_planned_from_the_sizes():
    need = lambda name, dims: ly._entry(name)(ctypes.byref(dims))
    for name, dims in (("ssd_norm_bwd_workspace_bytes", norm_dims()),
                       ("ssd_conv_bwd_workspace_bytes", conv_dims()),
                       ("ssd_selscan_bwd_workspace_bytes", scan_dims())):
        n = need(name, dims)
        assert n > 0 and n % 256 == 0 and n == need(name, dims)
    assert need("ssd_norm_bwd_workspace_bytes", norm_dims(width=0)) == 0
    assert need("ssd_conv_bwd_workspace_bytes", conv_dims(width=9)) == 0
    assert need("ssd_selscan_bwd_workspace_bytes", scan_dims(d_state=65)) == 0
    # weight gradients: at most one row of partial sums for every four rows
    big = norm_dims(rows=1 << 20)
    assert need("ssd_norm_bwd_workspace_bytes", big) <= 2048 * 2 * 64 * 4


@needs_no_gpu
def test_selscan_cuts_long_sequences_of_few_channels():
    """Spans (and a workspace for their states) only where whole sequences would
    leave most of the chip idle."""
    need = lambda **kw: ly._entry("ssd_selscan_fwd_workspace_bytes")(ctypes.byref(scan_dims(**kw)))
    assert need(batch=1, seqlen=65536, channels=64) > 0
    assert need(batch=1, seqlen=65536, channels=64, nseq=3) > 0
    assert need(batch=1, seqlen=256, channels=64) == 0       # one segment
    assert need(batch=8, seqlen=4096, channels=4096) == 0    # whole sequences fill the chip
    assert need(batch=1, seqlen=0, channels=64) == 0
    d = scan_dims(batch=1, seqlen=65536, channels=64)
    assert call("ssd_selscan_fwd", d, ws=None) == WORKSPACE
    assert call("ssd_selscan_fwd", d, wsb=256) == WORKSPACE
    assert call("ssd_selscan_fwd", d, ws=FAKE + 16) == ALIGN


def test_binding_refuses_mismatches():
    f, b = torch.float32, torch.bfloat16
    x = torch.zeros(2, 8, 16)
    w = torch.zeros(4, 16)
    cases = [
        lambda: m.ssd_norm_fwd(x, weight=torch.zeros(15)),
        lambda: m.ssd_norm_fwd(x, weight=torch.zeros(16, dtype=b)),
        lambda: m.ssd_norm_fwd(x.transpose(1, 2)[:, :, :8]),
        lambda: m.ssd_norm_bwd(x, None, torch.zeros(2, 8), torch.zeros(2, 8), x.to(b)),
        lambda: m.ssd_conv_fwd(x, torch.zeros(4, 15)),
        lambda: m.ssd_conv_fwd(x[0], w),
        lambda: m.ssd_conv_fwd(x, w, init_state=torch.zeros(2, 2, 16)),
        lambda: m.ssd_conv_fwd(x, w, cu_seqlens=torch.zeros(3, dtype=torch.int32)),   # b is 2
        lambda: m.ssd_conv_fwd(x[:1], w, cu_seqlens=torch.zeros(3, dtype=torch.int64)),
        lambda: m.ssd_conv_fwd(x[:1], w, cu_seqlens=torch.zeros(1, dtype=torch.int32)),
        lambda: m.ssd_conv_fwd(x.transpose(0, 1), w),
        lambda: m.ssd_conv_bwd(x, w, None, x, d_final=torch.zeros(2, 3, 15)),
        lambda: m.ssd_conv_step(x[0], torch.zeros(7, 3, 16), w),                      # 8 rows
        lambda: m.ssd_conv_step(x[0], torch.zeros(8, 3, 16, dtype=b), w),
        lambda: m.ssd_conv_step(x[0], torch.zeros(8, 3, 16), w, slots=torch.zeros(8)),
        lambda: m.ssd_conv_step(x[0], torch.zeros(8, 3, 16), w, new_state=torch.zeros(9, 3, 16)),
        lambda: m.ssd_selscan_fwd(x, x, torch.zeros(16), torch.zeros(4, 15), x[..., None], x[..., None]),
        lambda: m.ssd_selscan_step(x[0], x[0], torch.zeros(16), torch.zeros(4, 16),
                                   torch.zeros(8, 1, 5), torch.zeros(8, 1, 4), torch.zeros(8, 4, 16)),
        lambda: m.ssd_step(torch.zeros(2, 4, 16), torch.zeros(2, 3), -1.0, torch.zeros(2, 1, 16),
                           torch.zeros(2, 1, 16), torch.zeros(2, 4, 16, 16)),
    ]
    for i, c in enumerate(cases):
        with pytest.raises((ValueError, RuntimeError)):
            print(i, c())
    with pytest.raises(TypeError):
        m.ssd_norm_fwd(x.double())
    # right arguments, wrong place
    for c in (lambda: m.ssd_norm_fwd(x), lambda: m.ssd_conv_fwd(x, w)):
        with pytest.raises(ValueError, match="GPU"):
            c()
