"""Layouts the operators take or refuse (no GPU): rows that share elements, strides of
dimensions of size 1, workspaces.  Made-up pointers are only
passed where no GPU exists; the binding's calls run with the launch left out."""
import contextlib
import ctypes

import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from mamba_ssd_chunked_02_amd import _layer as ly
from test_abi_host import call as ssd_call
from test_abi_host import call_bwd, lay
from test_layer_host import FAKE, OVERLAP, SHAPE, WORKSPACE, call, needs_no_gpu, scan_dims


@pytest.fixture
def launches(monkeypatch):
    """The entry points' arguments instead of a launch."""
    seen = []
    monkeypatch.setattr(ly, "_launch", lambda name, x, *args: seen.append((name, args)))
    return seen


def scan_inputs(b, L, E, N):
    z = lambda *s: torch.zeros(s)
    return (z(b, L, E), z(b, L, E), z(E), z(N, E))


# ---- gradients of inputs whose rows share elements -----------------------------------------

def shares(T, t, G, g, n):
    """By writing down every element."""
    at = [i * t + j * g + k for i in range(T) for j in range(G) for k in range(n)]
    return len(set(at)) < len(at)


@needs_no_gpu
def test_selscan_bwd_refuses_shared_rows():
    """B and C whose rows share elements are refused where their gradients would be
    written there, whatever way they do; layouts that keep them apart are not."""
    N, seen = 4, set()
    for b, L, G in ((1, 1, 1), (1, 1, 3), (2, 1, 1), (1, 3, 1), (2, 2, 3), (1, 5, 2)):
        for t in (0, 3, 4, 5, 8, 11, 12, 13, 21):
            for g in (0, 2, 4, 5, 9, 16, 20, 24):
                bad = shares(b * L, t, G, g, N)
                seen.add((b * L > 1, G > 1, bad))
                d = scan_dims(batch=b, seqlen=L, ngroups=G, channels=6 * G, d_state=N)
                for lay in ([t, g, G * N, N], [G * N, N, t, g]):
                    full = m.SsdSelscanLayout(*[6 * G] * 3, *lay, *[6 * G] * 2)
                    rc = call("ssd_selscan_bwd", d, layout=full, ws=None)  # else stopped here
                    assert rc == (SHAPE if bad else WORKSPACE), (b, L, G, t, g, rc)
    assert len(seen) == 7  # one row never shares, everything else both does and does not
    # with no tokens nothing is written
    d = scan_dims(seqlen=0, ngroups=2)
    assert call("ssd_selscan_bwd", d, layout=m.SsdSelscanLayout(64, 64, 64, 0, 0, 0, 0, 64, 64),
                ws=None) == WORKSPACE


def test_selscan_bwd_gives_expanded_inputs_dense_gradients(launches):
    """Where B or C is expanded over groups, tokens or the batch, each token and
    group has a gradient of its own; other layouts are kept."""
    b, L, E, N, G = 2, 3, 8, 4, 2
    x, raw, dinit, A = scan_inputs(b, L, E, N)
    dense = torch.zeros(b, L, G, N)
    for B in (torch.zeros(b, L, 1, N).expand(b, L, G, N), torch.zeros(1, 1, G, N).expand(b, L, G, N),
              torch.zeros(1, L, G, N).expand(b, L, G, N),
              torch.zeros(100).as_strided((b, L, G, N), (3 * L, 3, 12, 1))):
        for args in ((B, dense), (dense, B)):
            g = m.ssd_selscan_bwd(x, raw, dinit, A, *args, x)
            for k in ("dB", "dC"):
                assert g[k].shape == dense.shape and g[k].is_contiguous()
            lay = launches.pop()[1][1]
            assert (lay.B_token, lay.B_group, lay.C_token, lay.C_group) == (G * N, N, G * N, N)
    wide = torch.zeros(b, L, 5 + G * N)[..., 5:].unflatten(-1, (G, N))
    swapped = torch.zeros(G, b, L, N).permute(1, 2, 0, 3)
    for B in (wide, swapped):
        g = m.ssd_selscan_bwd(x, raw, dinit, A, B, dense, x)
        assert g["dB"].stride() == B.stride()


@needs_no_gpu
@pytest.mark.parametrize("name,inner,row", [("x", "x_head", 16), ("d_raw", "d_raw_head", 1),
                                            ("B", "B_group", 16), ("C", "C_group", 16)])
def test_ssd_bwd_refuses_shared_rows(name, inner, row):
    """The SSD scan's gradients are laid out like x, d_raw, B and C too."""
    for b, L in ((1, 1), (1, 5), (2, 3)):
        d = m.make_dims(b, L, 2, 16, 16, ngroups=2)
        for t in (0, 8, 16, 24, 32, 40, 48):
            for h in (0, 8, 16, 24, 80, 96):
                l = lay(m, d, **{name + "_token": t, inner: h})
                bad = shares(b * L, t, 2, h, row)
                assert call_bwd(m, d, layout=l, ws=None) == (SHAPE if bad else WORKSPACE), (b, L, t, h)
                assert ssd_call(m, d, layout=l, ws=None) == WORKSPACE  # the forward only reads them
    l = lay(m, m.make_dims(1, 0, 2, 16, 16), **{name + "_token": 0, inner: 0})
    assert call_bwd(m, m.make_dims(1, 0, 2, 16, 16), layout=l, ws=None) == WORKSPACE


def test_ssd_bwd_binding_of_expanded_inputs(monkeypatch):
    """A single call takes dense copies; a prepared one, which may run again after its
    inputs have changed, refuses."""
    import mamba_ssd_chunked_02_amd._binding as bind
    b, L, H, P, G, N = 2, 3, 4, 16, 2, 16
    full = {"x": torch.zeros(b, L, H, P), "d_raw": torch.zeros(b, L, H),
            "B": torch.zeros(b, L, G, N), "C": torch.zeros(b, L, G, N)}
    dy = torch.zeros(b, L, H, P)
    seen = []
    monkeypatch.setattr(bind.PreparedBwd, "run", lambda self: seen.append(self) or self.grads)
    for k, t in full.items():
        for dim in (0, 1, 2):
            ins = full | {k: t.narrow(dim, 0, 1).expand_as(t)}
            with pytest.raises(ValueError, match=k + ".*share"):
                m.prepare_bwd(ins["x"], ins["d_raw"], -1.0, ins["B"], ins["C"], None, dy)
            with monkeypatch.context() as c:
                c.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
                g = m.ssd_bwd(ins["x"], ins["d_raw"], -1.0, ins["B"], ins["C"], None, dy)
            assert g["d" + k].is_contiguous() and g["d" + k].shape == t.shape
    l = seen[-1].layout
    assert (l.B_token, l.B_group, l.C_token, l.C_group) == (G * N, N, G * N, N)


# ---- strides of dimensions of size 1 -------------------------------------------------------

FAR = 1 << 25  # past the largest stride there is


def apart(*shape, **far):
    """A view of this shape whose dimensions dN of size 1 have the stride given: nothing is
    that far apart."""
    stride, step = [], 1
    for n in reversed(shape):
        stride.insert(0, step)
        step *= n
    for k, v in far.items():
        assert shape[int(k[1:])] == 1
        stride[int(k[1:])] = v
    return torch.zeros(max(step, 1)).as_strided(shape, stride)


def padded(*shape):
    """Rows 3 elements further apart than dense ones."""
    return torch.zeros(*shape[:-1], shape[-1] + 3)[..., :shape[-1]]


def strides_passed(launches):
    name, args = launches.pop()
    return [getattr(s, f) for s in args[:2] if isinstance(s, ctypes.Structure) for f, t in s._fields_
            if t is ctypes.c_int64 and f not in ("seqlen", "rows")]


def test_strides_over_one_index_do_not_count(launches):
    """One sequence, one token or one group: torch keeps any stride for such a dimension,
    also one that the library refuses."""
    for E in (8, 1):
        for far in ({"d0": FAR}, {"d1": FAR}, {"d0": FAR, "d1": FAR}, {"d0": 0, "d1": 0}):
            x = apart(1, 1, E, **far)
            m.ssd_conv_fwd(x, torch.zeros(4, E), y=x)
            assert max(strides_passed(launches)) <= E
            m.ssd_norm_fwd(x, y=x)
            assert max(strides_passed(launches)) <= E
            m.ssd_selscan_fwd(x, x, torch.zeros(E), torch.zeros(4, E), apart(1, 1, 1, 4, **far),
                              apart(1, 1, 1, 4, d2=FAR, **far), y=x, z=x)
            assert max(strides_passed(launches)) <= max(E, 4)
            m.ssd_selscan_bwd(x, x, torch.zeros(E), torch.zeros(4, E), apart(1, 1, 1, 4, **far),
                              apart(1, 1, 1, 4, d2=FAR, **far), x, z=x)
            assert max(strides_passed(launches)) <= max(E, 4)
            m.ssd_conv_bwd(x, torch.zeros(4, E), None, x)
            assert max(strides_passed(launches)) <= E
            m.ssd_norm_bwd(x, None, torch.zeros(1, 1), torch.zeros(1, 1), x)
            assert max(strides_passed(launches)) <= E
        for far in (FAR, 0):
            x = apart(1, E, d0=far)
            m.ssd_conv_step(x, torch.zeros(1, 3, E), torch.zeros(4, E), y=x)
            assert max(strides_passed(launches)) <= E
            m.ssd_norm_fwd(x, y=x)
            assert max(strides_passed(launches)) <= E
            m.ssd_selscan_step(x, x, torch.zeros(E), torch.zeros(4, E), apart(1, 1, 4, d0=far, d1=far),
                               apart(1, 1, 4, d0=far), torch.zeros(1, 4, E), y=x, z=x)
            assert max(strides_passed(launches)) <= max(E, 4)
    # a group of its own behind the tokens: [b, 1, L, N] transposed
    B = torch.zeros(1, 1, 5, 4).transpose(1, 2)
    B = B.as_strided(B.shape, (FAR, 4, FAR, 1))
    x = torch.zeros(1, 5, 8)
    m.ssd_selscan_fwd(x, x, torch.zeros(8), torch.zeros(4, 8), B, B)
    assert max(strides_passed(launches)) <= 8
    m.ssd_selscan_fwd(x, x, torch.zeros(8), torch.zeros(4, 8), padded(1, 5, 1, 4), B)
    assert strides_passed(launches)[3:7] == [7, 4, 4, 4]
    for far in (FAR, 0):
        for H in (1, 3):
            x = apart(1, H, 16, d0=far, **({"d1": far} if H == 1 else {}))
            raw = apart(1, H, d0=far, **({"d1": far} if H == 1 else {}))
            B = apart(1, 1, 16, d0=far, d1=far)
            m.ssd_step(x, raw, -1.0, B, B, torch.zeros(1, H, 16, 16), y=x)
            assert max(strides_passed(launches)) <= 16 * H
    # the strides that count are passed on
    m.ssd_step(padded(2, 3, 16), padded(2, 3), -1.0, padded(2, 1, 16), padded(2, 1, 16),
               torch.zeros(2, 3, 16, 16))
    assert strides_passed(launches)[:8] == [57, 19, 6, 1, 19, 16, 19, 16]


# ---- workspaces ----------------------------------------------------------------------------

def workspace_calls():
    x, w = torch.zeros(2, 8, 16), torch.zeros(4, 16)
    long = torch.zeros(1, 4096, 16)  # cut into spans: the forward scan wants a workspace
    B = torch.zeros(1, 4096, 1, 4)
    args = lambda t: (t, t, torch.zeros(16), torch.zeros(4, 16), B[:, :t.shape[1]].expand(len(t), -1, -1, -1),
                      B[:, :t.shape[1]].expand(len(t), -1, -1, -1).contiguous())
    mean = torch.zeros(2, 8)
    return {"norm_bwd": lambda ws: m.ssd_norm_bwd(x, None, mean, mean, x, workspace=ws),
            "conv_bwd": lambda ws: m.ssd_conv_bwd(x, w, None, x, workspace=ws),
            "selscan_fwd": lambda ws: m.ssd_selscan_fwd(*args(long), workspace=ws),
            "selscan_bwd": lambda ws: m.ssd_selscan_bwd(*args(long), long, workspace=ws)}


@pytest.mark.parametrize("name", list(workspace_calls()))
def test_workspaces_hold_the_bytes_that_are_passed(launches, name):
    """A workspace of any type counts its bytes; one elsewhere, or whose elements are not
    all there, is refused before a kernel writes into it."""
    call = workspace_calls()[name]
    call(torch.zeros(1000, dtype=torch.float64))
    assert launches.pop()[1][-1] == 8000
    call(None)
    own = launches.pop()[1][-1]
    assert own > 0
    for bad in (torch.zeros(own, dtype=torch.uint8, device="meta"), torch.zeros(1, dtype=torch.uint8).expand(own),
                torch.zeros(own, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            call(bad)
    assert not launches


# ---- outputs whose rows share elements -----------------------------------------------------

@needs_no_gpu
def test_ssd_step_refuses_shared_rows_of_y():
    """y's strides, which no other tensor's bound, must keep its rows apart; the inputs
    are only read and may share theirs."""
    for b, H in ((1, 1), (1, 3), (4, 1), (4, 3)):
        d = m.make_dims(b, 1, H, 16, 16)
        for t in (0, 8, 15, 16, 32, 48, 64):
            for h in (0, 8, 16, 17, 64, 80):
                l = m.SsdLayout(*[0] * 8, t, h)
                bad = shares(b, t, H, h, 16)
                rc = call("ssd_step", d, layout=l, state=FAKE, new_state=FAKE + 4)  # else stopped here
                assert rc == (SHAPE if bad else OVERLAP), (b, H, t, h, rc)
