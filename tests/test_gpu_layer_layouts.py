"""Layouts of the operators around the scan on the GPU: gradients of inputs that are
expanded views.  Tolerances as test_gpu_layer's."""
import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from oracle import layer_ops as lo
from test_gpu_layer import TYPES, Source, dd, scan_call, scan_problem, up, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", [(2, 70, 40, 16, 2, None), (3, 1, 36, 8, 3, None),
                                  (1, 90, 24, 16, 2, [0, 40, 41, 90])], ids=str)
@pytest.mark.parametrize("over", ["groups", "tokens", "batch"])
def test_selscan_bwd_of_expanded_inputs(dtype, case, over):
    """dB and dC of B and C that are expanded over groups, over all tokens or over the
    batch: every group and token has its own, as with dense copies of the same values."""
    b, L, E, N, G, cu = case
    p, (dy, df), _ = scan_problem(dtype, case)
    first = {"groups": (slice(None), slice(None), slice(0, 1)),
             "tokens": (slice(0, 1), slice(0, 1)), "batch": (slice(0, 1),)}[over]
    small = {k: p[k][first] for k in "BC"}
    p |= {k: small[k].expand(b, L, G, N).contiguous() for k in "BC"}
    args, kw = scan_call(p, cu)
    want = m.ssd_selscan_bwd(*args, up(dy), **kw, d_final=up(df))
    views = [up(small[k]).expand(b, L, G, N) for k in "BC"]
    got = m.ssd_selscan_bwd(*args[:4], *views, up(dy), **kw, d_final=up(df))
    assert got.keys() == want.keys() and all(torch.equal(got[k], want[k]) for k in want)
    rg = lo.gradients(lambda **k: lo.selscan(**k, cu=cu), {k: dd(v) for k, v in p.items()},
                      [dd(dy), dd(df)])
    K = 4 * (64 + 4 * b * L) + 4 * E
    for k in "BC":
        within(got["d" + k], rg[k], K, "d" + k)


@pytest.mark.parametrize("name,dim", [("B", 2), ("C", 2), ("B", 1), ("C", 0), ("x", 2), ("d_raw", 2)])
def test_ssd_bwd_of_expanded_inputs(name, dim):
    """The SSD scan's gradients of expanded views, as with dense copies."""
    s = Source(31, "bf16")
    b, L, H, P, G, N = 2, 130, 4, 32, 2, 32
    ins = {"x": s(b, L, H, P), "d_raw": s(b, L, H), "B": s(b, L, G, N), "C": s(b, L, G, N)}
    small = ins[name].narrow(dim, 0, 1)
    ins[name] = small.expand_as(ins[name]).contiguous()
    dy, ins = up(s(b, L, H, P)), {k: up(v) for k, v in ins.items()}

    def grads(x, d_raw, B, C):
        return m.ssd_bwd(x, d_raw, -2.0, B, C, None, dy)

    want = grads(**ins)
    got = grads(**(ins | {name: up(small).expand_as(ins[name])}))
    assert got.keys() == want.keys() and all(torch.equal(got[k], want[k]) for k in want)
