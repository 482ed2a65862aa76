"""The retention layer of the examples: linear attention, group norm and layer norm together,
as a program uses them.  It runs, its gradients are those of the same layer written in fp64,
and serving token by token agrees with one packed pass."""
import importlib.util
import os

import pytest
import torch

from oracle import layer_ops, linattn_ops

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "retention_layer.py")


def load():
    spec = importlib.util.spec_from_file_location("retention_layer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_runs_and_serves(dtype):
    """Both ways of serving take about ten roundings (norm, two projections, attention, head norm,
    sum), each half a step of a value of the output's size, and a head norm divides by a
    deviation that may be a fourth of that: 10 x 4 steps, and as much again for float32's sums."""
    losses, worst = load().main(["--width", "64", "--tokens", "75", "--dtype", dtype])
    assert all(v == v and v < 1e3 for v in losses)
    assert worst <= {"f32": 80 * 2.0 ** -24 * 64, "bf16": 40 * 2.0 ** -8}[dtype], worst


@pytest.mark.parametrize("packed", [False, True])
def test_gradients(packed):
    mod = load()
    layer = mod.Layer(32, heads=2, dtype=torch.float32)
    g = torch.Generator().manual_seed(4)
    b, L = (1, 90) if packed else (2, 45)
    cu = [0, 40, 41, 90] if packed else None
    x, dy = torch.randn((b, L, 32), generator=g), torch.randn((b, L, 32), generator=g)
    leaves = {"x": x.cuda().requires_grad_()} | {n: t.requires_grad_() for n, t in layer.params.items()}
    out = layer(leaves["x"], None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"))
    got = dict(zip(leaves, torch.autograd.grad((out * dy.cuda()).sum(), list(leaves.values()))))

    ref = {n: t.detach().cpu().double().requires_grad_() for n, t in leaves.items()}
    h, _, _ = layer_ops.norm(ref["x"], ref["norm_w"], ref["norm_b"], 1e-5)
    q, k, v, z = (h @ ref["w_in"]).split(layer.parts, dim=-1)
    H = layer.heads
    y, _ = linattn_ops.linattn(q.unflatten(-1, (H, -1)), k.unflatten(-1, (H, -1)), v.unflatten(-1, (H, -1)),
                               layer.decay.cpu().double(), layer.scale, cu=cu)
    y = linattn_ops.groupnorm(y.reshape(b * L, -1), H, ref["head_w"], ref["head_b"], z.reshape(b * L, -1))[0]
    full = ref["x"] + (y @ ref["w_out"]).view(b, L, -1)
    assert (out.double().cpu() - full).abs().max() <= 1e-4 * full.abs().max()
    want = torch.autograd.grad((full * dy.double()).sum(), list(ref.values()))
    for (n, a), w in zip(got.items(), want):
        # float32 throughout: some hundred roundings of terms that a norm's division by the
        # deviations of its head (at least 1e-2 here) may enlarge: 128 2^-24 100 = 8e-4
        assert (a.double().cpu() - w).norm() <= 8e-4 * w.norm(), n
