"""The example layer: its loss falls, and serving token by token agrees with one
packed pass over the same tokens."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "mamba_layer.py")


@pytest.mark.parametrize("dtype,close", [("f32", 1e-4), ("bf16", 4e-2)])
def test_layer_trains_and_serves(dtype, close):
    """bf16: the output adds about ten roundings of 2^-8 (norm, projections,
    convolution, scan, sum), each of values of the output's size."""
    spec = importlib.util.spec_from_file_location("mamba_layer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, worst = mod.main(["--width", "64", "--tokens", "75", "--dtype", dtype])
    assert losses[-1] < 0.8 * losses[0], losses
    assert worst <= close, worst
