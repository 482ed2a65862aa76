"""Arguments of linear attention and group norm that are refused (no GPU)."""
import pytest
import torch

import mamba_ssd_chunked_02_amd as m
from test_linattn_host import SHAPE, call, gn_dims, needs_no_gpu


@needs_no_gpu
def test_groupnorm_reserved():
    """dims->reserved is 0, as the header says, so that a later meaning can be told apart."""
    for f in ("ssd_groupnorm_fwd", "ssd_groupnorm_bwd"):
        assert call(f, gn_dims(reserved=1)) == SHAPE
    assert call("ssd_groupnorm_fwd", gn_dims(samples=0), x=None, y=None) == 0


def test_maps_that_have_no_one_stride():
    """A crop of a map, whose rows of positions lie apart, and a gradient expanded from one number:
    an error of the binding's, which names the tensor."""
    z = torch.zeros
    x, dy, st = z(2, 6, 6, 8), z(2, 6, 6, 8), z(2, 2)
    crop = z(2, 6, 9, 8)[:, :, :6]
    one = z(()).expand(2, 6, 6, 8)
    for name, c in (("x", lambda: m.ssd_groupnorm_fwd(crop, 2)),
                    ("z", lambda: m.ssd_groupnorm_fwd(x, 2, z=crop)),
                    ("y", lambda: m.ssd_groupnorm_fwd(x, 2, y=crop)),
                    ("dy", lambda: m.ssd_groupnorm_bwd(x, 2, None, None, st, st, crop)),
                    ("dy", lambda: m.ssd_groupnorm_bwd(x, 2, None, None, st, st, one)),
                    ("x", lambda: m.ssd_groupnorm_bwd(crop, 2, None, None, st, st, dy))):
        with pytest.raises(ValueError, match=rf"^{name} needs"):
            c()
    # positions that form one stride, in any order of the samples, are taken (and reach the GPU check)
    for t in (z(2, 6, 6, 9)[..., :8], z(6, 6, 2, 8).permute(2, 0, 1, 3), z(36, 8).expand(2, 36, 8), z(2, 1, 6, 8)):
        with pytest.raises(ValueError, match="GPU"):
            m.ssd_groupnorm_fwd(t, 2)
