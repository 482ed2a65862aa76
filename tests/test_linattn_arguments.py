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
