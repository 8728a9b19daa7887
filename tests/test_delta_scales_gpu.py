"""The gated delta rule where the sizes of its factors differ widely."""
import math

import pytest

from tests import delta_ref as ref
from tests.test_delta_gpu import SIMT, TENSOR, on_gpu, run_packed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("kernel", [0, SIMT, TENSOR])
def test_an_empty_sequence_hands_its_state_on_as_it_is(cuda_lib, kernel, inplace):
    """Of any size, bit for bit, beside sequences that are long enough for the chunked kernels."""
    import torch
    cfg = ref.config(nheads=4, ngroups=2)
    cu = [0, 0, 200, 200, 300, 300]
    g = on_gpu(ref.inputs(cfg, cu[-1], 5, seed=3))
    g["h0"][0] *= 1e30
    g["h0"][2] *= 30
    g["h0"][4, 0] = 1e-38
    g["h0"][4, 1, 3, 7], g["h0"][4, 1, 3, 8] = math.inf, math.nan
    want = g["h0"].clone()
    out = g["h0"] if inplace else None
    y, h = run_packed(cuda_lib, cfg, g, cu, True, kernel, h_final=out)
    assert cuda_lib.get_device_error() == 0
    for i in (0, 2, 4):
        assert torch.equal(h[i].view(torch.int32), want[i].view(torch.int32)), i
    assert torch.isfinite(y).all() and torch.isfinite(h[1]).all() and torch.isfinite(h[3]).all()
