"""The gated delta rule where the sizes of its factors differ widely."""
import math

import numpy as np
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


def steady(cfg, n, A, dt, seed=0, h0=0.3):
    """n tokens of one decay each: dt as it is, no bias; heads 0 .. of A."""
    d = ref.inputs(cfg, n, 1, seed=seed)
    d["A"] = np.array(A, np.float32)
    d["dt_bias"] = np.zeros(len(A), np.float32)
    d["dt"] = ref.store(np.full((n, len(A)), dt), cfg)
    d["h0"] = (h0 / 0.3 * d["h0"]).astype(np.float32)
    return d


HARD = dict(dt_softplus=False, dt_min=0.0, dt_max=math.inf)


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("size", [1e-3, 1000.0, 1e6, 1e30])
def test_a_state_that_decays_to_nothing_stays_finite(cuda_lib, size, kernel):
    """Chunks without values that decay by 2^-148, behind them tokens with values again."""
    import torch
    cfg = ref.config(**HARD)
    g = on_gpu(steady(cfg, 300, [-16.0, -16.0, -0.01, -4.0], 0.1, seed=2, h0=size))
    for zeros in (64, 128, 150, 300):
        part = dict(g, v=g["v"].clone())
        part["v"][:zeros] = 0
        y, h = run_packed(cuda_lib, cfg, part, [0, 300], True, kernel)
        assert torch.isfinite(y).all() and torch.isfinite(h).all() and cuda_lib.get_device_error() == 0
        # what comes after no longer knows the state that came in: heads 0 and 1 decay by 2^-148 per 64 tokens
        y0, h0 = run_packed(cuda_lib, cfg, part, [0, 300], False, kernel)
        assert torch.allclose(h[0, :2], h0[0, :2], rtol=0, atol=2.0 ** -20 * float(h0[0, :2].abs().max()) + 1e-30)
