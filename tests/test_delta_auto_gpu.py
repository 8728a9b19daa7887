"""Which kernels AUTO takes, as the workspace it asks for (none for the recurrence) and the bits it gives show."""
import math

import numpy as np
import pytest

from tests import delta_ref as ref
from tests.test_delta_gpu import SIMT, TENSOR, check, on_gpu, run_packed

pytestmark = pytest.mark.gpu


def chunked(ssd, cfg, batch=1, seqlen=200, **kw):
    c = dict(nheads=8, ngroups=2, dtype="bf16")
    c.update(cfg, **kw)
    n = ssd.delta_workspace_size(c, batch, seqlen)
    assert n in (0, ssd.delta_workspace_size(dict(c, kernel=TENSOR), batch, seqlen))
    return n > 0


@pytest.mark.parametrize("kw,want", [
    (dict(), True), (dict(dt_min=1e-3, dt_max=0.1), True), (dict(dt_softplus=False), True),
    (dict(dt_softplus=False, dt_min=-0.1), False), (dict(dt_softplus=False, dt_min=-math.inf), False),
    (dict(dt_min=-1.0), True), (dict(dt_min=-1.0, dt_max=-0.5), False), (dict(dt_min=-1.0, dt_max=0.0), True),
    (dict(qk_norm=False), False), (dict(beta_sigmoid=False), False), (dict(beta_scale=2.0), True),
    (dict(beta_scale=2.5), False), (dict(beta_scale=-1.0), False), (dict(dtype="f32"), False),
], ids=str)
def test_configurations_whose_operands_are_bounded(cuda_lib, kw, want):
    """beta |k|^2 <= 2, and alpha <= 1 where A <= 0: a dt that can be negative goes to the recurrence."""
    assert chunked(cuda_lib, kw) == want
    assert not chunked(cuda_lib, kw, kernel=SIMT)


@pytest.mark.parametrize("nheads,headdim,batch,seqlen,want", [
    (8, 64, 1, 127, False), (8, 64, 1, 128, True), (37, 64, 1, 127, False), (37, 64, 1, 128, True),
    (38, 64, 1, 27, False), (38, 64, 1, 28, True), (8, 64, 8, 27, False), (8, 64, 8, 28, True),
    (18, 128, 1, 127, False), (19, 128, 1, 28, True), (8, 64, 1, 0, False),
])
def test_thresholds(cuda_lib, nheads, headdim, batch, seqlen, want):
    assert chunked(cuda_lib, dict(nheads=nheads, ngroups=1, headdim=headdim), batch, seqlen) == want


@pytest.mark.parametrize("nheads,seqlen,kernel", [(4, 127, SIMT), (4, 128, TENSOR), (40, 27, SIMT), (40, 28, TENSOR)])
def test_both_sides_of_both_thresholds(cuda_lib, nheads, seqlen, kernel):
    """The definition's result, in the bits of the kernel that is chosen."""
    import torch
    cfg = ref.config(nheads=nheads, ngroups=2)
    d = ref.inputs(cfg, seqlen, 1, seed=seqlen)
    cu = [0, seqlen]
    check(cuda_lib, cfg, d, cu, kernel, what="explicit")
    g = on_gpu(d)
    auto = run_packed(cuda_lib, cfg, g, cu, True, 0)
    assert all(torch.equal(a, b) for a, b in zip(auto, run_packed(cuda_lib, cfg, g, cu, True, kernel)))
    rows = [g[n][None] for n in ("q", "k", "v", "dt", "b")]
    y, h = cuda_lib.delta_prefill(cfg, *rows, g["A"], g["dt_bias"], g["h0"])
    assert torch.equal(y[0], auto[0]) and torch.equal(h, auto[1])


@pytest.mark.parametrize("cu", [[0, 1, 2, 3, 31, 32], [0, 5, 5, 140, 141], [0, 3, 30, 57]], ids=str)
def test_packed_by_the_longest(cuda_lib, cu):
    """Sequences of one token beside one that is long enough for the chunked kernels, and none that is."""
    import torch
    cfg = ref.config(nheads=40, ngroups=2)
    d = ref.inputs(cfg, cu[-1], len(cu) - 1, seed=5)
    kernel = TENSOR if max(b - a for a, b in zip(cu, cu[1:])) >= 28 else SIMT
    check(cuda_lib, cfg, d, cu, kernel, what=f"{cu}")
    g = on_gpu(d)
    assert all(torch.equal(a, b) for a, b in zip(run_packed(cuda_lib, cfg, g, cu, True, 0), run_packed(cuda_lib, cfg, g, cu, True, kernel)))


@pytest.mark.parametrize("cu", [[0, 27], [0, 28], [0, 128], [0, 200], [0, 30, 30, 200]], ids=str)
def test_negative_steps(cuda_lib, cu):
    """dt without softplus and with a negative dt_min: alpha above one, for prompts of any length as for decode."""
    cfg = ref.config(nheads=8, dt_softplus=False, dt_min=-0.1, dt_max=0.1)
    d = ref.inputs(cfg, cu[-1], len(cu) - 1, seed=6)
    d["A"] = np.full(8, -4.0, np.float32)
    d["dt_bias"] = np.zeros(8, np.float32)
    d["dt"] = ref.store(-0.07 + 0.01 * ref.values(d["dt"]), cfg)  # alpha = 2^0.4 on the average
    d["b"] = ref.store(3 + ref.values(d["b"]), cfg)
    check(cuda_lib, cfg, d, cu, 0, what=f"{cu}")


def test_packed_fp32(cuda_lib):
    """Several fp32 sequences, one of them empty, with and without a state."""
    for headdim in (64, 128):
        cfg = ref.config(dtype="f32", headdim=headdim)
        cu = [0, 40, 40, 41, 200]
        d = ref.inputs(cfg, cu[-1], len(cu) - 1, seed=7)
        check(cuda_lib, cfg, d, cu, 0, what="fp32")
        check(cuda_lib, cfg, d, cu, 0, h0=False, what="fp32, no state")
