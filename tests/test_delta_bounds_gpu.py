"""The debug build's device-side index checks (libssd_debug.so) in the gated delta rule and the state cache.

Each build runs in a subprocess of its own, as in test_debug_bounds_gpu.py: with the full extents the
checked build gives the same bits and no error; with half of each buffer's extent allowed the stores of the
second half are skipped and reported, on buffers that are valid throughout."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SSD_ERR_DEVICE_BOUNDS = 6

CASE = """
import sys
import numpy as np
import torch
from mamba_ssd_scan_02_b200 import ssd
from tests import delta_ref as ref
ssd.load(sys.argv[1])
cfg = ref.config(nheads=4, ngroups=2)
d = {k: ssd.to_device(v) for k, v in ref.inputs(cfg, 200, 2, seed=4).items()}
rows = [d[n][None] for n in ("q", "k", "v", "dt", "b")]
nan = float("nan")
new = lambda *s, dtype=torch.float32: torch.full(s, nan, dtype=dtype, device="cuda")
out, status = {}, {}
ssd.get_device_error()
ssd.test_bounds_scale(int(sys.argv[2]))
for kernel in (1, 2):
    y, h = new(1, 200, 256, dtype=torch.bfloat16), new(1, 4, 64, 128)
    ssd.delta_prefill(cfg, *rows, d["A"], d["dt_bias"], d["h0"][:1], y=y, h_final=h, kernel=kernel)
    status[f"prefill{kernel}"] = ssd.get_device_error()
    out[f"prefill{kernel}_y"], out[f"prefill{kernel}_h"] = y[0], h[0]
y, state = new(2, 256, dtype=torch.bfloat16), d["h0"].clone()
ssd.delta_decode_step(cfg, *(d[n][:2] for n in ("q", "k", "v", "dt", "b")), d["A"], d["dt_bias"], state, y=y)
status["decode"] = ssd.get_device_error()
out["decode_y"], out["decode_h"] = y, state
cache, scales = ssd.state_cache(2, (4, 64, 128), "int8")
ssd.state_store(d["h0"], cache, scales)
status["store"] = ssd.get_device_error()
back = new(2, 4, 64, 128)
ssd.state_load(cache, scales, back)
status["load"] = ssd.get_device_error()
out["store_q"], out["load_x"] = cache, back
ssd.test_bounds_scale(1)
np.savez(sys.argv[3], debug=int(ssd.debug_bounds_build()), **{k: v.float().cpu().numpy() for k, v in out.items()},
         **{"status_" + k: v for k, v in status.items()})
"""


def run(tmp_path, lib, denom):
    out = str(tmp_path / f"{os.path.basename(lib)}_{denom}.npz")
    r = subprocess.run([sys.executable, "-c", CASE, lib, str(denom), out], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return dict(np.load(out))


def test_index_checks_of_the_debug_build(cuda_lib, tmp_path):
    from mamba_ssd_scan_02_b200 import ssd
    if not os.path.exists(ssd.DEBUG_LIB_PATH):  # normally built beside libssd.so by build()
        from mamba_ssd_scan_02_b200 import build as _b
        _b.build(debug_bounds=True)
    want = run(tmp_path, ssd.LIB_PATH, 1)
    full = run(tmp_path, ssd.DEBUG_LIB_PATH, 1)
    half = run(tmp_path, ssd.DEBUG_LIB_PATH, 2)
    assert (want["debug"], full["debug"], half["debug"]) == (0, 1, 1)
    status = [k for k in want if k.startswith("status_")]
    assert all(want[k] == 0 and full[k] == 0 and half[k] == SSD_ERR_DEVICE_BOUNDS for k in status), half
    for k in want:
        if k not in status and k != "debug":
            assert np.array_equal(want[k], full[k]), k
    for kernel in (1, 2):
        y, h = half[f"prefill{kernel}_y"], half[f"prefill{kernel}_h"]
        assert np.array_equal(y[:99], want[f"prefill{kernel}_y"][:99]) and np.isnan(y[100:]).all()
        assert np.array_equal(h[:2], want[f"prefill{kernel}_h"][:2]) and np.isnan(h[2:]).all()
    assert np.array_equal(half["decode_h"][0], want["decode_h"][0]) and not np.array_equal(half["decode_h"][1], want["decode_h"][1])
    assert np.array_equal(half["store_q"][0], want["store_q"][0]) and not half["store_q"][1].any()
    assert np.array_equal(half["load_x"][0], want["load_x"][0]) and np.isnan(half["load_x"][1]).all()
