"""The gated delta rule on the GPU against its definition in fp64 (tests/delta_ref.py)."""
import math

import numpy as np
import pytest

from tests import delta_ref as ref

pytestmark = pytest.mark.gpu

SIMT, TENSOR = 1, 2


def on_gpu(d):
    from mamba_ssd_scan_02_b200 import ssd
    return {k: ssd.to_device(v) for k, v in d.items()}


def host(t):
    return t.double().cpu().numpy()


def run_packed(ssd, cfg, g, cu, h0, kernel, **kw):
    return ssd.delta_prefill_varlen(cfg, cu, g["q"], g["k"], g["v"], g["dt"], g["b"], g["A"], g["dt_bias"],
                                    g["h0"][: len(cu) - 1] if h0 else None, kernel=kernel, **kw)


def check(ssd, cfg, d, cu, kernel, h0=True, what=""):
    import torch
    g = on_gpu(d)
    y, h = run_packed(ssd, cfg, g, cu, h0, kernel)
    torch.cuda.synchronize()
    assert ssd.get_device_error() == 0
    wy, wh = ref.prefill(cfg, d, cu, h0)
    longest = max(b - a for a, b in zip(cu, cu[1:]))
    ref.check_state(host(h), wh, longest, what)
    ref.check_y(host(y), wy, cfg, kernel == TENSOR, longest, what)


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 333])
def test_lengths(cuda_lib, L, kernel):
    cfg = ref.config()
    d = ref.inputs(cfg, L, 1, seed=L)
    check(cuda_lib, cfg, d, [0, L], kernel, what=f"L={L} kernel={kernel}")


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("kw", [
    dict(nheads=2, ngroups=1, headdim=128), dict(nheads=3, ngroups=3), dict(nheads=16, ngroups=1),
    dict(qk_norm=False, q_scale=0.5), dict(beta_scale=2.0), dict(beta_sigmoid=False, beta_scale=0.3),
    dict(dt_min=0.0, dt_max=math.inf), dict(dt_softplus=False, dt_min=0.0, dt_max=0.05), dict(q_scale=-3.0),
], ids=str)
def test_options(cuda_lib, kw, kernel):
    cfg = ref.config(**kw)
    d = ref.inputs(cfg, 150, 1, seed=3)
    if not cfg.get("qk_norm", True):  # keys of length about one keep the rule stable
        d["k"] = ref.store(ref.values(d["k"]) * 0.1, cfg)
    check(cuda_lib, cfg, d, [0, 150], kernel, what=f"{kw}")


@pytest.mark.parametrize("headdim", [64, 128])
def test_fp32(cuda_lib, headdim):
    cfg = ref.config(dtype="f32", headdim=headdim)
    d = ref.inputs(cfg, 217, 1, seed=9)
    check(cuda_lib, cfg, d, [0, 217], SIMT, what="fp32")
    check(cuda_lib, cfg, d, [0, 217], 0, h0=False, what="fp32, no state")


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("cu", [[0, 0], [0, 1, 1, 65, 70, 70, 198, 331], [0, 200, 201], [0, 0, 0, 64]], ids=str)
def test_packed(cuda_lib, cu, kernel):
    """Empty sequences hand their state on; every sequence equals its own call."""
    import torch
    cfg = ref.config(nheads=4, ngroups=2)
    d = ref.inputs(cfg, cu[-1], len(cu) - 1, seed=len(cu))
    check(cuda_lib, cfg, d, cu, kernel, what=f"{cu}")
    check(cuda_lib, cfg, d, cu, kernel, h0=False, what=f"{cu}, no state")
    g = on_gpu(d)
    y, h = run_packed(cuda_lib, cfg, g, cu, True, kernel)
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        rows = {n: g[n][None, a:b] for n in ("q", "k", "v", "dt", "b")}
        yi, hi = cuda_lib.delta_prefill(cfg, *rows.values(), g["A"], g["dt_bias"], g["h0"][i: i + 1], kernel=kernel)
        assert torch.equal(yi[0], y[a:b]) and torch.equal(hi[0], h[i])


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
def test_split_calls_and_decode_continue(cuda_lib, kernel):
    """A prompt in two calls, the state handed on in place, then tokens one at a time."""
    cfg = ref.config(nheads=8, ngroups=2)
    L, cut, steps = 230, 101, 5
    d = ref.inputs(cfg, L + steps, 1, seed=21)
    g = on_gpu(d)
    S = d["h0"].astype(np.float64)
    want = ref.rule(cfg, d, range(L + steps), S[0])
    state = g["h0"].clone()
    got = []
    for a, b in ((0, cut), (cut, L)):
        rows = [g[n][None, a:b] for n in ("q", "k", "v", "dt", "b")]
        y, h = cuda_lib.delta_prefill(cfg, *rows, g["A"], g["dt_bias"], state, h_final=state, kernel=kernel)
        assert h is state
        got.append(host(y[0]))
    for t in range(L, L + steps):
        rows = [g[n][t: t + 1] for n in ("q", "k", "v", "dt", "b")]
        got.append(host(cuda_lib.delta_decode_step(cfg, *rows, g["A"], g["dt_bias"], state)))
    ref.check_state(host(state), S, L + steps, "split")
    ref.check_y(np.concatenate(got), want, cfg, kernel == TENSOR, L + steps, "split")


@pytest.mark.parametrize("B", [1, 3, 70])
@pytest.mark.parametrize("headdim,dtype", [(64, "bf16"), (128, "bf16"), (64, "f32")])
def test_decode_pool(cuda_lib, B, headdim, dtype):
    """Slots in any order; skipped rows and unused states stay as they were."""
    import torch
    cfg = ref.config(headdim=headdim, dtype=dtype)
    n = B + 4
    d = ref.inputs(cfg, B, n, seed=B)
    g = on_gpu(d)
    slots = np.random.default_rng(B).permutation(n)[:B].astype(np.int32)
    slots[1::3] = -1
    y = torch.full((B, cfg["nheads"] * headdim), 7.0, dtype=g["q"].dtype, device="cuda")
    state = g["h0"].clone()
    out = cuda_lib.delta_decode_step(cfg, *(g[x] for x in ("q", "k", "v", "dt", "b")), g["A"], g["dt_bias"], state,
                                     torch.from_numpy(slots).cuda(), y=y)
    assert out is y and cuda_lib.get_device_error() == 0
    S = d["h0"].astype(np.float64)
    want = np.full(y.shape, 7.0)
    for i, s in enumerate(slots):
        if s >= 0:
            want[i] = ref.rule(cfg, d, [i], S[s])[0]
    ref.check_state(host(state), S, 1, "pool")
    live = slots >= 0
    ref.check_y(host(y)[live], want[live], cfg, False, 1, "pool")
    assert np.array_equal(host(y)[~live], want[~live])
    untouched = np.setdiff1d(np.arange(n), slots)
    assert torch.equal(state[untouched], g["h0"][untouched])


def test_decode_bad_slots_are_skipped_and_reported(cuda_lib):
    """A slot outside the pool, or the second row with the same slot: skipped, SSD_ERR_DEVICE_BOUNDS."""
    import torch
    cfg = ref.config()
    d = ref.inputs(cfg, 4, 3, seed=1)
    g = on_gpu(d)
    for slots in ([0, 2, 0, -1], [0, 3, 2, -5]):
        state = g["h0"].clone()
        y = cuda_lib.delta_decode_step(cfg, *(g[x] for x in ("q", "k", "v", "dt", "b")), g["A"], g["dt_bias"], state,
                                       torch.tensor(slots, dtype=torch.int32, device="cuda"))
        assert cuda_lib.get_device_error() == 6
        S = d["h0"].astype(np.float64)
        seen = set()
        for i, s in enumerate(slots):
            if 0 <= s < 3 and s not in seen:
                seen.add(s)
                ref.rule(cfg, d, [i], S[s])
            else:
                assert torch.count_nonzero(y[i]) == 0
        ref.check_state(host(state), S, 1, "bad slots")
    assert cuda_lib.get_device_error() == 0


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
def test_strided_rows(cuda_lib, kernel):
    """q, k, v, the gates and y as columns of wider matrices; rows between them stay as they were."""
    import torch
    cfg = ref.config(nheads=4, ngroups=2)
    L, qk, w = 140, 256, 256
    d = ref.inputs(cfg, 2 * L, 2, seed=4)
    g = on_gpu(d)
    big = torch.full((2, L, 3 * 256 + 64), 3.0, dtype=torch.bfloat16, device="cuda")
    big[..., :256], big[..., 256:512], big[..., 512:768] = (g[n].view(2, L, -1) for n in ("q", "k", "v"))
    big[..., 768:772], big[..., 777:781] = g["dt"].view(2, L, 4), g["b"].view(2, L, 4)
    out = torch.full((2, L, w + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    y, h = cuda_lib.delta_prefill(cfg, big[..., :qk], big[..., qk:2 * qk], big[..., 2 * qk:2 * qk + w], big[..., 768:772],
                                  big[..., 777:781], g["A"], g["dt_bias"], g["h0"], y=out[..., 8:8 + w], kernel=kernel)
    wy, wh = ref.prefill(cfg, d, [0, L, 2 * L])
    ref.check_state(host(h), wh, L, "strided")
    ref.check_y(host(y).reshape(2 * L, -1), wy, cfg, kernel == TENSOR, L, "strided")
    assert torch.all(out[..., :8] == 5) and torch.all(out[..., 8 + w:] == 5)
    # one token of longer rows: the batch rows are the rows
    one = [x[:, 7:8] for x in (big[..., :qk], big[..., qk:2 * qk], big[..., 2 * qk:2 * qk + w], big[..., 768:772],
                               big[..., 777:781])]
    y1, h1 = cuda_lib.delta_prefill(cfg, *one, g["A"], g["dt_bias"], g["h0"], kernel=kernel)
    for b in range(2):
        S = d["h0"][b].astype(np.float64)
        want = ref.rule(cfg, d, [b * L + 7], S)
        ref.check_state(host(h1[b]), S, 1, "one token")
        ref.check_y(host(y1[b]), want, cfg, kernel == TENSOR, 1, "one token")


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("scale", [1e-6, 1e4])
def test_small_and_large_values(cuda_lib, scale, kernel):
    """The rule is linear in (v, h0): any size of them keeps the relative accuracy."""
    cfg = ref.config()
    d = ref.inputs(cfg, 190, 1, seed=8, scale=scale)
    check(cuda_lib, cfg, d, [0, 190], kernel, what=f"scale {scale}")


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
def test_hard_rows(cuda_lib, kernel):
    """Zero keys and queries, equal keys with beta near one (the erase undoes itself), strong and no
    decay, a jump in the size of v."""
    cfg = ref.config(dt_min=0.0, dt_max=math.inf)
    d = ref.inputs(cfg, 200, 1, seed=6)
    k, q, v = (ref.values(d[n]) for n in ("k", "q", "v"))
    k[10:20] = 0
    q[30] = 0
    k[64:110] = k[64]
    v[130:140] *= 300
    d["k"], d["q"], d["v"] = (ref.store(x, cfg) for x in (k, q, v))
    b, dt = ref.values(d["b"]), ref.values(d["dt"])
    b[64:110] = 8
    dt[:, 0] = 6      # alpha about e^-6 A
    dt[:, 1] = -40    # alpha = 1
    d["b"], d["dt"] = ref.store(b, cfg), ref.store(dt, cfg)
    check(cuda_lib, cfg, d, [0, 200], kernel, what="hard rows")


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
def test_streams_graphs_and_repeats(cuda_lib, kernel):
    """The same bits on a side stream, in two graphs replayed in turn, and again."""
    import torch
    cfg = ref.config(nheads=8, ngroups=2)
    cu = [0, 100, 100, 290]
    d = ref.inputs(cfg, 290, 3, seed=2)
    g = on_gpu(d)
    y0, h0 = run_packed(cuda_lib, cfg, g, cu, True, kernel)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, h1 = run_packed(cuda_lib, cfg, g, cu, True, kernel, stream=side)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(h0, h1)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = run_packed(cuda_lib, cfg, g, list(cu), True, kernel)  # a host list of its own
        graphs.append((gr, out))
    for gr, out in graphs * 2:
        for t in out:
            t.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(y0, out[0]) and torch.equal(h0, out[1])
    assert cuda_lib.get_device_error() == 0
    y2, none = run_packed(cuda_lib, cfg, g, cu, True, kernel, want_state=False)
    assert none is None and torch.equal(y0, y2)


FIRST_CALL = """
import torch
from mamba_ssd_scan_02_b200 import ssd
cfg = dict(nheads=4, headdim=64, dstate=128, ngroups=2, dtype="bf16")
z = lambda *s: torch.randn(*s, device="cuda").bfloat16()
t = [z(200, 256), z(200, 256), z(200, 256), z(200, 4), z(200, 4), -torch.rand(4, device="cuda"), torch.zeros(4, device="cuda")]
step = [x[:2].clone() for x in t[:5]] + t[5:]

def calls(kernel):
    y, h = ssd.delta_prefill_varlen(cfg, [0, 120, 200], *t, kernel=kernel)
    cache, scales = ssd.state_cache(2, (4, 64, 128))
    ssd.state_store(h, cache, scales)
    back = ssd.state_load(cache, scales, torch.empty_like(h))
    y_t = ssd.delta_decode_step(cfg, *step, back)
    return y, h, back, y_t

torch.cuda.synchronize()
for kernel in (2, 1):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(kernel)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, calls(kernel))), kernel
assert ssd.get_device_error() == 0
"""


def test_first_calls_of_a_process_in_a_capture(cuda_lib):
    """A prompt, its states through the cache, a token: captured before anything else has run."""
    import subprocess
    import sys
    from pathlib import Path
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=Path(__file__).resolve().parent.parent, capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("headdim,dtype", [(64, "bf16"), (128, "f32")])
def test_decode_of_a_large_batch(cuda_lib, headdim, dtype):
    """More states than the L2 cache keeps (over 64 MB), in slots, some rows without one."""
    import torch
    cfg = ref.config(nheads=64, ngroups=8, headdim=headdim, dtype=dtype)
    B = 131072 // (64 * headdim) + 3
    d = ref.inputs(cfg, B, B, seed=21)
    g = on_gpu(d)
    slots = np.random.default_rng(3).permutation(B).astype(np.int32)
    slots[4::9] = -1
    state = g["h0"].clone()
    y = cuda_lib.delta_decode_step(cfg, *(g[x] for x in ("q", "k", "v", "dt", "b")), g["A"], g["dt_bias"], state,
                                   torch.from_numpy(slots).cuda())
    S = d["h0"].astype(np.float64)
    want = np.zeros((B, 64 * headdim))
    for i, s in enumerate(slots):
        if s >= 0:
            want[i] = ref.rule(cfg, d, [i], S[s])[0]
    ref.check_state(host(state), S, 1, "large")
    ref.check_y(host(y), want, cfg, False, 1, "large")


def test_two_calls_at_once(cuda_lib):
    """Chunked kernels and the recurrence on two streams at the same time: the bits of each alone."""
    import torch
    cfg = ref.config(nheads=32, ngroups=4)
    g = on_gpu(ref.inputs(cfg, 1500, 1, seed=12))
    alone = {k: run_packed(cuda_lib, cfg, g, [0, 1500], True, k) for k in (SIMT, TENSOR)}
    streams = {k: torch.cuda.Stream() for k in alone}
    for s in streams.values():
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        for k, s in streams.items():
            got.append((k, run_packed(cuda_lib, cfg, g, [0, 1500], True, k, stream=s)))
    torch.cuda.synchronize()
    for k, out in got:
        assert all(torch.equal(a, b) for a, b in zip(alone[k], out)), k
    assert cuda_lib.get_device_error() == 0


def test_states_beyond_32_bits_of_offset(cuda_lib):
    """A pool of 2100 states of 128 heads: its last lie over 2^31 elements in (8.8 GB)."""
    import torch
    cfg = ref.config(nheads=128, ngroups=8)
    g = on_gpu(ref.inputs(cfg, 2, 2, seed=6))
    rows = [g[n] for n in ("q", "k", "v", "dt", "b")]
    few = g["h0"].clone()
    want = cuda_lib.delta_decode_step(cfg, *rows, g["A"], g["dt_bias"], few)
    pool = torch.empty(2100, 128, 64, 128, device="cuda")
    assert pool[:2099].numel() > 2 ** 31
    slots = torch.tensor([2099, 2060], dtype=torch.int32, device="cuda")
    pool[slots.long()] = g["h0"]
    y = cuda_lib.delta_decode_step(cfg, *rows, g["A"], g["dt_bias"], pool, slots)
    assert torch.equal(y, want) and torch.equal(pool[slots.long()], few)
    cache, scales = cuda_lib.state_cache(2, (128, 64, 128))
    ref_cache, ref_scales = cuda_lib.state_cache(2, (128, 64, 128))
    cuda_lib.state_store(pool, cache, scales, state_slots=slots)
    cuda_lib.state_store(few, ref_cache, ref_scales)
    assert torch.equal(cache.view(torch.uint8), ref_cache.view(torch.uint8)) and torch.equal(scales, ref_scales)
    cuda_lib.state_load(cache, scales, pool, state_slots=slots)
    assert torch.equal(pool[2099], cuda_lib.state_load(cache, scales, few)[0])
    assert cuda_lib.get_device_error() == 0


@pytest.mark.parametrize("packed", [False, True])
def test_no_tokens_need_only_the_states(cuda_lib, packed):
    """With no token at all, every pointer but the states' (and a packed call's workspace) may be null."""
    import ctypes
    import torch
    cfg = ref.config(nheads=4)
    h0 = torch.randn(3, 4, 64, 128, device="cuda")
    out = torch.zeros_like(h0)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    args = cuda_lib.DeltaArgs(h0=h0.data_ptr(), h_final=out.data_ptr(), workspace=ws.data_ptr(), workspace_bytes=4096)
    lib, stream = cuda_lib.load(), torch.cuda.current_stream().cuda_stream
    if packed:
        c = cuda_lib.make_delta_config(cfg, 1, 0)
        status = lib.ssd_delta_prefill_varlen(ctypes.byref(c), ctypes.byref(args), (ctypes.c_int * 4)(0, 0, 0, 0), 3, stream)
    else:
        c = cuda_lib.make_delta_config(cfg, 3, 0)
        status = lib.ssd_delta_prefill(ctypes.byref(c), ctypes.byref(args), stream)
    torch.cuda.synchronize()
    assert status == 0 and torch.equal(out, h0) and cuda_lib.get_device_error() == 0


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
def test_a_full_machine_gives_equal_bits(cuda_lib, kernel):
    """Many sequences at once, on every SM: the same bits whatever the workspace held and whatever the L2
    cache holds, and each sequence has the bits of its own call."""
    import torch
    cfg = ref.config(nheads=64, ngroups=8)
    r = np.random.default_rng(5)
    cu = np.concatenate([[0], np.cumsum(r.integers(1, 500, 24))]).tolist()
    g = on_gpu(ref.inputs(cfg, cu[-1], len(cu) - 1, seed=1))
    n = cuda_lib.delta_varlen_workspace_size(cfg, cu, kernel)
    flood = torch.empty(1 << 26, device="cuda")
    first = None
    for i in range(12):
        if i % 3 == 1:
            flood.fill_(float(i))
        ws = torch.full((max(n, 1),), 37 * i % 251, dtype=torch.uint8, device="cuda")
        got = run_packed(cuda_lib, cfg, g, cu, True, kernel, workspace=ws)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got)), i
    for i in (0, 7, 23):
        part = {k: v[cu[i]:cu[i + 1]] if k in ("q", "k", "v", "dt", "b") else v for k, v in g.items()}
        part["h0"] = g["h0"][i:i + 1]
        y, h = run_packed(cuda_lib, cfg, part, [0, cu[i + 1] - cu[i]], True, kernel)
        assert torch.equal(y, first[0][cu[i]:cu[i + 1]]) and torch.equal(h[0], first[1][i]), i


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("name", ["q", "k", "v", "dt", "b"])
def test_nan_and_infinity_stay_where_they_belong(cuda_lib, name, bad, kernel):
    """In one token of one head (or group): no y or state is finite where the definition's is not, and outside of
    that head, and before that token (its chunk, on the tensor cores), nothing changes."""
    import torch
    cfg = ref.config(nheads=4, ngroups=2)
    cu, t = [0, 90, 290], 200  # token 110 of the second sequence
    d = ref.inputs(cfg, cu[-1], 2, seed=8)
    clean = run_packed(cuda_lib, cfg, on_gpu(d), cu, True, kernel)
    at = {"q": 128 + 5, "k": 128 + 5, "v": 2 * 64 + 9, "dt": 2, "b": 2}[name]  # head 2, group 1
    g = on_gpu(d)
    g[name][t, at] = bad
    y, h = run_packed(cuda_lib, cfg, g, cu, True, kernel)
    torch.cuda.synchronize()
    assert cuda_lib.get_device_error() == 0
    heads = [2, 3] if name in ("q", "k") else [2]
    other = [i for i in range(4) if i not in heads]
    first = t if kernel == SIMT else cu[1] + 64
    yh, ch = (x.view(-1, 4, 64) for x in (y, clean[0]))
    assert torch.equal(yh[:, other], ch[:, other]) and torch.equal(yh[:first], ch[:first])
    assert torch.equal(h[0], clean[1][0]) and torch.equal(h[1, other], clean[1][1, other])
    x = {k: ref.values(v).copy() for k, v in d.items()}
    x[name][t, at] = bad
    with np.errstate(all="ignore"):
        wy, wh = ref.prefill(cfg, x, cu, True)
    assert not np.any(np.isfinite(host(y)) & ~np.isfinite(wy.reshape(host(y).shape)))
    assert not np.any(np.isfinite(host(h)) & ~np.isfinite(wh))
    if name == "q":
        assert torch.equal(h, clean[1])


def test_decode_graph(cuda_lib):
    """Captured decode steps over a pool, with the slots changed between replays."""
    import torch
    cfg = ref.config()
    d = ref.inputs(cfg, 2, 5, seed=13)
    g = on_gpu(d)
    state, slots = g["h0"].clone(), torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    args = [g[x] for x in ("q", "k", "v", "dt", "b")]
    cuda_lib.delta_decode_step(cfg, *args, g["A"], g["dt_bias"], state.clone(), slots)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y = cuda_lib.delta_decode_step(cfg, *args, g["A"], g["dt_bias"], state, slots)
    state.copy_(g["h0"])
    S = d["h0"].astype(np.float64)
    for s in ([4, 1], [1, 4], [-1, 0]):
        slots.copy_(torch.tensor(s, dtype=torch.int32))
        gr.replay()
        torch.cuda.synchronize()
        for i, x in enumerate(s):
            if x >= 0:
                want = ref.rule(cfg, d, [i], S[x])
                ref.check_y(host(y[i: i + 1]), want, cfg, False, 3, "replayed")
    ref.check_state(host(state), S, 3, "replayed")
