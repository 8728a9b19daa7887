"""fp32 states into the 8-bit cache and back, against exact arithmetic (tests/delta_ref.py)."""
import numpy as np
import pytest

from tests import delta_ref as ref

pytestmark = pytest.mark.gpu


def elements(cache):
    import torch
    raw = cache.view(torch.uint8).cpu().numpy()
    return ref.E4M3[raw] if cache.dtype == torch.float8_e4m3fn else raw.view(np.int8).astype(np.float64)


def states(n, shape, seed):
    """Blocks of many sizes: zeros, subnormals, ties, the format's limits, the largest floats."""
    r = np.random.default_rng(seed)
    x = (r.standard_normal((n, *shape)) * np.exp(r.uniform(-60, 60, (n, *shape[:-1], 1)))).astype(np.float32)
    b = x.reshape(-1, 32)
    special = [np.zeros(32), np.full(32, 2.0 ** -149), np.full(32, 448.0), np.full(32, 448.00003), np.full(32, 127.0),
               np.full(32, 127.00001), np.arange(32) + 0.5, np.arange(-448, 448, 28.0), 8.5 * np.arange(32),
               np.full(32, 3.4028234e38), np.full(32, -1.1754944e-38), 2.0 ** -np.arange(32.0)]
    for i, s in enumerate(special[: len(b)]):
        b[i] = s
    return x


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("shape", [(1, 1, 128), (3, 64, 128), (2, 128, 128), (5, 7, 128), (4, 32)], ids=str)
def test_roundtrip(cuda_lib, fmt, shape):
    import torch
    x = states(3, shape, 1)
    cache, scales = cuda_lib.state_cache(3, shape, fmt)
    dev = torch.from_numpy(x).cuda()
    out = cuda_lib.state_store(dev, cache, scales)
    assert out[0] is cache and out[1] is scales
    q, e = ref.cache_blocks(x, fmt)
    assert np.array_equal(scales.cpu().numpy(), e)
    assert np.array_equal(elements(cache), q)
    back = cuda_lib.state_load(cache, scales, torch.empty_like(dev))
    want = (q.reshape(*q.shape[:-1], -1, 32) * np.exp2(e.astype(np.float64) - 127)[..., None]).reshape(x.shape)
    assert np.array_equal(back.cpu().numpy().astype(np.float64), want.astype(np.float32).astype(np.float64))
    assert cuda_lib.get_device_error() == 0
    # the documented bound: one rounding of half a step
    top = np.abs(x.astype(np.float64)).reshape(*x.shape[:-1], -1, 32).max(-1, keepdims=True)
    err = np.abs(want - x).reshape(*x.shape[:-1], -1, 32)
    size = np.exp2(e.astype(np.float64) - 127)[..., None]
    if fmt == "int8":
        assert np.all(err <= np.maximum(top / 127, 2.0 ** -128))
    else:
        assert np.all(err <= 2.0 ** -4 * np.abs(x.astype(np.float64)).reshape(err.shape) + 2.0 ** -10 * size)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_infinities_and_nans_mark_their_block(cuda_lib, fmt):
    import torch
    x = np.ones((1, 2, 128), np.float32)
    x[0, 0, 5], x[0, 0, 70], x[0, 1, 127] = np.nan, np.inf, -np.inf
    cache, scales = cuda_lib.state_cache(1, (2, 128), fmt)
    cuda_lib.state_store(torch.from_numpy(x).cuda(), cache, scales)
    back = cuda_lib.state_load(cache, scales, torch.zeros(1, 2, 128, device="cuda")).cpu().numpy().reshape(8, 32)
    bad = [0, 2, 7]
    assert scales.cpu().numpy().reshape(-1)[bad].tolist() == [255] * 3
    assert np.isnan(back[bad]).all()
    assert (np.delete(back, bad, axis=0) == 1).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_slots(cuda_lib, fmt):
    """Any order on both sides; skipped entries and other places stay as they were."""
    import torch
    shape = (2, 64, 128)
    x = torch.from_numpy(states(6, shape, 2)).cuda()
    cache, scales = cuda_lib.state_cache(9, shape, fmt)
    full = cuda_lib.state_cache(6, shape, fmt)
    cuda_lib.state_store(x, *full)
    s = torch.tensor([5, 0, -1, 3, 2], dtype=torch.int32, device="cuda")
    c = torch.tensor([8, 1, 4, -2, 0], dtype=torch.int32, device="cuda")
    cuda_lib.state_store(x, cache, scales, s, c)
    raw, wraw = cache.view(torch.uint8), full[0].view(torch.uint8)
    for i, j in ((5, 8), (0, 1), (2, 0)):
        assert torch.equal(raw[j], wraw[i]) and torch.equal(scales[j], full[1][i])
    for j in (2, 3, 4, 5, 6, 7):
        assert not raw[j].any() and not scales[j].any()
    y = torch.full((4, *shape), 9.0, device="cuda")
    a = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    b = torch.tensor([8, 8], dtype=torch.int32, device="cuda")  # one place may be read twice
    cuda_lib.state_load(cache, scales, y, a, b)
    want = cuda_lib.state_load(*full, torch.empty_like(x))
    assert torch.equal(y[3], want[5]) and torch.equal(y[1], want[5])
    assert (y[0] == 9).all() and (y[2] == 9).all()
    assert cuda_lib.get_device_error() == 0


def test_bad_slots_are_skipped_and_reported(cuda_lib):
    import torch
    shape = (1, 64, 128)
    x = torch.randn(3, *shape, device="cuda")
    cache, scales = cuda_lib.state_cache(3, shape, "int8")
    i32 = dict(dtype=torch.int32, device="cuda")
    for s, c in (([0, 1, 2], [1, 2, 1]), ([0, 3, 1], [0, 1, 2]), ([0, 1, 2], [0, 3, 2])):
        want = cuda_lib.state_cache(3, shape, "int8")
        seen = set()
        for i, j in zip(s, c):
            if i < 3 and j < 3 and j not in seen:
                seen.add(j)
                cuda_lib.state_store(x[i:i + 1], want[0][j:j + 1], want[1][j:j + 1])
        cache.view(torch.uint8).zero_()
        scales.zero_()
        cuda_lib.state_store(x, cache, scales, torch.tensor(s, **i32), torch.tensor(c, **i32))
        assert cuda_lib.get_device_error() == 6
        assert torch.equal(cache, want[0]) and torch.equal(scales, want[1])
    y = torch.zeros(2, *shape, device="cuda")
    cuda_lib.state_load(cache, scales, y, torch.tensor([0, 0], **i32), torch.tensor([0, 2], **i32))
    assert cuda_lib.get_device_error() == 6
    assert torch.equal(y[0], cuda_lib.state_load(cache, scales, torch.empty_like(x))[0]) and not y[1].any()
    assert cuda_lib.get_device_error() == 0


def test_both_layers_states_through_the_cache(cuda_lib):
    """A served sequence: prefill, the state put away and brought back, decode; for the scan and for the
    delta rule.  The state comes back within the format's rounding, and the call that follows runs
    on it."""
    import torch
    from tests.gpu_util import dev, make_case, run_gpu_prefill, small_cfg
    cfg = small_cfg(batch=2, seqlen=70, norm_groups=0)
    inp = make_case(cfg)
    _, h, _ = run_gpu_prefill(cfg, inp)
    dc = ref.config(nheads=16, ngroups=2)
    d = ref.inputs(dc, 2 * 70, 2, seed=5)
    g = {k: dev(v) for k, v in d.items()}
    rows = [g[n].view(2, 70, -1) for n in ("q", "k", "v", "dt", "b")]
    _, hd = cuda_lib.delta_prefill(dc, *rows, g["A"], g["dt_bias"])
    for state in (h, hd):
        for fmt, bound in (("e4m3", 2.0 ** -4), ("int8", 1 / 127)):
            cache, scales = cuda_lib.state_cache(4, state.shape[1:], fmt)
            at = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
            cuda_lib.state_store(state, cache, scales, cache_slots=at)
            back = cuda_lib.state_load(cache, scales, torch.empty_like(state), cache_slots=at)
            top = state.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True)
            assert ((back - state).abs().unflatten(-1, (-1, 32)) <= bound * top).all()
    y = cuda_lib.delta_decode_step(dc, *(r[:, 0].contiguous() for r in rows), g["A"], g["dt_bias"], back.clone())
    S = back.cpu().numpy().astype(np.float64)
    want = np.stack([ref.rule(dc, d, [i * 70], S[i])[0] for i in range(2)])
    ref.check_y(y.double().cpu().numpy(), want, dc, False, 1, "after the cache")
    assert cuda_lib.get_device_error() == 0
