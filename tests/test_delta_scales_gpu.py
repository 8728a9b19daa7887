"""The gated delta rule where the sizes of its factors differ widely, judged head by head.

`definition` follows, for each head, the root mean square of the largest thing that its state was made of, as
it decays: token t writes a term of beta_t |k_t| |v_t| / sqrt(P N), and the state itself, as large as it was
after any token, is rounded by every form of the rule.  The chunked kernels keep 22 bits of each factor of a term, about
2^-21 of it; the 64 terms of a chunk add up like the root of their number, 2^-18 of the largest, and so do
chunks.  The recurrence rounds its state to 24 bits, half a step or 2^-24 of it, a few times per token: for 64
tokens less than 2^-18 even if all of them add up.  What a head was before it decayed, and what the others
are, must not matter."""
import math

import numpy as np
import pytest

from tests import delta_ref as ref
from tests.test_delta_gpu import SIMT, TENSOR, host, on_gpu, run_packed

pytestmark = pytest.mark.gpu


def definition(cfg, d, cu):
    """y [rows, H, P], final states [nseq, H, P, N], and the sizes [nseq, H] described above."""
    H, P, N, G = cfg["nheads"], cfg["headdim"], cfg["dstate"], cfg["ngroups"]
    S = d["h0"][: len(cu) - 1].astype(np.float64)
    y, size = np.zeros((cu[-1], H, P)), np.zeros((len(cu) - 1, H))
    rms = lambda x: np.sqrt(np.mean(x * x, axis=(1, 2)))
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        r = rms(S[i])
        for t in range(a, b):
            k = ref.values(d["k"][t]).reshape(G, N)
            if cfg.get("qk_norm", True):
                k = k / np.sqrt((k * k).sum(-1, keepdims=True) + cfg.get("qk_eps", 1e-6))
            k = np.repeat(np.sqrt((k * k).sum(-1)), H // G)
            v = np.sqrt(np.square(ref.values(d["v"][t]).reshape(H, P)).sum(-1))
            x = ref.values(d["dt"][t]) + d["dt_bias"]
            dt = np.clip(np.logaddexp(x, 0) if cfg.get("dt_softplus", True) else x, cfg.get("dt_min", 0.0), cfg.get("dt_max", math.inf))
            z = ref.values(d["b"][t])
            beta = cfg.get("beta_scale", 1.0) * (1 / (1 + np.exp(-z)) if cfg.get("beta_sigmoid", True) else z)
            y[t] = ref.rule(cfg, d, [t], S[i]).reshape(H, P)
            r = np.maximum(np.maximum(r * np.exp(d["A"] * dt), beta * k * v / math.sqrt(P * N)), rms(S[i]))
        size[i] = r
    return y, S, size


def check_heads(ssd, cfg, d, cu, kernel, what=""):
    """Every head of every sequence against the definition."""
    import torch
    y, h = run_packed(ssd, cfg, on_gpu(d), cu, True, kernel)
    torch.cuda.synchronize()
    assert ssd.get_device_error() == 0
    wy, wh, size = definition(cfg, d, cu)
    y, h = host(y).reshape(wy.shape), host(h)
    assert np.isfinite(y).all() and np.isfinite(h).all(), what
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        # (a decay below fp32's smallest normal number, 2^-126, is zero)
        floor = 2.0 ** -126 * np.maximum(1.0, np.abs(d["h0"][i]).max(axis=(1, 2)))
        bound = 2.0 ** -18 * math.sqrt((b - a + 63) // 64) * size[i] + floor
        err = np.sqrt(np.mean(np.square(h[i] - wh[i]), axis=(1, 2)))
        assert (err <= bound).all(), f"{what}: sequence {i}, state off by {err} where {bound} is allowed"
        for at in range(a, b, 64):  # y: one rounding to bf16; 11 bits of the products of its chunk and head (as check_y)
            g, w = y[at:min(at + 64, b)], wy[at:min(at + 64, b)]
            rms = np.sqrt(np.mean(w * w, axis=(0, 2), keepdims=True))
            excess = np.abs(g - w) - 2.0 ** -8 * np.abs(w) - 1e-2 * rms
            assert (excess <= 2.0 ** -126).all(), f"{what}: sequence {i}, tokens {at} .., y beyond its bound"


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


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("tokens", [64, 128, 150])
@pytest.mark.parametrize("size", [1e-3, 1000.0, 1e6])
def test_no_values_under_strong_decay(cuda_lib, size, tokens, kernel):
    """V is zero and a chunk decays by 2^-148 (heads 0, 1), by next to nothing (head 2): no NaN, no infinity, and the
    last tokens' values count again."""
    cfg = ref.config(**HARD)
    d = steady(cfg, tokens + 70, [-16.0, -16.0, -0.01, -4.0], 0.1, seed=2, h0=size)
    v = ref.values(d["v"])
    v[:tokens] = 0
    d["v"] = ref.store(v, cfg)
    check_heads(cuda_lib, cfg, d, [0, tokens + 70], kernel, f"size {size}")
    short = {k: x[:tokens] if k in ("q", "k", "v", "dt", "b") else x for k, x in d.items()}
    check_heads(cuda_lib, cfg, short, [0, tokens], kernel, f"size {size}, no value at all")


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("tokens", [64, 128, 171])
@pytest.mark.parametrize("name,value,last", [("b", -12.0, 20), ("b", -30.0, 20), ("b", -30.0, 12), ("v", 0.0, 12), ("v", 0.0, 20),
                                             ("b", -12.0, 1000), ("v", 1e-6, 20)])
@pytest.mark.parametrize("dt", [0.03, 0.1])
def test_a_tail_that_writes_next_to_nothing(cuda_lib, name, value, last, dt, tokens, kernel):
    """The state is then what earlier tokens of the chunk wrote, decayed by up to 2^-46 since."""
    cfg = ref.config(**HARD)
    d = steady(cfg, tokens, [-16.0, -16.0, -1.0, -4.0], dt, seed=tokens, h0=0.0)
    x = ref.values(d[name])
    x[-last:] = value
    d[name] = ref.store(x, cfg)
    check_heads(cuda_lib, cfg, d, [0, tokens], kernel, f"{name} {value} {last}")


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("size", [1e-3, 1e-5, 1e-7, 1e-9])
def test_small_keys(cuda_lib, size, kernel):
    """Keys far below the root of qk_eps (normalised) and as they are, with beta about one."""
    for norm in (True, False):
        cfg = ref.config(qk_norm=norm)
        d = ref.inputs(cfg, 200, 1, seed=7)
        d["h0"][:] = 0
        d["k"] = ref.store(size * ref.values(d["k"]), cfg)
        check_heads(cuda_lib, cfg, d, [0, 200], kernel, f"norm {norm} size {size}")


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("values", [0.0, 1.0])
@pytest.mark.parametrize("size", [1e-5, 1e-4, 1e-2, 10.0, 1e3, 1e5])
def test_keys_of_any_size_with_beta_to_match(cuda_lib, size, values, kernel):
    """beta |k|^2 of up to 1.9 with keys far from one in size, on a carried state, with and without values."""
    cfg = ref.config(qk_norm=False, beta_sigmoid=False)
    d = ref.inputs(cfg, 200, 1, seed=8)
    d["k"] = ref.store(size * ref.values(d["k"]), cfg)
    d["v"] = ref.store(values * ref.values(d["v"]), cfg)
    k2 = np.square(ref.values(d["k"]).reshape(200, 2, 128)).sum(-1).repeat(2, axis=1)
    d["b"] = ref.store(np.random.default_rng(1).uniform(0.1, 1.88, (200, 4)) / k2, cfg)
    check_heads(cuda_lib, cfg, d, [0, 200], kernel, f"size {size}")


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("kw", [{}, dict(headdim=128), dict(beta_scale=2.0), HARD], ids=str)
def test_every_head_within_a_millionth_of_its_state(cuda_lib, kw, kernel):
    """What is documented for ordinary inputs, heads of a thousandfold range of sizes, two sequences."""
    import torch
    cfg = ref.config(nheads=8, ngroups=2, **kw)
    cu = [0, 333, 1033]
    d = ref.inputs(cfg, cu[-1], 2, seed=11)
    if kw is HARD:
        d["dt"] = ref.store(0.05 * np.abs(ref.values(d["dt"])), cfg)
        d["dt_bias"] = np.zeros(8, np.float32)
    scale = 10.0 ** np.linspace(-2, 1, 8)
    v = ref.values(d["v"]).reshape(cu[-1], 8, -1) * scale[:, None]
    d["v"] = ref.store(v.reshape(cu[-1], -1), cfg)
    d["h0"] = (d["h0"] * scale[:, None, None]).astype(np.float32)
    check_heads(cuda_lib, cfg, d, cu, kernel, f"{kw}")
    _, h = run_packed(cuda_lib, cfg, on_gpu(d), cu, True, kernel)
    _, wh = ref.prefill(cfg, d, cu, True)
    err = np.sqrt(np.mean(np.square(host(h) - wh), axis=(2, 3)) / np.mean(np.square(wh), axis=(2, 3)))
    assert (err <= 1e-6).all(), err


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
def test_a_state_that_the_first_token_forgets(cuda_lib, kernel):
    """A state of 1e8 decays by e^-30 at the first token of a chunk: y is what the tokens of 1e-3 write."""
    cfg = ref.config(**HARD)
    d = steady(cfg, 150, [-100.0] * 4, 1e-4, seed=9, h0=1e8)
    for t in (0, 64):
        d["dt"][t] = ref.store(np.full(4, 0.3), cfg)
    d["v"] = ref.store(1e-3 * ref.values(d["v"]), cfg)
    check_heads(cuda_lib, cfg, d, [0, 150], kernel)


@pytest.mark.parametrize("kernel", [SIMT, TENSOR])
@pytest.mark.parametrize("headdim", [64, 128])
def test_the_largest_and_smallest_values(cuda_lib, headdim, kernel):
    """Keys along an axis, values and states within a factor of four of what bf16 and fp32 hold, and near 2^-90."""
    cfg = ref.config(headdim=headdim)
    d = ref.inputs(cfg, 100, 1, seed=12)
    k = np.zeros((100, 256))
    k[np.arange(100), np.arange(100) % 128] = k[np.arange(100), 128 + np.arange(100) % 128] = 3.0
    d["k"] = ref.store(k, cfg)
    x = ref.values(d["v"])
    for size in (8e37, 1e-27):
        d["v"] = ref.store(np.clip(x, -1, 1) * size, cfg)
        d["h0"] = (np.clip(d["h0"] / np.abs(d["h0"]).max(), -1, 1) * size).astype(np.float32)
        check_heads(cuda_lib, cfg, d, [0, 100], kernel, f"{size}")
