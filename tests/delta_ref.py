"""The gated delta rule and the 8-bit state cache in fp64 numpy, written from their definitions, and
the inputs that their tests draw."""
from __future__ import annotations

import math

import numpy as np

from mamba_ssd_scan_02_b200 import datagen


def config(**kw):
    c = dict(nheads=4, headdim=64, dstate=128, ngroups=2, dtype="bf16", dt_min=1e-3, dt_max=1e-1)
    c.update(kw)
    return c


def values(a):
    """Stored numbers (uint16 = bf16 bits) as float64."""
    return datagen.bf16_value(a).astype(np.float64) if a.dtype == np.uint16 else a.astype(np.float64)


def store(a, cfg):
    return datagen.bf16_bits(a.astype(np.float32)) if cfg["dtype"] == "bf16" else a.astype(np.float32)


def inputs(cfg, rows, n_states, seed=0, scale=1.0):
    """q, k, v, dt, b [rows, width] in the io dtype, A, dt_bias, and states [n_states, H, P, N]."""
    r = np.random.default_rng(seed)
    H, P, N, G = cfg["nheads"], cfg["headdim"], cfg["dstate"], cfg["ngroups"]

    def act(width):
        x = r.standard_normal((rows, width))
        return x / (1 + np.exp(-x))

    d = {n: store(act(w), cfg) for n, w in (("q", G * N), ("k", G * N))}
    d["v"] = store(scale * act(H * P), cfg)
    d.update({n: store(r.standard_normal((rows, H)), cfg) for n in ("dt", "b")})
    p = datagen.head_params(seed + 5, H)
    d["A"], d["dt_bias"] = p["A"], p["dt_bias"]
    d["h0"] = (scale * 0.3 * r.standard_normal((n_states, H, P, N))).astype(np.float32)
    return d


def rule(cfg, d, rows, S):
    """The recurrence over the token rows `rows` of d from the state S [H, P, N] (float64, changed in
    place); returns y [len(rows), H*P]."""
    H, P, N, G = cfg["nheads"], cfg["headdim"], cfg["dstate"], cfg["ngroups"]
    eps, norm = cfg.get("qk_eps", 1e-6), cfg.get("qk_norm", True)
    q_scale = cfg.get("q_scale", 1 / math.sqrt(N))
    A, bias = d["A"].astype(np.float64), d["dt_bias"].astype(np.float64)
    y = np.zeros((len(rows), H * P))
    for i, t in enumerate(rows):
        q, k = (values(d[n][t]).reshape(G, N) for n in ("q", "k"))
        if norm:
            q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True) + eps) for x in (q, k))
        q, k = (np.repeat(x, H // G, axis=0) for x in (q * q_scale, k))
        x = values(d["dt"][t]) + bias
        dt = np.logaddexp(x, 0) if cfg.get("dt_softplus", True) else x
        dt = np.clip(dt, cfg.get("dt_min", 0.0), cfg.get("dt_max", math.inf))
        b = values(d["b"][t])
        beta = cfg.get("beta_scale", 1.0) * (1 / (1 + np.exp(-b)) if cfg.get("beta_sigmoid", True) else b)
        S *= np.exp(A * dt)[:, None, None]
        u = beta[:, None] * (values(d["v"][t]).reshape(H, P) - np.einsum("hpn,hn->hp", S, k))
        S += u[:, :, None] * k[:, None, :]
        y[i] = np.einsum("hpn,hn->hp", S, q).reshape(-1)
    return y


def prefill(cfg, d, cu, h0=True):
    """Packed sequences cu: y [rows, H*P] and the final states [nseq, H, P, N]."""
    H, P, N = cfg["nheads"], cfg["headdim"], cfg["dstate"]
    n = len(cu) - 1
    S = d["h0"][:n].astype(np.float64) if h0 else np.zeros((n, H, P, N))
    y = [rule(cfg, d, range(cu[i], cu[i + 1]), S[i]) for i in range(n)]
    return np.concatenate(y) if y else np.zeros((0, H * P)), S


def check_state(got, want, tokens, what):
    """A step adds, to each element, the rounding of a sum of N products to fp32, under 32 units of
    2^-24 of the largest (the chunked kernel: operands of 22 bits, sums of 64 to 128 products); the
    transition does not expand errors, and independent ones add up like the root of their
    number."""
    got, want = np.asarray(got, np.float64), np.asarray(want)
    assert np.all(np.isfinite(got)), what
    bound = 32 * 2.0 ** -24 * math.sqrt(tokens + 1) * max(np.abs(want).max(), 1e-30)
    err = np.abs(got - want).max()
    assert err <= bound, f"{what}: state off by {err:.3e} > {bound:.3e}"


def check_y(got, want, cfg, chunked, tokens, what):
    """fp32: as the state.  bf16: one rounding (2^-8 of the value) on top of the products' error; the
    chunked kernel's in-chunk products round four factors to 11 bits (2^-11 of a sum's root mean square
    each, at up to five standard deviations: 1e-2 of the output's root mean square)."""
    got, want = np.asarray(got, np.float64), np.asarray(want)
    assert np.all(np.isfinite(got)), what
    rms = math.sqrt(np.mean(want * want)) if want.size else 0.0
    err = np.abs(got - want)
    if cfg["dtype"] == "bf16":
        bound = 2.0 ** -8 * np.abs(want) + (1e-2 if chunked else 1e-4) * rms
    else:
        bound = np.full(want.shape, 32 * 2.0 ** -24 * math.sqrt(tokens + 1) * max(np.abs(want).max(initial=0), 1e-30))
    worst = (err - bound).max(initial=-1)
    assert worst <= 0, f"{what}: y beyond its bound by {worst:.3e} (rms {rms:.3e})"


# ---- state cache -------------------------------------------------------------------------------
def e4m3_value(byte):
    s, e, m = byte >> 7, (byte >> 3) & 15, byte & 7
    v = math.nan if (e == 15 and m == 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if s else v


E4M3 = np.array([e4m3_value(i) for i in range(256)])


def cache_blocks(x, fmt):
    """(element values, scale bytes) of fp32 x [..., N]: exact arithmetic in float64."""
    x = x.astype(np.float64).reshape(*x.shape[:-1], -1, 32)
    top = np.abs(x).max(-1)
    limit = 448.0 if fmt == "e4m3" else 127.0
    bad = ~np.isfinite(top)
    e = np.full(top.shape, -127)
    for _ in range(260):  # the smallest power of two that holds the block
        e = np.where(~bad & (top > limit * np.exp2(e.astype(np.float64))), e + 1, e)
    scaled = np.where(bad[..., None], 0.0, x) * np.exp2(-e.astype(np.float64))[..., None]
    if fmt == "int8":
        q = np.round(scaled)  # ties to even
    else:
        pos = np.sort(np.unique(np.abs(E4M3[:127])))  # 0 .. 448, in the order of their codes
        a = np.abs(scaled)
        hi = np.clip(np.searchsorted(pos, a), 0, len(pos) - 1)
        lo = np.maximum(hi - 1, 0)
        up = (pos[hi] - a < a - pos[lo]) | ((pos[hi] - a == a - pos[lo]) & (hi % 2 == 0))
        q = np.copysign(np.where(up, pos[hi], pos[lo]), scaled)
    return q.reshape(*q.shape[:-2], -1), np.where(bad, 255, e + 127).astype(np.uint8)
