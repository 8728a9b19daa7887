"""What is measured of the gated delta rule and of the state cache in 8 bits.

The gated delta rule keeps, per batch row and head, a state S (headdim x dstate) and does per token
  alpha = exp(A_h clamp(softplus(dt + dt_bias_h)))     beta = sigmoid(b)
  k^ = k / sqrt(|k|^2 + eps)      q^ = q / (sqrt(|q|^2 + eps) sqrt(dstate))
  S <- alpha S + beta (v - alpha S k^) k^T             y = S q^
with q and k shared by the heads of a group.  A state cache holds fp32 states in blocks of 32
elements with one power-of-two scale each, the elements in e4m3 or in int8.

Where `own` is true, `run` calls this repository's entry points; otherwise it computes the same in
elementary torch operations.
"""
import math

import torch

own = False

N = 128            # state dimension (dstate)
QK_EPS = 1e-6
DT_MIN, DT_MAX = 1e-3, 1e-1


# ---- the cases ---------------------------------------------------------------------------------
def listed():
    return [
        # the 8k prefill of the 128-head layer: one long prompt
        dict(name="prefill_8k", op="prefill", batch=1, seqlen=8192, nheads=128, headdim=64, ngroups=8, dtype="bf16", carry=False),
        # the second part of two prompts whose first parts are done: an odd length, wide heads
        dict(name="prefill_wide_carry", op="prefill", batch=2, seqlen=1031, nheads=32, headdim=128, ngroups=16, dtype="bf16", carry=True),
        # the small fp32 workload
        dict(name="prefill_tiny_fp32", op="prefill", batch=1, seqlen=256, nheads=8, headdim=64, ngroups=1, dtype="f32", carry=False),
        # a scheduler's batch of prompts of 1 to 700 tokens
        dict(name="varlen_64", op="varlen", nseq=64, maxlen=700, nheads=128, headdim=64, ngroups=8, carry=False),
        # a few short ones, some of them continued, one empty
        dict(name="varlen_few", op="varlen", nseq=6, maxlen=90, nheads=16, headdim=64, ngroups=2, carry=True),
        # token generation: the batch of the decode workload
        dict(name="decode_64", op="decode", batch=64, nheads=128, headdim=64, ngroups=8, slots=False),
        # one user: latency counts
        dict(name="decode_1", op="decode", batch=1, nheads=128, headdim=64, ngroups=8, slots=False),
        # a running batch over a pool of states, padded with rows that have none
        dict(name="decode_pool", op="decode", batch=37, nheads=32, headdim=128, ngroups=16, slots=True),
        # all states of a running batch put away, and some brought back
        dict(name="store_64_e4m3", op="store", count=64, nheads=128, headdim=64, format="e4m3"),
        dict(name="store_3_int8", op="store", count=3, nheads=112, headdim=64, format="int8"),
        dict(name="load_64_int8", op="load", count=64, nheads=128, headdim=64, format="int8"),
        dict(name="load_1_e4m3", op="load", count=1, nheads=128, headdim=64, format="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _heads(rng):
    headdim = rng.choice((64, 64, 128))
    nheads = rng.choice((8, 16, 32, 64) if headdim == 128 else (8, 16, 32, 64, 112, 120, 128))
    groups = [g for g in (1, 2, 4, 8, 16) if nheads % g == 0 and nheads >= 2 * g]
    return dict(nheads=nheads, headdim=headdim, ngroups=rng.choice(groups))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "varlen", "decode", "store", "load"))
    h = _heads(rng)
    if op == "prefill":
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        most = 8192 * 128 * 64 // (h["nheads"] * h["headdim"])
        seqlen = _log_int(rng, 1, 1024 if dtype == "f32" else 8192)
        batch = max(1, min(_log_int(rng, 1, 8), most // seqlen))
        return dict(op=op, batch=batch, seqlen=seqlen, dtype=dtype, carry=rng.random() < 0.5, **h)
    if op == "varlen":
        return dict(op=op, nseq=_log_int(rng, 1, 64), maxlen=_log_int(rng, 2, 700), carry=rng.random() < 0.5, **h)
    if op == "decode":
        return dict(op=op, batch=_log_int(rng, 1, 64), slots=rng.random() < 0.5, **h)
    h.pop("ngroups")
    return dict(op=op, count=_log_int(rng, 1, 64), format=rng.choice(("e4m3", "int8")), **h)


# ---- inputs --------------------------------------------------------------------------------------
def _lengths(case, seed):
    """Lengths of 0 to maxlen tokens, spread evenly, a different order for each seed."""
    n, top = case["nseq"], case["maxlen"]
    r = torch.Generator().manual_seed(seed + 77)
    low = 0 if case["carry"] else 1
    lens = [max(low, top * (i + 1) // n if i % 5 else low) for i in range(n)]
    lens[-1] = top
    return [lens[i] for i in torch.randperm(n, generator=r).tolist()]


def _params(case, g, dev):
    H = case["nheads"]
    A = -torch.exp(torch.rand(H, generator=g, device=dev) * math.log(16.0))
    dt0 = torch.exp(math.log(1e-3) + torch.rand(H, generator=g, device=dev) * math.log(100.0))
    return A, dt0 + torch.log(-torch.expm1(-dt0))  # softplus(dt_bias) = dt0


def _tokens(shape, case, g, dev, dtype):
    """Rows as the layer's convolution and activation leave them, and the raw gates."""
    G, H, P = case["ngroups"], case["nheads"], case["headdim"]

    def act(width):
        x = torch.randn(*shape, width, generator=g, device=dev)
        return (x * torch.sigmoid(x)).to(dtype)

    q, k, v = act(G * N), act(G * N), act(H * P)
    dt, b = (torch.randn(*shape, H, generator=g, device=dev).to(dtype) for _ in range(2))
    return dict(q=q, k=k, v=v, dt=dt, b=b)


def _state(n, case, g, dev):
    """States of the size that some hundred tokens leave, heads of different sizes among them."""
    size = torch.exp(0.5 * torch.randn(n, case["nheads"], 1, 1, generator=g, device=dev))
    return 0.3 * size * torch.randn(n, case["nheads"], case["headdim"], N, generator=g, device=dev)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    s = dict(case=case)
    op = case["op"]
    if op in ("prefill", "varlen", "decode"):
        s["A"], s["dt_bias"] = _params(case, g, dev)
    if op == "prefill":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s.update(_tokens((case["batch"], case["seqlen"]), case, g, dev, dtype))
        s["h0"] = _state(case["batch"], case, g, dev) if case["carry"] else None
    elif op == "varlen":
        cu = [0]
        for n in _lengths(case, seed):
            cu.append(cu[-1] + n)
        s["cu"] = cu
        s.update(_tokens((cu[-1],), case, g, dev, torch.bfloat16))
        s["h0"] = _state(case["nseq"], case, g, dev) if case["carry"] else None
        lens = torch.tensor([b - a for a, b in zip(cu, cu[1:])], device=dev)
        at = torch.arange(max(1, max(b - a for a, b in zip(cu, cu[1:]))), device=dev)
        s["valid"] = at[None, :] < lens[:, None]  # [nseq, longest]
    elif op == "decode":
        B = case["batch"]
        s.update(_tokens((B,), case, g, dev, torch.bfloat16))
        n = B + B // 2 + 1 if case["slots"] else B
        s["state"] = _state(n, case, g, dev)
        s["slots"] = None
        if case["slots"]:  # every eighth row is padding
            slots = torch.randperm(n, generator=g, device=dev)[:B].to(torch.int32)
            slots[7::8] = -1
            s["slots"] = slots
        s["y"] = torch.zeros(B, case["nheads"] * case["headdim"], dtype=torch.bfloat16, device=dev)
    else:
        n = case["count"]
        pool = n + n // 4 + 1  # places in the cache
        kind = torch.float8_e4m3fn if case["format"] == "e4m3" else torch.int8
        shape = (case["nheads"], case["headdim"])
        s["slots"] = torch.randperm(pool, generator=g, device=dev)[:n].to(torch.int32)
        if op == "store":
            s["states"] = _state(n, case, g, dev)
            s["cache"] = torch.zeros(pool, *shape, N, dtype=torch.uint8, device=dev).view(kind)
            s["scales"] = torch.zeros(pool, *shape, N // 32, dtype=torch.uint8, device=dev)
        else:
            if case["format"] == "e4m3":
                s["cache"] = (100 * torch.randn(pool, *shape, N, generator=g, device=dev)).clamp(-448, 448).to(kind)
            else:
                s["cache"] = torch.randint(-127, 128, (pool, *shape, N), generator=g, device=dev, dtype=kind)
            s["scales"] = torch.randint(108, 125, (pool, *shape, N // 32), generator=g, device=dev, dtype=torch.uint8)
            s["states"] = torch.zeros(n, *shape, N, device=dev)
    return s


# ---- the plain forms -------------------------------------------------------------------------------
def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(x.clamp(max=20))))


def _plain_gates(dt, b, A, dt_bias):
    """(log of the decay, beta)."""
    step = _softplus(dt.double() + dt_bias.double()).clamp(DT_MIN, DT_MAX)
    return step * A.double(), torch.sigmoid(b.float())


def _plain_unit(x, G):
    x = x.float().unflatten(-1, (G, N))
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + QK_EPS)


def _plain_chunks(q, k, v, logdec, beta, h0):
    """q, k [B, L, H, N], v [B, L, H, P], logdec, beta [B, L, H] in chunks of 64 tokens: y [B, L, H, P]
    and the last state [B, H, P, N].  Within a chunk (I + L) U = beta (V - e^cs K S^T) with
    L_ij = beta_i e^{cs_i - cs_j} k_i.k_j for j < i, cs the chunk's prefix sums of logdec."""
    B, L, H, _ = q.shape
    P, C = v.shape[-1], 64
    nc = (L + C - 1) // C
    pad = nc * C - L

    def chunks(x):
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, pad))
        x = x.unflatten(1, (nc, C))  # [B, nc, C, H, ...]
        return x.movedim(3, 1)       # [B, H, nc, C, ...]

    qc, kc, vc, bc = chunks(q), chunks(k), chunks(v), chunks(beta)[..., None]
    cs = chunks(logdec).cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    dec = torch.exp((cs[..., :, None] - cs[..., None, :]).masked_fill_(~low, -math.inf)).float()
    left = (kc @ kc.transpose(-1, -2)) * dec * bc
    att = (qc @ kc.transpose(-1, -2)) * dec
    T = torch.eye(C, device=q.device).expand(B, H, nc, C, C).contiguous()
    for i in range(1, C):  # forward substitution, a row of every chunk at a time
        T[..., i, :i] = -(left[..., i : i + 1, :i] @ T[..., :i, :i]).squeeze(-2)
    from_start = torch.exp(cs).float()[..., None]
    to_end = torch.exp(cs[..., -1:] - cs).float()[..., None]
    S = h0.transpose(-1, -2).float() if h0 is not None else torch.zeros(B, H, N, P, device=q.device)
    y = torch.empty(B, H, nc, C, P, device=q.device)
    for c in range(nc):
        U = T[:, :, c] @ (bc[:, :, c] * (vc[:, :, c] - from_start[:, :, c] * (kc[:, :, c] @ S)))
        y[:, :, c] = from_start[:, :, c] * (qc[:, :, c] @ S) + att[:, :, c] @ U
        S = from_start[:, :, c, -1:] * S + (kc[:, :, c] * to_end[:, :, c]).transpose(-1, -2) @ U
    return y.flatten(2, 3)[:, :, :L].transpose(1, 2), S.transpose(-1, -2).contiguous()


def _plain_rule(s, q, k, v, dt, b, keep=None):
    """The rule over [B, L, ...] rows; tokens outside `keep` change nothing."""
    c = s["case"]
    G, H, P = c["ngroups"], c["nheads"], c["headdim"]
    logdec, beta = _plain_gates(dt, b, s["A"], s["dt_bias"])
    if keep is not None:
        logdec, beta = logdec * keep[..., None], beta * keep[..., None]
    q, k = (_plain_unit(x, G).repeat_interleave(H // G, dim=-2) for x in (q, k))
    return _plain_chunks(q / math.sqrt(N), k, v.float().unflatten(-1, (H, P)), logdec, beta, s["h0"])


def _plain_varlen(s):
    valid = s["valid"]

    def padded(x):
        p = torch.zeros(*valid.shape, x.shape[-1], dtype=x.dtype, device=x.device)
        p[valid] = x
        return p

    y, h = _plain_rule(s, *(padded(s[n]) for n in ("q", "k", "v", "dt", "b")), keep=valid)
    return y[valid], h


def _plain_decode(s):
    c = s["case"]
    G, H, P = c["ngroups"], c["nheads"], c["headdim"]
    rows = torch.arange(c["batch"], device="cuda") if s["slots"] is None else torch.nonzero(s["slots"] >= 0)[:, 0]
    at = rows if s["slots"] is None else s["slots"][rows].long()
    logdec, beta = _plain_gates(s["dt"][rows], s["b"][rows], s["A"], s["dt_bias"])
    q, k = (_plain_unit(s[n][rows], G).repeat_interleave(H // G, dim=-2)[..., None] for n in ("q", "k"))
    S = s["state"][at] * torch.exp(logdec).float()[..., None, None]
    u = beta[..., None, None] * (s["v"][rows].float().unflatten(-1, (H, P, 1)) - S @ k)
    S = S + u * k.transpose(-1, -2)
    s["state"][at] = S
    s["y"][rows] = (S @ (q / math.sqrt(N))).flatten(1).to(s["y"].dtype)
    return [s["y"], s["state"]]


def _plain_store(s):
    e4m3 = s["case"]["format"] == "e4m3"
    x = s["states"].unflatten(-1, (N // 32, 32))
    m, e = torch.frexp(x.abs().amax(-1))  # the largest is m 2^e with m in [1/2, 1)
    # the smallest power of two that brings it to 448 = 7/8 2^9, or to 127 = 127/128 2^7
    e = torch.where(m <= 0.875, e - 9, e - 8) if e4m3 else torch.where(m <= 127 / 128, e - 7, e - 6)
    e = e.clamp(min=-127)
    x = torch.ldexp(x.double(), -e[..., None])
    x = x.float().flatten(-2).to(torch.float8_e4m3fn) if e4m3 else torch.round(x).flatten(-2).to(torch.int8)
    at = s["slots"].long()
    s["cache"].view(torch.uint8)[at] = x.view(torch.uint8)
    s["scales"][at] = (e + 127).to(torch.uint8)
    return [s["cache"], s["scales"]]


def _plain_load(s):
    at = s["slots"].long()
    x = s["cache"].view(torch.uint8)[at].view(s["cache"].dtype).float().unflatten(-1, (N // 32, 32))
    e = s["scales"][at].to(torch.int32) - 127
    s["states"].copy_(torch.ldexp(x, e[..., None]).flatten(-2))
    return [s["states"]]


# ---- one pass ------------------------------------------------------------------------------------
def _config(case):
    return dict(batch=case.get("batch", 1), seqlen=case.get("seqlen", 1), nheads=case["nheads"], headdim=case["headdim"],
                dstate=N, ngroups=case["ngroups"], dtype=case.get("dtype", "bf16"), qk_norm=True, qk_eps=QK_EPS,
                q_scale=1.0 / math.sqrt(N), dt_min=DT_MIN, dt_max=DT_MAX)


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        from mamba_ssd_scan_02_b200 import ssd

        if op in ("prefill", "varlen", "decode") and "cfg" not in s:
            s["cfg"] = _config(s["case"])
        if op == "prefill":
            return list(ssd.delta_prefill(s["cfg"], s["q"], s["k"], s["v"], s["dt"], s["b"], s["A"], s["dt_bias"], s["h0"]))
        if op == "varlen":
            return list(ssd.delta_prefill_varlen(s["cfg"], s["cu"], s["q"], s["k"], s["v"], s["dt"], s["b"], s["A"], s["dt_bias"], s["h0"]))
        if op == "decode":
            ssd.delta_decode_step(s["cfg"], s["q"], s["k"], s["v"], s["dt"], s["b"], s["A"], s["dt_bias"], s["state"], s["slots"], y=s["y"])
            return [s["y"], s["state"]]
        if op == "store":
            ssd.state_store(s["states"], s["cache"], s["scales"], cache_slots=s["slots"])
            return [s["cache"], s["scales"]]
        ssd.state_load(s["cache"], s["scales"], s["states"], cache_slots=s["slots"])
        return [s["states"]]
    if op == "prefill":
        y, h = _plain_rule(s, *(s[n] for n in ("q", "k", "v", "dt", "b")))
        return [y.flatten(2).to(s["v"].dtype), h]
    if op == "varlen":
        y, h = _plain_varlen(s)
        return [y.flatten(1).to(s["v"].dtype), h]
    if op == "decode":
        return _plain_decode(s)
    return _plain_store(s) if op == "store" else _plain_load(s)


def work(case):
    op = case["op"]
    H, P = case["nheads"], case["headdim"]
    state = H * P * N
    if op in ("store", "load"):  # each state once in fp32, once in 8 bits with a scale per 32
        n = case["count"] * state
        return dict(bytes=n * (4 + 1 + 1 / 32) + 4 * case["count"], flops=2 * n)
    G = case["ngroups"]
    size = 4 if case.get("dtype") == "f32" else 2
    row = size * (2 * G * N + 2 * H * P + 2 * H)  # q, k, v, y and the gates of a token
    if op == "decode":
        rows = case["batch"] - (case["batch"] // 8 if case["slots"] else 0)
        return dict(bytes=rows * (row + 8 * state) + 8 * H, flops=7 * rows * state)
    if op == "prefill":
        tokens, seqs = case["batch"] * case["seqlen"], case["batch"]
    else:
        tokens, seqs = sum(_lengths(case, 0)), case["nseq"]
    return dict(bytes=tokens * row + seqs * state * (8 if case["carry"] else 4) + 8 * H, flops=7 * tokens * state)


# ---- the definition in 64 bits -----------------------------------------------------------------
def _exact_steps(case, s, q, k, v, dt, b, valid, S):
    """Token after token, as the rule is written down: [rows, steps, ...] inputs, S changed in place."""
    H, P, G = case["nheads"], case["headdim"], case["ngroups"]
    head = torch.arange(H, device=q.device) // (H // G)
    A, bias = s["A"].double(), s["dt_bias"].double()
    y = torch.zeros(q.shape[0], q.shape[1], H, P, dtype=torch.float64, device=q.device)
    for t in range(q.shape[1]):
        x = dt[:, t].double() + bias
        step = torch.logaddexp(x, torch.zeros_like(x)).clamp(DT_MIN, DT_MAX)
        live = valid[:, t, None].double()
        alpha = torch.exp(step * A * live)
        beta = live / (1 + torch.exp(-b[:, t].double()))
        kt = k[:, t].double().reshape(-1, G, N)
        qt = q[:, t].double().reshape(-1, G, N)
        kt = (kt / (kt.square().sum(-1, keepdim=True) + QK_EPS).sqrt())[:, head]
        qt = (qt / (qt.square().sum(-1, keepdim=True) + QK_EPS).sqrt())[:, head] / math.sqrt(N)
        S.mul_(alpha[..., None, None])
        u = beta[..., None] * (v[:, t].double().reshape(-1, H, P) - torch.einsum("bhpn,bhn->bhp", S, kt))
        S.addcmul_(u[..., None], kt[:, :, None, :])
        y[:, t] = torch.einsum("bhpn,bhn->bhp", S, qt)
    return y


def _exact_blocks(x, e4m3):
    """(elements, scale exponents) of the 32-element blocks of x, in 64 bits."""
    x = x.double().unflatten(-1, (N // 32, 32))
    top = x.abs().amax(-1, keepdim=True)
    limit = 448.0 if e4m3 else 127.0
    e = torch.ceil(torch.log2(top / limit)).clamp(min=-127, max=127)
    e = torch.where(top > limit * torch.exp2(e), e + 1, e)  # the logarithm's own rounding
    e = torch.where((top <= limit * torch.exp2(e - 1)) & (e > -127), e - 1, e)
    x = x / torch.exp2(e)
    if e4m3:  # three bits after the leading one, down to steps of 2^-9
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0**-6))) - 3)
        return (torch.round(x / step) * step).flatten(-2), e[..., 0]
    return torch.round(x).flatten(-2), e[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    H, P = case["nheads"], case["headdim"]
    if op == "prefill":
        B, L = case["batch"], case["seqlen"]
        S = s["h0"].double() if s["h0"] is not None else torch.zeros(B, H, P, N, dtype=torch.float64, device="cuda")
        y = _exact_steps(case, s, *(s[n] for n in ("q", "k", "v", "dt", "b")), torch.ones(B, L, device="cuda"), S)
        return [y.reshape(B, L, H * P), S]
    if op == "varlen":
        n = case["nseq"]
        S = s["h0"].double() if s["h0"] is not None else torch.zeros(n, H, P, N, dtype=torch.float64, device="cuda")
        start = torch.tensor(s["cu"][:-1], device="cuda")
        valid = s["valid"]
        row = (start[:, None] + torch.arange(valid.shape[1], device="cuda")).clamp(max=max(0, s["cu"][-1] - 1))
        y = _exact_steps(case, s, *(s[x][row] for x in ("q", "k", "v", "dt", "b")), valid, S)
        return [y[valid].reshape(-1, H * P), S]
    if op == "decode":
        live = list(range(case["batch"])) if s["slots"] is None else [i for i, x in enumerate(s["slots"].tolist()) if x >= 0]
        at = torch.tensor(live if s["slots"] is None else s["slots"][live].tolist(), device="cuda")
        state, y = s["state"].double(), s["y"].double()
        S = state[at]
        got = _exact_steps(case, s, *(s[n][live][:, None] for n in ("q", "k", "v", "dt", "b")), torch.ones(len(live), 1, device="cuda"), S)
        state[at] = S
        y[live] = got.reshape(len(live), H * P)
        return [y, state]
    at = s["slots"].long()
    if op == "store":
        x, e = _exact_blocks(s["states"], case["format"] == "e4m3")
        cache = s["cache"].double()
        cache[at] = x
        scales = s["scales"].clone()
        scales[at] = (e + 127).to(torch.uint8)
        return [cache if case["format"] == "e4m3" else cache.to(torch.int8), scales]
    x = s["cache"].double()[at].unflatten(-1, (N // 32, 32)) * torch.exp2(s["scales"][at].double() - 127)[..., None]
    return [x.flatten(-2)]
