"""The state-space mixer's operators: what is measured, and their plain forms.

Four groups, as a model's mixer uses them: the short causal convolution, the
selective state-space scan, the RMS norm with the residual's addition and an
8-bit output, and 8-bit activation checkpoints with the backward passes that
read them.  Per-token tensors are time-major, [B, T, D]; parameters, states and
their gradients are fp32 (the convolution's state holds raw inputs and has
their type).

    conv:  p_t = bias + sum_j w[:, j] x_{t-W+1+j},  y = p sigmoid(p)  (or p)
    scan:  dt = softplus(delta + dt_bias),  h_t = exp(dt A) h_{t-1} + dt u_t B_t,
           y_t = (C_t . h_t + D u_t) z_t sigmoid(z_t)
    norm:  s = x + residual,  y = weight s / sqrt(mean(s^2) + eps)
    act8:  per row and 128 channels, scale = the least power of two >= amax / 448
           (at least 2^-117), code = e4m3(x / scale)

``own`` False computes these with elementary torch operations, True through
the library.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # a batch of long prompts through the convolution, at the library's prefill shape (8 x 4096 tokens, 32 heads of 64 channels)
        {"name": "conv-prompt", "kind": "conv", "dtype": "bf16", "B": 8, "T": 4096, "D": 2048, "W": 4, "silu": True, "ragged": False},
        # right-padded prompts of odd sizes that continue earlier ones, x a slice of a wider projection (fp32, no activation)
        {"name": "conv-ragged", "kind": "conv", "dtype": "f32", "B": 5, "T": 2999, "D": 531, "W": 3, "silu": False, "ragged": True},
        # one token for each of 256 sequences, at the library's decode shape (40 heads of 64 channels)
        {"name": "conv-step", "kind": "conv_step", "dtype": "bf16", "B": 256, "D": 2560, "W": 4, "silu": True},
        # a training step of the convolution whose input is kept in 8 bits: forward, recomputation and gradients from the codes
        {"name": "conv-train8", "kind": "conv_train8", "dtype": "bf16", "B": 8, "T": 4096, "D": 2048, "W": 4, "silu": True},
        # a batch of long prompts through the scan
        {"name": "scan-prompt", "kind": "scan", "dtype": "bf16", "B": 8, "T": 4096, "D": 2048, "N": 16, "G": 1, "ragged": False},
        # one long document (the library's long-context shape): few channels, so time itself is split
        {"name": "scan-long", "kind": "scan", "dtype": "bf16", "B": 1, "T": 65536, "D": 2048, "N": 16, "G": 1, "ragged": False},
        # right-padded prompts of odd sizes in fp32, two groups, continuing from a state
        {"name": "scan-ragged", "kind": "scan", "dtype": "f32", "B": 3, "T": 1021, "D": 202, "N": 8, "G": 2, "ragged": True},
        # one token for each of 256 sequences
        {"name": "scan-step", "kind": "scan_step", "dtype": "bf16", "B": 256, "D": 2560, "N": 16, "G": 1},
        # a training step of the scan: forward that keeps its states, and every gradient
        {"name": "scan-train", "kind": "scan_train", "dtype": "bf16", "B": 4, "T": 4096, "D": 2048, "N": 16, "G": 1},
        # the norm in front of a projection in 8 bits: a decode batch
        {"name": "norm8-tokens", "kind": "norm8", "dtype": "bf16", "rows": 256, "D": 2560},
        # and a batch of prompts
        {"name": "norm8-prompt", "kind": "norm8", "dtype": "bf16", "rows": 32768, "D": 2048},
        # a training step of the norm with its input kept in 8 bits
        {"name": "norm-train8", "kind": "norm_train8", "dtype": "bf16", "rows": 32768, "D": 2048},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["conv", "conv_step", "conv_train8", "scan", "scan", "scan_step", "scan_train", "scan_train", "norm8", "norm_train8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = _log(rng, 33, 4096)
    if rng.random() < 0.6:
        D = max(64, D // 64 * 64)                   # whole heads, else any width
    if kind in ("norm8", "norm_train8"):
        D = min(4 * D, 12288)
        return {"kind": kind, "dtype": dtype, "rows": _log(rng, 1, max(1, 30_000_000 // D)), "D": D}
    if kind == "conv_step":
        return {"kind": kind, "dtype": dtype, "B": _log(rng, 1, 512), "D": D, "W": rng.choice([2, 3, 4]), "silu": rng.random() < 0.7}
    if kind in ("conv", "conv_train8"):
        B = _log(rng, 1, 16)
        T = _log(rng, 1, max(1, min(65536, 30_000_000 // (B * D))))
        case = {"kind": kind, "dtype": dtype, "B": B, "T": T, "D": D, "W": rng.choice([2, 3, 4]), "silu": rng.random() < 0.7}
        return {**case, "ragged": rng.random() < 0.4} if kind == "conv" else case
    N = rng.choice([16, 16, 16, 8, 5, 32, 64])
    G = rng.choice([1, 1, 2]) if D % 2 == 0 else 1
    if kind == "scan_step":
        return {"kind": kind, "dtype": dtype, "B": _log(rng, 1, 512 * 16 // max(N, 16)), "D": D, "N": N, "G": G}
    B = _log(rng, 1, 16)
    most = 10_000_000 * 16 // max(N, 16)
    T = _log(rng, 1, max(1, min(8192, most // (B * D))))
    case = {"kind": kind, "dtype": dtype, "B": B, "T": T, "D": D, "N": N, "G": G}
    return {**case, "ragged": rng.random() < 0.4} if kind == "scan" else case


# ---- inputs -------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _DT[case["dtype"]]
    kind = case["kind"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)

    def wide(B, T, D, std=1.0):                     # a slice of a wider projection's output, as a model has it
        return normal(B, T, D + 48, std=std)[..., 24:24 + D]

    s = {"case": dict(case)}
    if kind in ("norm8", "norm_train8"):
        R, D = case["rows"], case["D"]
        s["x"] = normal(R, D)
        s["residual"] = normal(R, D, std=2.0)
        s["weight"] = 1.0 + normal(D, std=0.2, dtype=torch.float32)
        if kind == "norm_train8":
            s["dy"] = normal(R, D)
            s["dresidual"] = normal(R, D)
        return s
    B, D = case["B"], case["D"]
    lens = None
    if case.get("ragged"):
        lens = torch.randint(0, case["T"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        lens[0] = case["T"]
    if kind in ("conv", "conv_step", "conv_train8"):
        W = case["W"]
        s["weight"] = normal(D, W, std=W ** -0.5, dtype=torch.float32)
        s["bias"] = normal(D, std=0.1, dtype=torch.float32)
        if kind == "conv_step":
            s["x"] = normal(B, D)
            s["state"] = normal(B, W - 1, D)
            return s
        T = case["T"]
        s["x"] = wide(B, T, D) if case.get("ragged") else normal(B, T, D)
        s["state"] = normal(B, W - 1, D) if case.get("ragged") else None
        s["lens"] = lens
        if case.get("ragged"):
            s["out"] = torch.zeros(B, T, D, dtype=dt, device="cuda")    # rows behind a sequence's end stay as they are
        if kind == "conv_train8":
            s["dy"] = normal(B, T, D)
        return s
    N, G = case["N"], case["G"]
    T = case.get("T", 1)
    # decay rates 1..N with a spread, time steps log-uniform in [0.001, 0.1] before the token's own part
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(D, N, std=0.2, dtype=torch.float32))
    step = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["D"] = 1.0 + normal(D, std=0.1, dtype=torch.float32)
    s["u"] = normal(B, T, D)
    s["delta"] = normal(B, T, D, std=0.7)
    s["z"] = wide(B, T, D)
    bc = normal(B, T, 2 * G * N + 16)               # B and C are slices of one small projection
    s["B"] = bc[..., 8:8 + G * N].unflatten(-1, (G, N))
    s["C"] = bc[..., 8 + G * N:8 + 2 * G * N].unflatten(-1, (G, N))
    s["state"] = normal(B, D, N, dtype=torch.float32) if case.get("ragged") or kind == "scan_step" else None
    s["lens"] = lens
    if kind == "scan_step":
        for k in ("u", "delta", "z", "B", "C"):
            s[k] = s[k][:, 0]
    if case.get("ragged"):
        s["out"] = torch.zeros(B, T, D, dtype=dt, device="cuda")
    if kind == "scan_train":
        s["dy"] = normal(B, T, D)
    return s


# ---- one pass -----------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state["case"]["kind"], state)


def _run_own(kind, s):
    from linear_rnn_sequence_wkv7_b200 import ssm
    c = s["case"]
    dt = _DT[c["dtype"]]
    if kind == "conv":
        return ssm.conv_forward(s["x"], s["weight"], s["bias"], s["state"], silu=c["silu"], lens=s["lens"], y=s.get("out"),
                                return_state=True)
    if kind == "conv_step":
        return ssm.conv_step(s["x"], s["weight"], s["bias"], s["state"], silu=c["silu"]), s["state"]
    if kind == "conv_train8":
        y, kept = ssm.conv_forward(s["x"], s["weight"], s["bias"], silu=c["silu"], save8=True)
        again = ssm.conv_forward(kept, s["weight"], s["bias"], silu=c["silu"], y_dtype=dt)
        dx, dw, db, _ = ssm.conv_backward(kept, s["weight"], s["bias"], s["dy"], silu=c["silu"], grad_dtype=dt)
        return y, again, dx, dw, db
    if kind == "scan":
        return ssm.ssm_forward(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["state"],
                               lens=s["lens"], y=s.get("out"))
    if kind == "scan_step":
        return ssm.ssm_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["state"], s["D"], s["z"], s["dt_bias"]), s["state"]
    if kind == "scan_train":
        y, hT, kept = ssm.ssm_forward_train(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"])
        grads = ssm.ssm_backward(s["u"], s["delta"], s["A"], s["B"], s["C"], s["dy"], s["D"], s["z"], s["dt_bias"],
                                 states=kept, grad_dtype=dt)
        return (y, hT) + tuple(grads)
    if kind == "norm8":
        o = ssm.rmsnorm_forward(s["x"], s["weight"], s["residual"], eps=EPS, out8=True)
        return ssm.act8_load(o.y, torch.bfloat16), o.residual
    o = ssm.rmsnorm_forward(s["x"], s["weight"], s["residual"], eps=EPS, save8=True)
    dx, dw = ssm.rmsnorm_backward(s["dy"], o.saved, o.rstd, s["weight"], dresidual=s["dresidual"], grad_dtype=dt)
    return o.y, o.residual, dx, dw


def _run_plain(kind, s):
    c = s["case"]
    dt = _DT[c["dtype"]]
    if kind == "conv":
        y, st = _conv(s["x"].float(), s["weight"], s["bias"], None if s["state"] is None else s["state"].float(), c["silu"], s["lens"])
        y, st = y.to(dt), st.to(dt)
        if "out" in s:
            live = torch.arange(c["T"], device="cuda")[None, :, None] < s["lens"][:, None, None]
            y = s["out"].copy_(torch.where(live, y, s["out"]))
        return y, st
    if kind == "conv_step":
        y, st = _conv(s["x"].float()[:, None], s["weight"], s["bias"], s["state"].float(), c["silu"], None)
        s["state"].copy_(st)
        return y[:, 0].to(dt), s["state"]
    if kind == "conv_train8":
        y, _ = _conv(s["x"].float(), s["weight"], s["bias"], None, c["silu"], None)
        kept = _act8(s["x"].float())
        again, _ = _conv(kept, s["weight"], s["bias"], None, c["silu"], None)
        dx, dw, db = _conv_grad(kept, s["weight"], s["bias"], s["dy"].float(), c["silu"])
        return y.to(dt), again.to(dt), dx.to(dt), dw, db
    if kind == "scan":
        y, h = _scan(s)
        y = y.to(dt)
        if "out" in s:
            live = torch.arange(c["T"], device="cuda")[None, :, None] < s["lens"][:, None, None]
            y = s["out"].copy_(torch.where(live, y, s["out"]))
        return y, h
    if kind == "scan_step":
        one = {**s, "lens": None, **{k: s[k][:, None] for k in ("u", "delta", "z", "B", "C")}}
        y, h = _scan(one)
        s["state"].copy_(h)
        return y[:, 0].to(dt), s["state"]
    if kind == "scan_train":
        y, h, starts = _scan(s, keep=True)
        g = _scan_grad(s, starts)
        return (y.to(dt), h, g["u"].to(dt), g["delta"].to(dt), g["A"], g["B"].to(dt), g["C"].to(dt), g["D"], g["z"].to(dt), g["dt_bias"],
                g["state"])
    r = s["x"].float() + s["residual"].float()
    rstd = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    y = r * rstd * s["weight"]
    if kind == "norm8":
        return _act8(y).to(torch.bfloat16), r.to(dt)
    # the kept codes round the sum once: a sum next to a border between two codes needs its exact value
    xh = _act8(s["x"].double() + s["residual"].double()).float() * rstd
    wdy = s["weight"] * s["dy"].float()
    dx = s["dresidual"].float() + rstd * (wdy - xh * (wdy * xh).mean(-1, keepdim=True))
    return y.to(dt), r.to(dt), dx.to(dt), (s["dy"].float() * xh).sum(0, dtype=torch.float64).float()


# ---- the plain forms (32 bits) ----------------------------------------------------

def _act8(x):
    """The values that x's 8-bit codes stand for."""
    D = x.shape[-1]
    pad = -D % 128
    b = torch.nn.functional.pad(x, (0, pad)).unflatten(-1, (-1, 128))
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))          # amax = m 2^e, 448 = 0.875 * 2^9
    k = torch.where(m > 0, e - 9 + (m > 0.875).to(e.dtype), -117).clamp_min(-117)
    one = torch.ones_like(m)
    scale = torch.ldexp(one, k)
    q = b / scale
    step = torch.ldexp(one, torch.frexp(q)[1].clamp_min(-5) - 4)   # four significant bits, subnormals below 2^-6
    v = torch.round(q / step) * step * scale
    return v.flatten(-2)[..., :D]


def _conv(x, w, bias, state, silu, lens):
    B, T, D = x.shape
    W = w.shape[1]
    past = torch.zeros(B, W - 1, D, device=x.device) if state is None else state
    full = torch.cat([past, x], 1)
    p = bias + sum(w[:, j] * full[:, j:j + T] for j in range(W))
    if lens is None:
        st = full[:, T:]
    else:
        at = lens.long()[:, None] + torch.arange(W - 1, device=x.device)
        st = full.gather(1, at[..., None].expand(-1, -1, D))
    return (p * torch.sigmoid(p) if silu else p), st


def _conv_grad(x, w, bias, dy, silu):
    B, T, D = x.shape
    W = w.shape[1]
    full = torch.cat([torch.zeros(B, W - 1, D, device=x.device), x], 1)
    dp = dy
    if silu:
        p = bias + sum(w[:, j] * full[:, j:j + T] for j in range(W))
        sg = torch.sigmoid(p)
        dp = dy * sg * (1 + p * (1 - sg))
    dfull = torch.zeros_like(full)
    for j in range(W):
        dfull[:, j:j + T] += w[:, j] * dp
    dw = torch.stack([(dp * full[:, j:j + T]).sum((0, 1), dtype=torch.float64) for j in range(W)], 1).float()
    return dfull[:, W - 1:], dw, dp.sum((0, 1), dtype=torch.float64).float()


def _steps(s):
    """dt [B,T,D] and the softplus's derivative; dt = 0 behind a sequence's end keeps the state."""
    x = s["delta"].float() + s["dt_bias"]
    dt = x.clamp_min(0) + torch.log1p(torch.exp(-x.abs()))
    if s["lens"] is not None:
        dt = dt * (torch.arange(dt.shape[1], device=dt.device)[None, :, None] < s["lens"][:, None, None])
    return dt, torch.sigmoid(x)


def _piece(B, D, N):
    return max(1, min(128, (1 << 25) // (B * D * N)))


def _spread(v, D):
    """[B,L,G,N] -> [B,L,D,N]: each channel its group's row."""
    return v.float().repeat_interleave(D // v.shape[2], 2)


def _scan(s, keep=False):
    u = s["u"].float()
    dt, _ = _steps(s)
    Bn, T, D = u.shape
    N = s["A"].shape[1]
    h = torch.zeros(Bn, D, N, device=u.device) if s["state"] is None else s["state"]
    L = _piece(Bn, D, N)
    ys, starts = [], []
    for t0 in range(0, T, L):
        starts.append(h)
        d = dt[:, t0:t0 + L]
        a = torch.exp(d[..., None] * s["A"])
        b = (d * u[:, t0:t0 + L])[..., None] * _spread(s["B"][:, t0:t0 + L], D)
        hs = []
        for t in range(a.shape[1]):
            h = torch.addcmul(b[:, t], a[:, t], h)
            hs.append(h)
        ys.append((torch.stack(hs, 1) * _spread(s["C"][:, t0:t0 + L], D)).sum(-1))
    z = s["z"].float()
    y = (torch.cat(ys, 1) + s["D"] * u) * z * torch.sigmoid(z)
    return (y, h, starts) if keep else (y, h)


def _scan_grad(s, starts):
    u, z, dy = s["u"].float(), s["z"].float(), s["dy"].float()
    dt, slope = _steps(s)
    A = s["A"]
    Bn, T, D = u.shape
    N, G = A.shape[1], s["B"].shape[2]
    L = _piece(Bn, D, N)
    sg = torch.sigmoid(z)
    ds = dy * z * sg
    carry = torch.zeros(Bn, D, N, device=u.device)
    dA = torch.zeros(D, N, device=u.device, dtype=torch.float64)
    du, ddt, dB, dC, core = [], [], [], [], []
    for i in range(len(starts) - 1, -1, -1):
        t0 = i * L
        cut = slice(t0, min(T, t0 + L))
        d, uu, Bx, Cx = dt[:, cut], u[:, cut], _spread(s["B"][:, cut], D), _spread(s["C"][:, cut], D)
        a = torch.exp(d[..., None] * A)
        b = (d * uu)[..., None] * Bx
        h, hs = starts[i], [starts[i]]
        for t in range(a.shape[1]):
            h = torch.addcmul(b[:, t], a[:, t], h)
            hs.append(h)
        hs = torch.stack(hs, 1)
        own_part = Cx * ds[:, cut][..., None]
        gs = []
        for t in range(a.shape[1] - 1, -1, -1):
            g = own_part[:, t] + carry
            gs.append(g)
            carry = a[:, t] * g
        g = torch.stack(gs[::-1], 1)
        gb = (g * Bx).sum(-1)
        pg = a * hs[:, :-1] * g
        du.append(d * gb)
        ddt.append(uu * gb + (pg * A).sum(-1))
        dA += (pg * d[..., None]).sum((0, 1), dtype=torch.float64)
        dB.append((g * (d * uu)[..., None]).unflatten(2, (G, -1)).sum(3))
        dC.append((hs[:, 1:] * ds[:, cut][..., None]).unflatten(2, (G, -1)).sum(3))
        core.append((hs[:, 1:] * Cx).sum(-1))
    du, ddt, dB, dC, core = (torch.cat(v[::-1], 1) for v in (du, ddt, dB, dC, core))
    dx = ddt * slope
    return {"u": du + s["D"] * ds, "delta": dx, "A": dA.float(), "B": dB, "C": dC, "D": (ds * u).sum((0, 1), dtype=torch.float64).float(),
            "z": dy * (core + s["D"] * u) * sg * (1 + z * (1 - sg)), "dt_bias": dx.sum((0, 1), dtype=torch.float64).float(), "state": carry}


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    kind = case["kind"]
    e = 2 if case["dtype"] == "bf16" else 4
    if kind in ("norm8", "norm_train8"):
        n = case["rows"] * case["D"]
        q = 1 + 4 / 128
        if kind == "norm8":     # x, residual -> residual, codes
            return {"bytes": n * (3 * e + q) + 4 * case["D"], "flops": 6 * n}
        # x, residual -> y, residual, codes; then dy, dresidual, codes -> dx
        return {"bytes": n * (4 * e + q) + n * (3 * e + q) + 12 * case["D"], "flops": 16 * n}
    B, D, T = case["B"], case["D"], case.get("T", 1)
    n = B * T * D
    if kind in ("conv", "conv_step", "conv_train8"):
        W = case["W"]
        small = 4 * D * (W + 1)
        if kind == "conv":
            return {"bytes": n * 2 * e + 2 * B * (W - 1) * D * e + small, "flops": n * (2 * W + 4)}
        if kind == "conv_step":
            return {"bytes": n * 2 * e + 2 * B * (W - 1) * D * e + small, "flops": n * (2 * W + 4)}
        q = 1 + 4 / 128     # x -> y, codes; codes -> y; codes, dy -> dx
        return {"bytes": n * (2 * e + q) + n * (q + e) + n * (q + 2 * e) + 3 * small, "flops": n * (6 * W + 20)}
    N, G = case["N"], case["G"]
    bc = 2 * B * T * G * N * e
    par = 4 * D * (N + 2)
    if kind == "scan":
        return {"bytes": n * 4 * e + bc + par + 4 * B * D * N * (2 if case.get("ragged") else 1), "flops": n * (7 * N + 10)}
    if kind == "scan_step":
        return {"bytes": n * 4 * e + bc + par + 8 * B * D * N, "flops": n * (7 * N + 10)}
    # forward (u, delta, z -> y), then u, delta, z, dy -> du, ddelta, dz, with B, C twice and their gradients once
    return {"bytes": n * 11 * e + 3 * bc + 3 * par + 8 * B * D * N, "flops": n * (7 * N + 10) + n * (26 * N + 30)}


# ---- the definitions in 64 bits -----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if kind in ("norm8", "norm_train8"):
        return _exact_norm(kind, s)
    if kind.startswith("conv"):
        return _exact_conv(kind, s)
    return _exact_scan(kind, s)


def _exact8(x):
    shape = x.shape
    D = shape[-1]
    out = torch.empty_like(x)
    for c in range(0, D, 128):
        part = x[..., c:c + 128]
        top = part.abs().max(-1, keepdim=True).values
        scale = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp_min(-117))
        q = part / scale
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)    # three bits behind the leading one
        out[..., c:c + 128] = torch.round(q / step) * step * scale
    return out


def _exact_norm(kind, s):
    r = s["x"] + s["residual"]
    w = s["weight"]
    inv = (torch.linalg.vector_norm(r, dim=-1, keepdim=True) ** 2 / r.shape[-1] + EPS) ** -0.5
    y = w * (r * inv)
    if kind == "norm8":
        return _exact8(y), r
    kept = _exact8(r)
    G = s["dy"] * w
    inner = torch.einsum("rd,rd->r", G, kept)[:, None]
    dx = s["dresidual"] + inv * G - inv ** 3 * kept * inner / r.shape[-1]
    return y, r, dx, torch.einsum("rd,rd->d", s["dy"], kept * inv)


def _exact_conv(kind, s):
    c = s["case"]
    W = c["W"]
    x = s["x"][:, None] if kind == "conv_step" else s["x"]
    B, T, D = x.shape
    past = s.get("state")
    past = x.new_zeros(B, W - 1, D) if past is None else past

    def act(p):
        return p / (1 + torch.exp(-p)) if c["silu"] else p

    def slope(p):
        if not c["silu"]:
            return torch.ones_like(p)
        q = 1 / (1 + torch.exp(-p))
        return q + p * q * (1 - q)

    def pre(v):             # [B,T,D] from windows of W tokens
        return torch.einsum("btdw,dw->btd", torch.cat([past, v], 1).unfold(1, W, 1), s["weight"]) + s["bias"]

    if kind == "conv_step":
        return act(pre(x))[:, 0], torch.cat([past, x], 1)[:, 1:]
    if kind == "conv":
        y = act(pre(x))
        rows = torch.cat([past, x], 1)
        n = [T] * B if s["lens"] is None else s["lens"].tolist()
        state = torch.stack([rows[b, n[b]:n[b] + W - 1] for b in range(B)])
        for b in range(B):
            if n[b] < T:
                y[b, n[b]:] = 0
        return y, state
    kept = _exact8(x)
    p = pre(kept)
    dp = s["dy"] * slope(p)
    ahead = torch.cat([dp, dp.new_zeros(B, W - 1, D)], 1).unfold(1, W, 1)      # dp at t .. t+W-1
    dx = torch.einsum("btdw,dw->btd", ahead, s["weight"].flip(1))
    dw = torch.einsum("btd,btdw->dw", dp, torch.cat([past, kept], 1).unfold(1, W, 1))
    return act(pre(x)), act(p), dx, dw, dp.sum((0, 1))


def _exact_scan(kind, s):
    one = kind == "scan_step"
    u, delta, z, Bm, Cm = (s[k][:, None] if one else s[k] for k in ("u", "delta", "z", "B", "C"))
    A, D = s["A"], s["D"]
    Bn, T, Dn = u.shape
    N, G = A.shape[1], Bm.shape[2]
    x = delta + s["dt_bias"]
    dt = torch.logaddexp(x, torch.zeros_like(x))
    h = u.new_zeros(Bn, Dn, N) if s["state"] is None else s["state"]
    train = kind == "scan_train"
    hs = u.new_empty(Bn, T + 1, Dn, N) if train else None
    if train:
        hs[:, 0] = h
    core = torch.empty_like(u)
    lens = s["lens"]
    Af = A.view(1, G, Dn // G, N)
    for t in range(T):
        d = dt[:, t].view(Bn, G, -1, 1)
        n = torch.exp(d * Af) * h.view(Bn, G, -1, N) + (d[..., 0] * u[:, t].view(Bn, G, -1))[..., None] * Bm[:, t, :, None]
        core[:, t] = torch.einsum("bgdn,bgn->bgd", n, Cm[:, t]).reshape(Bn, Dn)
        n = n.reshape(Bn, Dn, N)
        h = n if lens is None else torch.where((t < lens)[:, None, None], n, h)
        if train:
            hs[:, t + 1] = h
    gate = z / (1 + torch.exp(-z))
    full = core + D * u
    y = full * gate
    if lens is not None:
        y = torch.where((torch.arange(T, device=y.device)[None] < lens[:, None])[..., None], y, torch.zeros_like(y))
    if not train:
        return (y[:, 0] if one else y), h
    ds = s["dy"] * gate
    sz = 1 / (1 + torch.exp(-z))
    dz = s["dy"] * full * (sz + z * sz * (1 - sz))
    adj = torch.zeros_like(h)
    dA = torch.zeros_like(A)
    du, ddt, dB, dC = torch.empty_like(u), torch.empty_like(u), torch.empty_like(Bm), torch.empty_like(Cm)
    for t in range(T - 1, -1, -1):
        adj = adj + (ds[:, t].view(Bn, G, -1, 1) * Cm[:, t, :, None]).reshape(Bn, Dn, N)
        grp = adj.view(Bn, G, -1, N)
        dC[:, t] = torch.einsum("bgdn,bgd->bgn", hs[:, t + 1].view(Bn, G, -1, N), ds[:, t].view(Bn, G, -1))
        dB[:, t] = torch.einsum("bgdn,bgd->bgn", grp, (dt[:, t] * u[:, t]).view(Bn, G, -1))
        through = torch.einsum("bgdn,bgn->bgd", grp, Bm[:, t]).reshape(Bn, Dn)
        du[:, t] = dt[:, t] * through
        adj = adj * torch.exp(dt[:, t, :, None] * A)
        back = adj * hs[:, t]
        ddt[:, t] = u[:, t] * through + (back * A).sum(-1)
        dA += (back * dt[:, t, :, None]).sum(0)
    ddelta = ddt / (1 + torch.exp(-x))
    return (y, h, du + D * ds, ddelta, dA, dB, dC, (ds * u).sum((0, 1)), dz, ddelta.sum((0, 1)), adj)
