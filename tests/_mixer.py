"""The state-space mixer's operators in 64 bits, from their formulas (torch on
the CPU), and the bounds their fp32 kernels are held to.

A sum of products evaluated in fp32 in any order differs from its exact value by
at most n u M, with u = 2^-24, n the roundings on the longest path from an input
to the result and M the same expression on absolute values (Higham, Accuracy and
Stability of Numerical Algorithms, section 3.1).  ``*_bound`` functions give M
and n.  Results stored in a 16- or 8-bit type may be off by half a step more.
"""
import torch

U32 = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return None if t is None else t.detach().double().cpu()


def check(got, ref, bound, name):
    """|got - ref| <= bound + half a step of got's type, everywhere."""
    g = f64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert torch.isfinite(g).all(), f"{name}: non-finite values"
    err, lim = (g - ref).abs(), bound + HALF_STEP[got.dtype] * (ref.abs() + bound)
    # below a type's normal range a step is absolute
    lim = lim + 2.0 ** -133
    if ref.numel():
        worst = (err - lim).argmax()
        assert (err <= lim).all(), (f"{name}: off by {err.flatten()[worst]:.3e}, allowed {lim.flatten()[worst]:.3e}, "
                                    f"value {ref.flatten()[worst]:.6e} at {int(worst)}")


# ---- 8 bits ---------------------------------------------------------------------

def act8_scale(amax):
    """Least power of two >= amax / 448, at least 2^-117 (amax fp64, finite)."""
    m, e = torch.frexp(amax)
    k = torch.where(m > 0.875, e - 8, e - 9)
    k = torch.where(amax > 0, k, torch.full_like(k, -117)).clamp_min(-117)
    return torch.ldexp(torch.ones_like(amax), k)


def e4m3_round(q):
    """Nearest e4m3 number, ties to even; |q| <= 448."""
    e = torch.frexp(q)[1].clamp_min(-5)             # q = m 2^e, 0.5 <= m < 1; subnormals below 2^-6
    step = torch.ldexp(torch.ones_like(q), e - 4)
    return torch.round(q / step) * step


def act8(x, scale=None):
    """(values, scales) of x [..., D] fp64."""
    D = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -D % 128)).unflatten(-1, (-1, 128))
    s = act8_scale(b.abs().amax(-1))
    v = e4m3_round(b / s[..., None]) * s[..., None]
    return v.flatten(-2)[..., :D], s


# ---- convolution ------------------------------------------------------------------

def conv(x, w, bias, state, silu, lens=None):
    """(y, state_out, p, M): M majorises p."""
    B, T, D = x.shape
    W = w.shape[1]
    past = torch.zeros(B, W - 1, D, dtype=x.dtype) if state is None else state
    full = torch.cat([past, x], 1)
    b = torch.zeros(D, dtype=x.dtype) if bias is None else bias
    p = b + sum(w[:, j] * full[:, j:j + T] for j in range(W))
    M = b.abs() + sum((w[:, j] * full[:, j:j + T]).abs() for j in range(W))
    n = [T] * B if lens is None else [min(max(int(v), 0), T) for v in lens]
    out = torch.stack([full[i, n[i]:n[i] + W - 1] for i in range(B)])
    return (p * torch.sigmoid(p) if silu else p + torch.zeros_like(p)), out, p, M


def conv_bound(p, M, W, silu):
    """p: W + 1 roundings.  The activation's slope is at most 1.1; its own
    roundings are below 12 + 2 |p| (the exponent's, |p| log2(e), where it is taken
    in one step; the exponential, sum, reciprocal and product otherwise)."""
    e = (W + 1) * U32 * M
    return 1.1 * e + (12 + 2 * p.abs()) * U32 * (p * torch.sigmoid(p)).abs() if silu else e


def conv_grads(x, w, bias, state, dy, dstate_out, silu):
    leaves = [t.clone().requires_grad_() for t in (x, w)]
    b = None if bias is None else bias.clone().requires_grad_()
    s = None if state is None else state.clone().requires_grad_()
    y, out, p, M = conv(leaves[0], leaves[1], b, s, silu)
    loss = (y * dy).sum()
    if dstate_out is not None:
        loss = loss + (out * dstate_out).sum()
    loss.backward()
    return leaves[0].grad, leaves[1].grad, None if b is None else b.grad, None if s is None else s.grad


# ---- scan -------------------------------------------------------------------------

def scan(u, delta, A, B, C, D=None, z=None, dt_bias=None, state0=None, softplus=True, lens=None, absolute=False):
    """(y, stateT), differentiable; ``absolute`` runs it on absolute values, a majorant."""
    Bn, T, Dn = u.shape
    G, N = B.shape[2], A.shape[1]
    rep = Dn // G
    x = delta if dt_bias is None else delta + dt_bias
    dt = torch.nn.functional.softplus(x, threshold=1e9) if softplus else x
    a_of = lambda t: torch.exp(dt[:, t, :, None] * A)
    if absolute:
        u, B, C = u.abs(), B.abs(), C.abs()
        D = None if D is None else D.abs()
        state0 = None if state0 is None else state0.abs()
    h = torch.zeros(Bn, Dn, N, dtype=u.dtype) if state0 is None else state0
    ys = []
    for t in range(T):
        new = a_of(t) * h + ((dt[:, t].abs() if absolute else dt[:, t]) * u[:, t])[..., None] * B[:, t].repeat_interleave(rep, 1)
        h = new if lens is None else torch.where((t < lens)[:, None, None], new, h)
        y = (h * C[:, t].repeat_interleave(rep, 1)).sum(-1)
        ys.append(y if D is None else y + D * u[:, t])
    y = torch.stack(ys, 1) if ys else torch.zeros_like(u)
    if z is not None:
        g = z * torch.sigmoid(z)
        y = y * (g.abs() if absolute else g)
    return y, h


def scan_count(T, N):
    """Roundings on the longest path of a scan.  A token: dt (its softplus: below
    10, plus the rounding of delta + dt_bias, at most |x| <= 8 of its own value),
    the rate's and the product's (weighted by |dt A| exp(dt A) <= 0.4), the
    exponential's 4, the update's 3: below 20.  Readout: 2 N, gate below 60."""
    return 20 * T + 2 * N + 60


def scan_grads(u, delta, A, B, C, dy, D=None, z=None, dt_bias=None, state0=None, dstateT=None, softplus=True):
    names = dict(u=u, delta=delta, A=A, B=B, C=C, D=D, z=z, dt_bias=dt_bias, state0=state0)
    v = {k: (None if t is None else t.clone().requires_grad_()) for k, t in names.items()}
    y, h = scan(**v, softplus=softplus)
    loss = (y * dy).sum() + (0 if dstateT is None else (h * dstateT).sum())
    loss.backward()
    return {k: (None if t is None else (torch.zeros_like(t) if t.grad is None else t.grad)) for k, t in v.items()}


def scan_grads_majorant(u, delta, A, B, C, dy, D=None, z=None, dt_bias=None, state0=None, dstateT=None, softplus=True):
    """The adjoint formulas with every factor by its absolute value."""
    Bn, T, Dn = u.shape
    G, N = B.shape[2], A.shape[1]
    rep = Dn // G
    x = delta if dt_bias is None else delta + dt_bias
    dt = torch.nn.functional.softplus(x, threshold=1e9) if softplus else x
    ad, au, aB, aC, aA = dt.abs(), u.abs(), B.abs(), C.abs(), A.abs()
    aD = torch.zeros(Dn, dtype=u.dtype) if D is None else D.abs()
    slope = torch.sigmoid(x) if softplus else torch.ones_like(x)
    h = torch.zeros(Bn, Dn, N, dtype=u.dtype) if state0 is None else state0.abs()
    hs = [h]
    for t in range(T):
        h = torch.exp(dt[:, t, :, None] * A) * h + (ad[:, t] * au[:, t])[..., None] * aB[:, t].repeat_interleave(rep, 1)
        hs.append(h)
    if z is None:
        ds = dy.abs()
    else:
        sg = torch.sigmoid(z)
        ds = (dy * z * sg).abs()
    w = torch.zeros(Bn, Dn, N, dtype=u.dtype) if dstateT is None else dstateT.abs()
    out = {k: torch.zeros_like(t) for k, t in dict(u=u, delta=u, A=A, B=B, C=C, z=u).items()}
    for t in range(T - 1, -1, -1):
        Bt, Ct = aB[:, t].repeat_interleave(rep, 1), aC[:, t].repeat_interleave(rep, 1)
        a = torch.exp(dt[:, t, :, None] * A)
        g = Ct * ds[:, t, :, None] + w
        q = a * hs[t] * g
        gb = (g * Bt).sum(-1)
        out["u"][:, t] = ad[:, t] * gb + aD * ds[:, t]
        out["delta"][:, t] = (au[:, t] * gb + (q * aA).sum(-1)) * slope[:, t]
        out["A"] += (q * ad[:, t, :, None]).sum(0)
        out["B"][:, t] = (g * (ad[:, t] * au[:, t])[..., None]).view(Bn, G, rep, N).sum(2)
        out["C"][:, t] = (hs[t + 1] * ds[:, t, :, None]).view(Bn, G, rep, N).sum(2)
        if z is not None:
            core = (hs[t + 1] * Ct).sum(-1) + aD * au[:, t]
            out["z"][:, t] = dy[:, t].abs() * core * (sg[:, t] * (1 + z[:, t].abs() * (1 - sg[:, t])))
        w = a * g
    out["state0"], out["D"], out["dt_bias"] = w, (ds * au).sum((0, 1)), out["delta"].sum((0, 1))
    return out
