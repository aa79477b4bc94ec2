"""The state-space mixer's kernels against the formulas in 64 bits (tests/_mixer.py)."""
import math

import pytest
import torch

from linear_rnn_sequence_wkv7_b200 import ssm, wkv7
from tests import _mixer as ref
from tests._mixer import U32, check, f64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rand(gen, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float64) * std).to(dtype).cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---- 8-bit activations ---------------------------------------------------------------

@pytest.mark.parametrize("rows,D", [(1, 1), (3, 127), (5, 128), (2, 129), (4, 300), (33, 512), (7, 2052)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_act8_is_exact(cuda_device, rows, D, dtype):
    g = gen(rows * 1000 + D)
    x = rand(g, rows, D, dtype=DT[dtype], std=1.0) * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g).float()).cuda()
    x = x.to(DT[dtype])
    if rows > 2:
        x[0] = 0.0                              # an empty block: codes 0
        x[1, : D // 2] *= 2.0 ** -14            # values in the codes' subnormals
    a = ssm.act8_save(x)
    want, scale = ref.act8(f64(x))
    assert torch.equal(f64(a.scales), scale)
    assert torch.equal(f64(ssm.act8_load(a, torch.float32)), want)
    assert torch.equal(f64(ssm.act8_load(a, torch.bfloat16)), want)      # exact in bf16 as well


def test_act8_borders_and_ties(cuda_device):
    """Every bf16 significand over the codes' range: ties to even, 448 kept, amax at 448 and just above."""
    m = torch.arange(128, 256, dtype=torch.float32) / 128
    x = torch.cat([m * 2.0 ** e for e in range(-12, 9)]).view(-1, 128)
    x[:, 0] = 448.0
    x = x.clamp_max(448.0).to(torch.bfloat16).cuda()
    a = ssm.act8_save(x)
    want, scale = ref.act8(f64(x))
    assert torch.equal(f64(a.scales), scale) and torch.all(a.scales == 1.0)
    assert torch.equal(f64(ssm.act8_load(a, torch.float32)), want)
    top = torch.full((2, 128), 448.0)
    top[1, 5] = 450.0
    s = ssm.act8_save(top.cuda()).scales.flatten().tolist()
    assert s == [1.0, 2.0]


def test_act8_extremes(cuda_device):
    x = torch.zeros(4, 130)
    x[0, 3], x[0, 4], x[0, 5], x[0, 6] = float("inf"), float("-inf"), float("nan"), 1.0
    x[1, :] = 3.4028234e38
    x[2, :] = 1e-45
    x[3, 129] = -7.0
    a = ssm.act8_save(x.cuda())
    v = ssm.act8_load(a, torch.float32).cpu()
    assert torch.isnan(v[0, 3:6]).all() and v[0, 6] == 1.0 and torch.isfinite(v[0, 6:]).all()
    assert torch.isfinite(v[1]).all() and (v[1] / 3.4028234e38 - 1).abs().max() <= 2.0 ** -4
    assert (v[2] == 0).all() and v[3, 129] == -7.0 and (v[3, :129] == 0).all()
    assert f64(a.scales).min() == 2.0 ** -117


def test_act8_strided_rows(cuda_device):
    x = rand(gen(1), 6, 5, 200, dtype=torch.bfloat16)
    v = x[:, :, 8:140]
    want, _ = ref.act8(f64(v))
    assert torch.equal(f64(ssm.act8_load(ssm.act8_save(v), torch.float32)), want)
    with pytest.raises(ValueError):
        ssm.act8_save(x[:, 1:3])                # rows not evenly spaced
    with pytest.raises(ValueError):
        ssm.act8_save(x.transpose(1, 2))


# ---- RMS norm -----------------------------------------------------------------------------

def norm_ref(x, res, w, eps):
    s = x if res is None else x + res
    rstd = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return s, rstd, s * rstd * w


@pytest.mark.parametrize("rows,D", [(1, 1), (2, 7), (3, 128), (5, 130), (4, 1024), (700, 2048), (2, 2560), (3, 4097), (2, 16384)])
@pytest.mark.parametrize("dtype,res", [("f32", None), ("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"),
                                       ("bf16", None)])
def test_rmsnorm_forward(cuda_device, rows, D, dtype, res):
    g = gen(rows + D)
    x = rand(g, rows, D, dtype=DT[dtype])
    r = None if res is None else rand(g, rows, D, dtype=DT[res], std=3.0)
    w = rand(g, D)
    eps = 1e-5
    s, rstd, y = norm_ref(f64(x), f64(r), f64(w), eps)
    o = ssm.rmsnorm_forward(x, w, r, eps=eps, save8=True)
    # rstd: a mean of positive terms in fp64 from every four on (4 roundings, halved by the root); y: the
    # sum's, rstd's and two products' more
    check(o.rstd, rstd[:, 0], 4 * U32 * rstd[:, 0], "rstd")
    check(o.y, y, 8 * U32 * y.abs(), "y")
    if res is not None:
        check(o.residual, s, 0 * s, "residual")
        assert o.residual.dtype == DT[res]
    # the kept codes are those of the exact sum
    assert torch.equal(f64(ssm.act8_load(o.saved, torch.float32)), ref.act8(s)[0])
    # 8-bit output: the code of the exact y, or its neighbour where y is within 2^-22 of the border between two
    q = ssm.rmsnorm_forward(x, w, r, eps=eps, out8=True).y
    lo, hi = y * (1 - 2.0 ** -22), y * (1 + 2.0 ** -22)
    sc = f64(q.scales)
    top = torch.nn.functional.pad(y, (0, -D % 128)).unflatten(-1, (-1, 128)).abs().amax(-1)
    assert ((sc == ref.act8_scale(top * (1 - 2.0 ** -22))) | (sc == ref.act8_scale(top * (1 + 2.0 ** -22)))).all()
    each = sc.repeat_interleave(128, -1)[..., :D]
    code = f64(ssm.act8_load(q, torch.float32)) / each
    a, b = ref.e4m3_round(lo / each), ref.e4m3_round(hi / each)
    assert ((code == a) | (code == b)).all()


def test_rmsnorm_zero_row_and_in_place(cuda_device):
    x = rand(gen(3), 4, 256, dtype=torch.bfloat16)
    x[1] = 0
    r = torch.zeros_like(x)
    w = torch.ones(256, device="cuda")
    o = ssm.rmsnorm_forward(x, w, r, eps=1e-6, residual_out=r)
    assert o.residual is r and torch.equal(r, x) and (o.y[1] == 0).all()
    assert torch.isinf(ssm.rmsnorm_forward(x[1:2], w, eps=0.0).rstd).all()


@pytest.mark.parametrize("rows,D", [(1, 1), (3, 130), (300, 256), (5, 2560), (3, 2048), (2, 9000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kept", ["act8", "sum"])
def test_rmsnorm_backward(cuda_device, rows, D, dtype, kept):
    g = gen(rows + D)
    x, r = rand(g, rows, D, dtype=DT[dtype]), rand(g, rows, D, dtype=DT[dtype])
    w, dy, dres = rand(g, D), rand(g, rows, D, dtype=DT[dtype]), rand(g, rows, D, dtype=DT[dtype])
    o = ssm.rmsnorm_forward(x, w, r, eps=1e-5, save8=True)
    src = o.saved if kept == "act8" else o.residual
    s = f64(ssm.act8_load(o.saved, torch.float32)) if kept == "act8" else f64(o.residual)
    rs, W, G = f64(o.rstd)[:, None], f64(w), f64(dy)
    xh = s * rs
    for extra in (dres, None):
        dx, dw = ssm.rmsnorm_backward(dy, src, o.rstd, w, dresidual=extra, grad_dtype=DT[dtype])
        d = f64(extra) if extra is not None else torch.zeros_like(xh)
        c, cM = (W * G * xh).mean(-1, keepdim=True), (W * G * xh).abs().mean(-1, keepdim=True)
        M = d.abs() + rs * ((W * G).abs() + cM * xh.abs())
        # c: products 3, up to 32 terms in a thread, 5 + 16 joins; dx: 6 more
        check(dx, d + rs * (W * G - xh * c), 64 * U32 * M, "dx")
        check(dw, (G * xh).sum(0), (rows + 16) * U32 * (G * xh).abs().sum(0), "dw")


def test_rmsnorm_backward_matches_differences(cuda_device):
    """The gradient from the kept sum (fp32) against central differences of the fp64 forward."""
    g = gen(11)
    x, r, w = rand(g, 3, 70), rand(g, 3, 70), rand(g, 70)
    dy = rand(g, 3, 70)
    o = ssm.rmsnorm_forward(x, w, r, eps=1e-5)
    dx, dw = ssm.rmsnorm_backward(dy, o.residual, o.rstd, w)
    X, R, Wt, G = map(f64, (x, r, w, dy))
    loss = lambda a, b: float((norm_ref(a, R, b, 1e-5)[2] * G).sum())
    h = 1e-5
    for k in range(0, 210, 37):
        e = torch.zeros(210, dtype=torch.float64)
        e[k] = h
        num = (loss(X + e.view(3, 70), Wt) - loss(X - e.view(3, 70), Wt)) / (2 * h)
        assert abs(float(f64(dx).flatten()[k]) - num) <= 1e-5 * (1 + abs(num))
    for k in (0, 33, 69):
        e = torch.zeros(70, dtype=torch.float64)
        e[k] = h
        num = (loss(X, Wt + e) - loss(X, Wt - e)) / (2 * h)
        assert abs(float(f64(dw)[k]) - num) <= 1e-5 * (1 + abs(num))


# ---- convolution ------------------------------------------------------------------------------

CONV = [(1, 1, 1, 2), (2, 3, 5, 4), (1, 2, 128, 4), (2, 33, 130, 3), (3, 70, 132, 2), (1, 100, 256, 4), (2, 1100, 36, 4)]


@pytest.mark.parametrize("B,T,D,W", CONV)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_forward(cuda_device, B, T, D, W, dtype, silu):
    g = gen(T * D)
    x = rand(g, B, T, D + 8, dtype=DT[dtype])[..., 4:4 + D]
    w, b = rand(g, D, W), rand(g, D)
    for state, bias in ((None, None), (rand(g, B, W - 1, D, dtype=DT[dtype]), b)):
        y, so, kept = ssm.conv_forward(x, w, bias, state, silu=silu, return_state=True, save8=True)
        yr, sr, p, M = ref.conv(f64(x), f64(w), f64(bias), f64(state), silu)
        check(y, yr, ref.conv_bound(p, M, W, silu), "y")
        assert torch.equal(f64(so), sr)                     # the raw inputs, bit for bit
        q, _ = ref.act8(f64(x))
        assert torch.equal(f64(ssm.act8_load(kept, torch.float32)), q)
        # recomputed from the codes
        st8 = None if state is None else state.to(DT[dtype])
        y8 = ssm.conv_forward(kept, w, bias, st8, silu=silu, y_dtype=DT[dtype])
        yr, _, p, M = ref.conv(q, f64(w), f64(bias), f64(st8), silu)
        check(y8, yr, ref.conv_bound(p, M, W, silu), "y from codes")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_padded_batch(cuda_device, dtype):
    B, T, D, W = 6, 67, 132, 4
    g = gen(5)
    x, w, b = rand(g, B, T, D, dtype=DT[dtype]), rand(g, D, W), rand(g, D)
    state = rand(g, B, W - 1, D, dtype=DT[dtype])
    n = [0, 1, 2, 33, 67, 67]
    lens = torch.tensor([-3, 1, 2, 33, 67, 99], dtype=torch.int32, device="cuda")     # clamped to 0 .. T
    for i in range(B):
        x[i, n[i]:] = float("nan")                          # padding is not read
    y = torch.full((B, T, D), 7.0, dtype=DT[dtype], device="cuda")
    _, so = ssm.conv_forward(x, w, b, state, lens=lens, y=y, return_state=True)
    clean = f64(x).nan_to_num(0.0)
    yr, sr, p, M = ref.conv(clean, f64(w), f64(b), f64(state), True, lens=n)
    bound = ref.conv_bound(p, M, W, True)
    for i in range(B):
        check(y[i, :n[i]], yr[i, :n[i]], bound[i, :n[i]], f"y[{i}]")
        assert (y[i, n[i]:] == 7.0).all()
    assert torch.equal(f64(so), sr)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_steps_equal_the_sequence(cuda_device, W, dtype):
    B, T, D = 3, 9, 37
    g = gen(W)
    x, w, b = rand(g, B, T, D, dtype=DT[dtype]), rand(g, D, W), rand(g, D)
    state = rand(g, B, W - 1, D, dtype=DT[dtype])
    yr, sr, p, M = ref.conv(f64(x), f64(w), f64(b), f64(state), True)
    bound = ref.conv_bound(p, M, W, True)
    for t in range(T):
        y = ssm.conv_step(x[:, t], w, b, state)             # rows a sequence apart
        check(y, yr[:, t], bound[:, t], f"y[{t}]")
    assert torch.equal(f64(state), sr)


@pytest.mark.parametrize("B,T,D,W", CONV)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_backward(cuda_device, B, T, D, W, dtype, silu):
    g = gen(T + D)
    dt = DT[dtype]
    x, w, b, dy = rand(g, B, T, D, dtype=dt), rand(g, D, W), rand(g, D), rand(g, B, T, D, dtype=dt)
    state, dso = rand(g, B, W - 1, D, dtype=dt), rand(g, B, W - 1, D)
    for src, xr in ((x, f64(x)), (ssm.act8_save(x), ref.act8(f64(x))[0])):
        for st, dS, bias in ((None, None, None), (state, dso, b)):
            dx, dw, db, ds = ssm.conv_backward(src, w, bias, dy, st, dS, silu=silu, grad_dtype=dt)
            want = ref.conv_grads(xr, f64(w), f64(bias), f64(st), f64(dy), f64(dS), silu)
            _, _, p, M = ref.conv(xr, f64(w), f64(bias), f64(st), silu)
            # dp = dy act'(p): the slope is at most 1.1 and moves by at most 0.5 a unit of p; its own
            # roundings as the activation's
            edp = f64(dy).abs() * ((0.5 * (W + 1) * M + 14 + 2 * p.abs()) * U32 if silu else torch.full_like(p, U32))
            full = torch.cat([torch.zeros(B, W - 1, D, dtype=torch.float64) if st is None else f64(st), xr], 1)
            slope = 1.1 if silu else 1.0
            adp = slope * f64(dy).abs()
            ex = torch.zeros(B, T + W - 1, D, dtype=torch.float64)
            for j in range(W):
                ex[:, j:j + T] += f64(w)[:, j].abs() * (edp + (W + 1) * U32 * adp)
            if dS is not None:
                ex[:, T:] += U32 * f64(dS).abs() * 2
            check(dx, want[0], ex[:, W - 1:], "dx")
            n = 64 + 8 + B * ((T + 511) // 512) + 2                 # a run, its block, the parts
            ew = torch.stack([((edp + n * U32 * adp) * full[:, j:j + T].abs()).sum((0, 1)) for j in range(W)], 1)
            check(dw, want[1], ew, "dweight")
            if bias is not None:
                check(db, want[2], (edp + n * U32 * adp).sum((0, 1)), "dbias")
                check(ds, want[3], ex[:, :W - 1], "dstate")


# ---- selective scan ------------------------------------------------------------------------------

def scan_inputs(seed, B, T, D, N, G, dtype, gate=True, skip=True, bias=True, state=True):
    g = gen(seed)
    dt = DT[dtype]
    bc = rand(g, B, T, 2 * G * N + 8, dtype=dt)
    return dict(
        u=rand(g, B, T, D, dtype=dt), delta=rand(g, B, T, D + 8, dtype=dt)[..., 8:],
        A=-torch.exp(rand(g, D, N) * 0.5 + 0.5),
        B=bc[..., 8:8 + G * N].unflatten(-1, (G, N)), C=bc[..., 8 + G * N:].unflatten(-1, (G, N)),
        D=rand(g, D) if skip else None, z=rand(g, B, T, D, dtype=dt) if gate else None,
        dt_bias=rand(g, D) - 2.0 if bias else None, state0=rand(g, B, D, N) if state else None)


SCAN = [  # B, T, D, N, G
    (1, 1, 1, 1, 1), (2, 2, 3, 5, 1), (1, 15, 64, 16, 1), (2, 16, 66, 16, 1), (2, 17, 130, 16, 2), (1, 40, 128, 8, 1),
    (1, 33, 40, 32, 1), (2, 20, 24, 64, 3), (1, 50, 17, 50, 1), (3, 31, 96, 4, 2), (1, 35, 65, 13, 5)]


@pytest.mark.parametrize("B,T,D,N,G", SCAN)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_forward(cuda_device, B, T, D, N, G, dtype):
    full = scan_inputs(T * D + N, B, T, D, N, G, dtype)
    bare = dict(full, D=None, z=None, dt_bias=None, state0=None)
    for v, softplus in ((full, True), (bare, True)):
        y, h = ssm.ssm_forward(**v, softplus=softplus)
        r = {k: f64(t) for k, t in v.items()}
        yr, hr = ref.scan(**r, softplus=softplus)
        yM, hM = ref.scan(**r, softplus=softplus, absolute=True)
        n = ref.scan_count(T, N)
        check(y, yr, n * U32 * yM, "y")
        check(h, hr, n * U32 * hM, "stateT")
        yt, ht, kept = ssm.ssm_forward_train(**v, softplus=softplus)
        assert torch.equal(yt, y) and torch.equal(ht, h)
        for k in range(kept.shape[1]):
            cut = {a: (t[:, :16 * k] if t is not None and a in ("u", "delta", "B", "C", "z") else t) for a, t in r.items()}
            check(kept[:, k], ref.scan(**cut)[1], n * U32 * ref.scan(**cut, absolute=True)[1], f"states[{k}]")


def test_scan_without_softplus_takes_dt_as_it_is(cuda_device):
    v = scan_inputs(3, 2, 21, 64, 16, 1, "f32")
    v["delta"] = v["delta"].abs() * 0.3
    v["dt_bias"] = None
    y, h = ssm.ssm_forward(**v, softplus=False)
    r = {k: f64(t) for k, t in v.items()}
    yr, hr = ref.scan(**r, softplus=False)
    yM, hM = ref.scan(**r, softplus=False, absolute=True)
    n = ref.scan_count(21, 16)
    check(y, yr, n * U32 * yM, "y")
    check(h, hr, n * U32 * hM, "stateT")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,N,G", [(66, 16, 2), (64, 16, 1), (24, 40, 1)])
def test_scan_padded_batch(cuda_device, dtype, D, N, G):
    B, T = 5, 45
    v = scan_inputs(9, B, T, D, N, G, dtype)
    n = [0, 1, 16, 33, 45]
    lens = torch.tensor([-1, 1, 16, 33, 1000], dtype=torch.int32, device="cuda")
    clean = {k: f64(t) for k, t in v.items()}
    for i in range(B):
        for k in ("u", "delta", "B", "C", "z"):
            v[k][i, n[i]:] = float("nan")                   # padding is not read
    y = torch.full((B, T, D), 5.0, dtype=DT[dtype], device="cuda")
    _, h = ssm.ssm_forward(**v, lens=lens, y=y)
    nl = torch.tensor(n)
    yr, hr = ref.scan(**clean, lens=nl)
    yM, hM = ref.scan(**clean, lens=nl, absolute=True)
    c = ref.scan_count(T, N)
    for i in range(B):
        check(y[i, :n[i]], yr[i, :n[i]], c * U32 * yM[i, :n[i]], f"y[{i}]")
        assert (y[i, n[i]:] == 5.0).all()
    check(h, hr, c * U32 * hM, "stateT")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_in_segments(cuda_device, dtype):
    """Few channels over many tokens run as segments; the ragged lengths end inside them, before them and at T."""
    B, T, D, N = 2, 1203, 70, 16
    assert ssm.ssm_forward_workspace_size(B, T, D, N) > 0
    v = scan_inputs(21, B, T, D, N, 1, dtype)
    r = {k: f64(t) for k, t in v.items()}
    c = ref.scan_count(T, N)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    for lens in (None, torch.tensor([100, 1203], dtype=torch.int32)):
        y = torch.zeros(B, T, D, dtype=DT[dtype], device="cuda")
        st = v["state0"].clone()
        ssm.ssm_forward(**dict(v, state0=st), lens=None if lens is None else lens.cuda(), y=y, stateT=st)   # in place
        yr, hr = ref.scan(**r, lens=lens)
        yM, hM = ref.scan(**r, lens=lens, absolute=True)
        for i in range(B):
            n = T if lens is None else int(lens[i])
            check(y[i, :n], yr[i, :n], c * U32 * yM[i, :n], "y")
            assert (y[i, n:] == 0).all()
        check(st, hr, c * U32 * hM, "stateT")
    y1, h1 = ssm.ssm_forward(**v, workspace=none)           # one piece
    check(h1, hr if lens is None else ref.scan(**r)[1], c * U32 * ref.scan(**r, absolute=True)[1], "one piece")


@pytest.mark.parametrize("N,G,D", [(16, 1, 64), (5, 1, 7), (64, 2, 10), (8, 2, 34), (32, 1, 33)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_steps_equal_the_sequence(cuda_device, N, G, D, dtype):
    B, T = 3, 6
    v = scan_inputs(N, B, T, D, N, G, dtype)
    r = {k: f64(t) for k, t in v.items()}
    yr, hr = ref.scan(**r)
    yM, hM = ref.scan(**r, absolute=True)
    c = ref.scan_count(T, N)
    st = v["state0"].clone()
    for t in range(T):
        y = ssm.ssm_step(v["u"][:, t], v["delta"][:, t], v["A"], v["B"][:, t], v["C"][:, t], st, v["D"], v["z"][:, t],
                         v["dt_bias"])
        check(y, yr[:, t], c * U32 * yM[:, t], f"y[{t}]")
    check(st, hr, c * U32 * hM, "state")


def check_grads(v, got, dy, dsT, T, softplus=True):
    r = {k: f64(t) for k, t in v.items()}
    want = ref.scan_grads(dy=f64(dy), dstateT=f64(dsT), softplus=softplus, **r)
    M = ref.scan_grads_majorant(dy=f64(dy), dstateT=f64(dsT), softplus=softplus, **r)
    B, D, N = dy.shape[0], dy.shape[2], v["A"].shape[1]
    # forward and adjoint, then the sums over tokens and sequences, or channels
    n = 2 * ref.scan_count(T, N) + B * T + D
    for k in ("u", "delta", "A", "B", "C", "D", "z", "dt_bias", "state0"):
        g = getattr(got, k)
        if g is None:
            assert v[k] is None
            continue
        if v[k] is None:        # a zero state's gradient
            assert k == "state0"
            zero = dict(r, state0=torch.zeros(B, D, N, dtype=torch.float64))
            w = ref.scan_grads(dy=f64(dy), dstateT=f64(dsT), softplus=softplus, **zero)["state0"]
        else:
            w = want[k]
        check(g, w, n * U32 * M[k], k)


@pytest.mark.parametrize("B,T,D,N,G", SCAN)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_backward(cuda_device, B, T, D, N, G, dtype):
    dt = DT[dtype]
    full = scan_inputs(T + D + N, B, T, D, N, G, dtype)
    g = gen(1)
    dy, dsT = rand(g, B, T, D, dtype=dt), rand(g, B, D, N)
    _, _, kept = ssm.ssm_forward_train(**full)
    a = ssm.ssm_backward(dy=dy, dstateT=dsT, states=kept, grad_dtype=dt, **full)
    check_grads(full, a, dy, dsT, T)
    b = ssm.ssm_backward(dy=dy, dstateT=dsT, grad_dtype=dt, **full)          # states computed by the call
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    bare = dict(full, D=None, z=None, dt_bias=None, state0=None)
    check_grads(bare, ssm.ssm_backward(dy=dy, grad_dtype=torch.float32, **bare), dy, None, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_backward_in_segments(cuda_device, dtype):
    B, T, D, N = 1, 391, 36, 16
    full = scan_inputs(77, B, T, D, N, 1, dtype)
    g = gen(2)
    dy, dsT = rand(g, B, T, D, dtype=DT[dtype]), rand(g, B, D, N)
    check_grads(full, ssm.ssm_backward(dy=dy, dstateT=dsT, grad_dtype=DT[dtype], **full), dy, dsT, T)


def test_scan_backward_matches_differences(cuda_device):
    v = scan_inputs(5, 1, 6, 8, 4, 1, "f32")
    g = gen(6)
    dy, dsT = rand(g, 1, 6, 8), rand(g, 1, 8, 4)
    got = ssm.ssm_backward(dy=dy, dstateT=dsT, **v)
    r = {k: f64(t).contiguous() for k, t in v.items()}

    def loss(p):
        y, h = ref.scan(**p)
        return float((y * f64(dy)).sum() + (h * f64(dsT)).sum())

    h = 1e-6
    for k, t in r.items():
        flat = f64(getattr(got, k)).flatten()
        for i in range(0, t.numel(), max(1, t.numel() // 5)):
            up, dn = t.clone().flatten(), t.clone().flatten()
            up[i] += h
            dn[i] -= h
            num = (loss(dict(r, **{k: up.view_as(t)})) - loss(dict(r, **{k: dn.view_as(t)}))) / (2 * h)
            assert abs(float(flat[i]) - num) <= 1e-4 * (1 + abs(num)), (k, i)


def test_scan_of_zero_steps_keeps_the_state_bit_for_bit(cuda_device):
    v = scan_inputs(4, 2, 300, 40, 16, 1, "f32", bias=False)
    v["delta"] = torch.zeros(2, 300, 40, device="cuda")
    _, h = ssm.ssm_forward(**v, softplus=False)
    assert torch.equal(h, v["state0"])
    st = v["state0"].clone()
    ssm.ssm_step(v["u"][:, 0], v["delta"][:, 0], v["A"], v["B"][:, 0], v["C"][:, 0], st, softplus=False)
    assert torch.equal(st, v["state0"])


def test_scan_strong_decay_and_large_steps(cuda_device):
    """Rates and steps at which exp(dt A) is 0, and delta far on both sides of the softplus."""
    v = scan_inputs(8, 1, 24, 32, 16, 1, "f32")
    v["delta"] = torch.linspace(-90, 90, 24 * 32).view(1, 24, 32).cuda()
    v["A"] = v["A"] * 50
    v["dt_bias"] = None
    y, h = ssm.ssm_forward(**v)
    r = {k: f64(t) for k, t in v.items()}
    yr, hr = ref.scan(**r)
    yM, hM = ref.scan(**r, absolute=True)
    # |x| up to 90 counts as that many roundings of dt's own value, and of dt A below exp's last normal value (88)
    n = ref.scan_count(24, 16) + 24 * (90 + 2 * 88)
    check(y, yr, n * U32 * yM + 1e-30, "y")
    check(h, hr, n * U32 * hM + 1e-30, "stateT")
    assert torch.isfinite(y).all()


# ---- together -----------------------------------------------------------------------------------

def block(p, x, res, save):
    """A mixer block as a model runs it: norm -> projections -> convolution -> scan with its gate."""
    o = ssm.rmsnorm_forward(x, p["nw"], res, save8=save)
    D, N = p["D"].numel(), p["A"].shape[1]
    h = (o.y @ p["win"])
    xc, z, delta, bc = h[..., :D], h[..., D:2 * D], h[..., 2 * D:3 * D], h[..., 3 * D:]
    Bm, Cm = bc[..., :N].unflatten(-1, (1, N)), bc[..., N:].unflatten(-1, (1, N))
    return o, xc, z, delta, Bm, Cm


def block_params(g, E, D, N):
    return dict(nw=rand(g, E) * 0.1 + 1, win=rand(g, E, 3 * D + 2 * N, dtype=torch.bfloat16, std=E ** -0.5),
                cw=rand(g, D, 4, std=0.5), cb=rand(g, D, std=0.1), A=-torch.exp(rand(g, D, N) * 0.3), D=rand(g, D),
                dt_bias=rand(g, D, std=0.3) - 3.0)


def test_block_prompt_then_tokens_equals_one_prompt(cuda_device):
    """A padded prompt, then tokens one by one, gives what the whole sequence gives."""
    g = gen(31)
    B, E, D, N, T = 3, 128, 192, 16, 40
    p = block_params(g, E, D, N)
    x, res = rand(g, B, T, E, dtype=torch.bfloat16), rand(g, B, T, E, dtype=torch.bfloat16)
    _, xc, z, delta, Bm, Cm = block(p, x, res, False)
    u = ssm.conv_forward(xc, p["cw"], p["cb"])
    whole, hT = ssm.ssm_forward(u, delta, p["A"], Bm, Cm, p["D"], z, p["dt_bias"])
    n = 29
    lens = torch.tensor([n, n, n], dtype=torch.int32, device="cuda")
    u1, cs = ssm.conv_forward(xc, p["cw"], p["cb"], lens=lens, y=torch.zeros_like(u), return_state=True)
    _, st = ssm.ssm_forward(u1, delta, p["A"], Bm, Cm, p["D"], z, p["dt_bias"], lens=lens, y=torch.zeros_like(u))
    for t in range(n, T):
        ut = ssm.conv_step(xc[:, t], p["cw"], p["cb"], cs)
        # the same sum in the same order
        assert torch.equal(ut, u[:, t])
        yt = ssm.ssm_step(ut, delta[:, t], p["A"], Bm[:, t], Cm[:, t], st, p["D"], z[:, t], p["dt_bias"])
        # the same state up to fp32's roundings; y rounded to bf16 on both sides
        d = (yt.float() - whole[:, t].float()).abs()
        assert (d <= 2 * 2.0 ** -8 * whole[:, t].float().abs() + 1e-4).all()
    assert ((st - hT).abs() <= 1e-4 * hT.abs().max()).all()


def test_block_training_step_from_8_bit_checkpoints(cuda_device):
    """Forward that keeps 8-bit activations; backward through scan, convolution and norm from them; the
    gradients against the same chain in 64 bits on the values the codes stand for."""
    g = gen(33)
    B, E, D, N, T = 2, 96, 72, 8, 37
    p = block_params(g, E, D, N)
    x, res = rand(g, B, T, E, dtype=torch.bfloat16), rand(g, B, T, E, dtype=torch.bfloat16)
    o, xc, z, delta, Bm, Cm = block(p, x, res, True)
    u, x8 = ssm.conv_forward(xc, p["cw"], p["cb"], save8=True)
    y, _, kept = ssm.ssm_forward_train(u, delta, p["A"], Bm, Cm, p["D"], z, p["dt_bias"])
    dy = rand(g, B, T, D, dtype=torch.bfloat16)
    u8 = ssm.conv_forward(x8, p["cw"], p["cb"])
    gs = ssm.ssm_backward(u8, delta, p["A"], Bm, Cm, dy, p["D"], z, p["dt_bias"])
    check_grads(dict(u=u8, delta=delta, A=p["A"], B=Bm, C=Cm, D=p["D"], z=z, dt_bias=p["dt_bias"], state0=None), gs, dy,
                None, T)
    du = gs.u.to(torch.bfloat16)
    dx, dw, db, _ = ssm.conv_backward(x8, p["cw"], p["cb"], du, grad_dtype=torch.bfloat16)
    x8v = ref.act8(f64(xc))[0]
    want = ref.conv_grads(x8v, f64(p["cw"]), f64(p["cb"]), None, f64(du), None, True)
    for got, w in zip((dx, dw, db), want):
        assert (f64(got) - w).abs().max() <= 2.0 ** -7 * w.abs().max()
    dh = torch.cat([dx, gs.z.to(torch.bfloat16), gs.delta.to(torch.bfloat16), gs.B.flatten(2).to(torch.bfloat16),
                    gs.C.flatten(2).to(torch.bfloat16)], -1)
    dn = dh @ p["win"].t()
    dxin, dnw = ssm.rmsnorm_backward(dn, o.saved, o.rstd, p["nw"], grad_dtype=torch.bfloat16)
    s8, rs = ref.act8(f64(x) + f64(res))[0], f64(o.rstd)[..., None]
    wd, xh = f64(dn) * f64(p["nw"]), s8 * rs
    wantx = rs * (wd - xh * (wd * xh).mean(-1, keepdim=True))
    assert (f64(dxin) - wantx).abs().max() <= 2.0 ** -7 * wantx.abs().max()


def test_captured_steps_on_a_side_stream(cuda_device):
    """conv_step and ssm_step captured into one graph and replayed; prompts captured into two graphs that
    share nothing; all on a stream of their own."""
    g = gen(41)
    B, D, N = 4, 128, 16
    p = block_params(g, 64, D, N)
    xs = rand(g, 5, B, D, dtype=torch.bfloat16)
    z, delta = rand(g, B, D, dtype=torch.bfloat16), rand(g, B, D, dtype=torch.bfloat16)
    Bm, Cm = rand(g, B, 1, N, dtype=torch.bfloat16), rand(g, B, 1, N, dtype=torch.bfloat16)

    def run(x, cs, st):
        return ssm.ssm_step(ssm.conv_step(x, p["cw"], p["cb"], cs), delta, p["A"], Bm, Cm, st, p["D"], z, p["dt_bias"])

    cs, st = torch.zeros(B, 3, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, D, N, device="cuda")
    want = [run(x, cs, st) for x in xs]
    want_st = st.clone()
    cs.zero_(), st.zero_()
    x = torch.zeros(B, D, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(x, cs, st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cs.zero_(), st.zero_()
        for i in range(5):
            x.copy_(xs[i])
            graph.replay()
            assert torch.equal(y, want[i])
    side.synchronize()
    assert torch.equal(st, want_st)
    # the stream argument: the call waits for nothing but that stream
    v = scan_inputs(3, 2, 500, 64, 16, 1, "bf16")
    a = ssm.ssm_forward(**v)
    torch.cuda.synchronize()
    b = ssm.ssm_forward(**v, stream=side)
    side.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_backward_replays(cuda_device):
    v = scan_inputs(13, 2, 300, 64, 16, 1, "bf16")
    dy = rand(gen(14), 2, 300, 64, dtype=torch.bfloat16)
    want = ssm.ssm_backward(dy=dy, **v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ssm.ssm_backward(dy=dy, **v)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)            # every sum in a fixed order


def same(got, want):
    for a, b in zip(got, want):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))


def test_broadcast_and_shared_inputs(cuda_device):
    """Inputs with stride 0, and one tensor as several inputs, equal the same call on copies: gradients are
    those of each input by itself."""
    B, T, D, N = 3, 37, 64, 16
    v = scan_inputs(71, 1, T, D, N, 1, "bf16")
    v["delta"] = v["delta"].contiguous()
    per_token = ("u", "delta", "B", "C", "z")
    wide = {k: t.expand(B, *t.shape[1:]) if k in per_token else t for k, t in v.items()}
    wide["u"] = wide["u"][:, :1].expand(B, T, D)                # stride 0 over tokens too
    wide["z"], wide["C"] = wide["delta"], wide["B"]
    wide["state0"] = v["state0"].repeat(B, 1, 1)
    flat = {k: t.clone(memory_format=torch.contiguous_format) for k, t in wide.items()}
    same(ssm.ssm_forward(**wide), ssm.ssm_forward(**flat))
    dy, dsT = rand(gen(72), B, T, D, dtype=torch.bfloat16), rand(gen(73), B, D, N)
    same(ssm.ssm_backward(dy=dy, dstateT=dsT, **wide), ssm.ssm_backward(dy=dy, dstateT=dsT, **flat))
    w, b = rand(gen(74), D, 4), rand(gen(75), D)
    same(ssm.conv_forward(wide["u"], w, b, return_state=True), ssm.conv_forward(flat["u"], w, b, return_state=True))
    same(ssm.conv_backward(wide["u"], w, b, dy), ssm.conv_backward(flat["u"], w, b, dy))


@pytest.mark.parametrize("D", [256, 260, 131, 2048])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rmsnorm_slices_and_gradients_in_place(cuda_device, D, dtype):
    """Rows cut out of wider ones, x as its own residual, dx over dresidual."""
    g, dt = gen(76), DT[dtype]
    x = rand(g, 5, 9, D + 16, dtype=dt)[..., 16:]
    w, dy, dres = rand(g, D), rand(g, 5, 9, D, dtype=dt), rand(g, 5, 9, D, dtype=dt)
    flat = x.contiguous()
    a, b = ssm.rmsnorm_forward(x, w, save8=True), ssm.rmsnorm_forward(flat, w, save8=True)
    same((a.y, a.rstd, *a.saved), (b.y, b.rstd, *b.saved))
    twice, added = ssm.rmsnorm_forward(flat, w, flat), ssm.rmsnorm_forward(flat, w, flat.clone())
    same((twice.y, twice.residual, twice.rstd), (added.y, added.residual, added.rstd))
    want = ssm.rmsnorm_backward(dy, b.saved, b.rstd, w, dresidual=dres, grad_dtype=dt)
    over = dres.clone()
    got = ssm.rmsnorm_backward(dy, b.saved, b.rstd, w, dresidual=over, grad_dtype=dt, dx=over)
    assert got[0] is over
    same(got, want)


def test_lengths_outside_the_batch_are_clamped(cuda_device):
    B, T, D, N = 3, 700, 32, 16
    v = scan_inputs(77, B, T, D, N, 1, "f32")
    w = rand(gen(78), D, 4)
    odd, plain = (torch.tensor(n, dtype=torch.int32, device="cuda") for n in ([-5, 2 ** 31 - 1, T + 1], [0, T, T]))
    runs = []
    for lens in (odd, plain):
        y, c = torch.full((B, T, D), 3.0, device="cuda"), torch.full((B, T, D), 3.0, device="cuda")
        st = ssm.conv_forward(v["u"], w, lens=lens, y=c, return_state=True)[1]
        runs.append((y, ssm.ssm_forward(**v, lens=lens, y=y)[1], c, st))
    same(*runs)
    assert (runs[0][0][0] == 3.0).all() and (runs[0][2][0] == 3.0).all() and torch.equal(runs[0][1][0], v["state0"][0])


def test_two_streams_at_once(cuda_device):
    """The same operators on two streams at a time, each with its own inputs, give what they give alone."""
    B, T, D, N = 2, 900, 128, 16
    w, b, nw = rand(gen(79), D, 4), rand(gen(80), D), rand(gen(81), D)

    def run(v, dy, stream=None):
        u, kept = ssm.conv_forward(v["u"], w, b, save8=True, stream=stream)
        y, _, states = ssm.ssm_forward_train(**dict(v, u=u), stream=stream)
        g = ssm.ssm_backward(dy=dy, states=states, grad_dtype=torch.bfloat16, **dict(v, u=u), stream=stream)
        c = ssm.conv_backward(kept, w, b, g.u, grad_dtype=torch.bfloat16, stream=stream)
        n = ssm.rmsnorm_forward(y, nw, save8=True, stream=stream)
        return (*g, *c, *ssm.rmsnorm_backward(dy, n.saved, n.rstd, nw, stream=stream))

    sets = [(scan_inputs(82 + i, B, T, D, N, 1, "bf16"), rand(gen(90 + i), B, T, D, dtype=torch.bfloat16)) for i in range(2)]
    alone = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    both = [[run(*s, stream=st) for s, st in zip(sets, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    for pair in both:
        for got, want in zip(pair, alone):
            same(got, want)


def test_captured_training_step_replays(cuda_device):
    """Convolution and norm, forward to backward, from one graph that is replayed on other inputs."""
    B, T, D = 2, 130, 256
    g = gen(95)
    w, b, nw = rand(g, D, 4), rand(g, D), rand(g, D)
    first, second = (rand(g, 2, B, T, D, dtype=torch.bfloat16) for _ in range(2))
    inputs = first.clone()

    def run():
        x, dy = inputs[0], inputs[1]
        y, kept = ssm.conv_forward(x, w, b, save8=True)
        n = ssm.rmsnorm_forward(y, nw, x, save8=True)
        dx, dnw = ssm.rmsnorm_backward(dy, n.saved, n.rstd, nw, grad_dtype=torch.bfloat16)
        return (n.y, dnw, *ssm.conv_backward(kept, w, b, dx, grad_dtype=torch.bfloat16))

    want_first = run()
    inputs.copy_(second)
    want_second = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for data, want in ((first, want_first), (second, want_second)):
        inputs.copy_(data)
        graph.replay()
        torch.cuda.synchronize()
        same(got, want)


def test_offsets_behind_two_to_the_31_elements(cuda_device):
    """One sequence of 2^31 + elements: its last tokens are those of the same call on its last stretch."""
    D = 2048
    T = (1 << 31) // D + 4096
    g = gen(51)
    tail = 512
    block = rand(g, tail, D, dtype=torch.bfloat16)
    x = block.repeat(T // tail, 1)[None]
    assert x.shape[1] == T and x.numel() > 1 << 31
    last = x[:, -tail:]
    w, cw, cb = rand(g, D), rand(g, D, 4, std=0.5), rand(g, D)
    state = x[:, -tail - 3:-tail].contiguous()
    assert torch.equal(ssm.conv_forward(x, cw, cb)[:, -tail:], ssm.conv_forward(last, cw, cb, state))
    o, p = ssm.rmsnorm_forward(x, w, out8=True), ssm.rmsnorm_forward(last, w, out8=True)
    assert torch.equal(ssm.act8_load(o.y)[:, -tail:], ssm.act8_load(p.y)) and torch.equal(o.rstd[:, -tail:], p.rstd)
    del o
    dx = ssm.conv_backward(x, cw, cb, x, grad_dtype=torch.bfloat16)[0]
    assert torch.equal(dx[:, -tail:], ssm.conv_backward(last, cw, cb, last.contiguous(), state, grad_dtype=torch.bfloat16)[0])
    del dx
    # decays of e^-0.3 a token and more: a state forgets within 512 tokens
    N = 4
    A = -torch.exp(rand(g, D, N) * 0.1)
    bc = rand(g, tail, 2 * N, dtype=torch.bfloat16).repeat(T // tail, 1)[None]
    Bm, Cm = bc[..., :N].unflatten(-1, (1, N)), bc[..., N:].unflatten(-1, (1, N))
    bias = torch.full((D,), 2.0, device="cuda")
    y, h = ssm.ssm_forward(x, x, A, Bm, Cm, None, x, bias)
    cut = lambda t: t[:, -2 * tail:]
    y2, h2 = ssm.ssm_forward(cut(x), cut(x), A, cut(Bm), cut(Cm), None, cut(x), bias)
    assert torch.equal(y[:, -tail:], y2[:, -tail:]) and torch.equal(h, h2)


def test_empty_calls(cuda_device):
    v = scan_inputs(1, 2, 0, 16, 8, 1, "f32")
    y, h = ssm.ssm_forward(**v)
    assert y.shape == (2, 0, 16) and torch.equal(h, v["state0"])
    g = ssm.ssm_backward(dy=torch.zeros(2, 0, 16, device="cuda"), dstateT=v["state0"], **v)
    assert torch.equal(g.state0, v["state0"]) and (g.A == 0).all() and (g.D == 0).all() and (g.dt_bias == 0).all()
    x = torch.zeros(2, 0, 16, device="cuda")
    w, b, st = torch.ones(16, 4, device="cuda"), torch.zeros(16, device="cuda"), rand(gen(1), 2, 3, 16)
    y, so = ssm.conv_forward(x, w, b, st, return_state=True)
    assert torch.equal(so, st)
    dx, dw, db, ds = ssm.conv_backward(x, w, b, x, st, st)
    assert (dw == 0).all() and (db == 0).all() and torch.equal(ds, st)
    e = torch.zeros(0, 64, device="cuda")
    assert ssm.rmsnorm_forward(e, torch.ones(64, device="cuda")).y.shape == (0, 64)
    dx, dw = ssm.rmsnorm_backward(e, e, torch.zeros(0, device="cuda"), torch.ones(64, device="cuda"))
    assert (dw == 0).all()
    assert ssm.act8_load(ssm.act8_save(e)).shape == (0, 64)


def test_binding_refusals(cuda_device):
    v = scan_inputs(1, 2, 5, 16, 8, 1, "f32")
    with pytest.raises(ValueError):
        ssm.ssm_forward(**dict(v, u=v["u"].bfloat16()))
    with pytest.raises(ValueError):
        ssm.ssm_forward(**dict(v, A=v["A"].double()))
    with pytest.raises(ValueError):
        ssm.ssm_forward(**dict(v, B=v["B"].transpose(1, 3)))
    with pytest.raises(ValueError):
        ssm.ssm_forward(**dict(v, state0=v["state0"].cpu()))
    with pytest.raises(TypeError):
        ssm.ssm_forward(**v, y_dtype=torch.float16)
    with pytest.raises(wkv7.WKV7Error):
        ssm.ssm_forward(**scan_inputs(1, 1, 2, 4, 65, 1, "f32"))
    x = v["u"]
    with pytest.raises(wkv7.WKV7Error):
        ssm.conv_forward(x, torch.zeros(16, 5, device="cuda"))
    st = torch.zeros(2, 3, 16, device="cuda")
    with pytest.raises(wkv7.WKV7Error):
        ssm.conv_forward(x, torch.zeros(16, 4, device="cuda"), None, st, state_out=st)
    with pytest.raises(ValueError):
        ssm.conv_forward(x, torch.zeros(16, 4, device="cuda"), lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
