"""The variants of the state-space mixer's kernels that only larger calls, or calls
of mixed types, run: against the formulas in 64 bits (tests/_mixer.py), at the
smallest sizes that reach them.  Each test first checks that its size does."""
import pytest
import torch

from linear_rnn_sequence_wkv7_b200 import ssm
from tests import _mixer as ref
from tests._mixer import U32, check, f64
from tests.test_gpu_mixer import DT, check_grads, gen, norm_ref, rand, scan_inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def sm_count():
    return torch.cuda.get_device_properties(0).multi_processor_count


def d64(t):
    return None if t is None else t.detach().double()


def pad_n(N):
    return 8 if N <= 8 else 16 if N <= 16 else 32 if N <= 32 else 64


# ---- scan ------------------------------------------------------------------------

@pytest.mark.parametrize("B,D,N,G", [(9, 8192, 16, 1), (10, 13000, 8, 1), (11, 13001, 5, 1), (9, 6400, 32, 2), (6, 4800, 50, 3),
                                     (15, 1210, 64, 1), (10, 6320, 13, 2), (5, 9600, 16, 4)])
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_step_of_four_sequences_a_thread(cuda_device, B, D, N, G, dtype, out):
    """Two steps; batches that are no multiple of four."""
    assert (B + 3) // 4 * D * (pad_n(N) // 4) >= 512 * sm_count()
    v = scan_inputs(B + D + N, B, 2, D, N, G, dtype)
    r = {k: f64(t) for k, t in v.items()}
    yr, hr = ref.scan(**r)
    yM, hM = ref.scan(**r, absolute=True)
    c = ref.scan_count(2, N)
    st = v["state0"].clone()
    for t in range(2):
        y = ssm.ssm_step(v["u"][:, t], v["delta"][:, t], v["A"], v["B"][:, t], v["C"][:, t], st, v["D"], v["z"][:, t],
                         v["dt_bias"], y_dtype=DT[out])
        check(y, yr[:, t], c * U32 * yM[:, t], f"y[{t}]")
    check(st, hr, c * U32 * hM, "state")


def test_step_of_four_sequences_bare(cuda_device):
    """Without gate, skip, bias and softplus; B and C contiguous, so their quads are vectors."""
    B, D, N = 6, 9600, 16
    assert (B + 3) // 4 * D * 4 >= 512 * sm_count()
    v = scan_inputs(5, B, 1, D, N, 1, "bf16", gate=False, skip=False, bias=False)
    one = {k: v[k][:, 0].contiguous() for k in ("u", "delta", "B", "C")}
    one["delta"] = one["delta"].abs() * 0.25
    v["delta"] = one["delta"][:, None]
    r = {k: f64(t) for k, t in v.items()}
    yr, hr = ref.scan(**r, softplus=False)
    yM, hM = ref.scan(**r, softplus=False, absolute=True)
    st = v["state0"].clone()
    y = ssm.ssm_step(one["u"], one["delta"], v["A"], one["B"], one["C"], st, softplus=False)
    c = ref.scan_count(1, N)
    check(y, yr[:, 0], c * U32 * yM[:, 0], "y")
    check(st, hr, c * U32 * hM, "state")


def scanning_warps(B, D, N, G):
    """Of the two-channel form in one piece."""
    NP = pad_n(N)
    CC = {8: 32, 16: 16, 32: 16, 64: 8}[NP]
    return B * G * ((D // G + CC - 1) // CC) * (CC * NP // 8) // 32


TWO = [(4, 35, 3600, 16, 1), (7, 18, 2050, 16, 2), (8, 17, 3560, 8, 1), (9, 16, 3201, 5, 1), (3, 20, 2384, 32, 1), (3, 33, 2400, 24, 5),
       (3, 18, 1192, 64, 1), (3, 31, 1197, 50, 1)]


@pytest.mark.parametrize("B,T,D,N,G", TWO)
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_scan_with_two_channels_a_thread(cuda_device, B, T, D, N, G, dtype, out):
    assert scanning_warps(B, D, N, G) >= 6 * sm_count()
    v = scan_inputs(T * D + N, B, T, D, N, G, dtype)
    r = {k: f64(t) for k, t in v.items()}
    c = ref.scan_count(T, N)
    y, h, kept = ssm.ssm_forward_train(**v, y_dtype=DT[out])
    yr, hr = ref.scan(**r)
    yM, hM = ref.scan(**r, absolute=True)
    check(y, yr, c * U32 * yM, "y")
    check(h, hr, c * U32 * hM, "stateT")
    for k in range(kept.shape[1]):
        cut = {a: (t[:, :16 * k] if a in ("u", "delta", "B", "C", "z") else t) for a, t in r.items()}
        check(kept[:, k], ref.scan(**cut)[1], c * U32 * ref.scan(**cut, absolute=True)[1], f"states[{k}]")
    n = [(i * 7 + 3) % (T + 1) for i in range(B)]
    n[0], n[1] = 0, T
    lens = torch.tensor(n, dtype=torch.int32)
    y = torch.full((B, T, D), 5.0, dtype=DT[out], device="cuda")
    _, h = ssm.ssm_forward(**v, lens=lens.cuda(), y=y)
    yr, hr = ref.scan(**r, lens=lens)
    yM, hM = ref.scan(**r, lens=lens, absolute=True)
    for i in range(B):
        check(y[i, :n[i]], yr[i, :n[i]], c * U32 * yM[i, :n[i]], f"y[{i}]")
        assert (y[i, n[i]:] == 5.0).all()
    check(h, hr, c * U32 * hM, "stateT with lens")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [720, 721])
def test_scan_in_segments_with_two_channels_a_thread(cuda_device, dtype, D):
    B, T, N = 2, 1300, 16
    assert ssm.ssm_forward_workspace_size(B, T, D, N) > 0 and scanning_warps(B, D, N, 1) * 10 >= 6 * sm_count()
    v = scan_inputs(D, B, T, D, N, 1, dtype)
    r = {k: f64(t) for k, t in v.items()}
    c = ref.scan_count(T, N)
    y, h = ssm.ssm_forward(**v)
    yr, hr = ref.scan(**r)
    yM, hM = ref.scan(**r, absolute=True)
    check(y, yr, c * U32 * yM, "y")
    check(h, hr, c * U32 * hM, "stateT")


@pytest.mark.parametrize("B,T,D,N,G", [(2, 37, 64, 16, 1), (2, 37, 66, 16, 2), (1, 20, 24, 40, 1), (4, 19, 3600, 16, 1)])
@pytest.mark.parametrize("dtype,grad", [("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
def test_scan_gradients_of_another_type(cuda_device, B, T, D, N, G, dtype, grad):
    v = scan_inputs(T + D, B, T, D, N, G, dtype)
    g = gen(17)
    dy, dsT = rand(g, B, T, D, dtype=DT[dtype]), rand(g, B, D, N)
    _, _, kept = ssm.ssm_forward_train(**v)
    got = ssm.ssm_backward(dy=dy, dstateT=dsT, states=kept, grad_dtype=DT[grad], **v)
    assert got.u.dtype == DT[grad]
    check_grads(v, got, dy, dsT, T)


@pytest.mark.parametrize("dtype,out", [("f32", "bf16"), ("bf16", "f32")])
def test_scan_output_of_another_type(cuda_device, dtype, out):
    for B, T, D, N, G in ((2, 37, 64, 16, 1), (2, 18, 67, 5, 1)):
        v = scan_inputs(T, B, T, D, N, G, dtype)
        r = {k: f64(t) for k, t in v.items()}
        y, h = ssm.ssm_forward(**v, y_dtype=DT[out])
        assert y.dtype == DT[out]
        c = ref.scan_count(T, N)
        check(y, ref.scan(**r)[0], c * U32 * ref.scan(**r, absolute=True)[0], "y")


# ---- convolution -------------------------------------------------------------------

def run_length(B, T, D):
    run = 64
    while run > 16 and B * ((T + run - 1) // run) * ((D + 127) // 128) < 12 * sm_count():
        run //= 2
    return run


@pytest.mark.parametrize("T,run", [(7130, 64), (4003, 32)])
@pytest.mark.parametrize("D", [36, 37])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_forward_in_long_runs(cuda_device, T, run, D, dtype, W):
    """Runs in which a slot of the ring is used again: with the 8-bit copy, from the codes, and with lengths."""
    B = 16
    assert run_length(B, T, D) == run
    g = gen(T + D)
    dt = DT[dtype]
    x, w, b, state = rand(g, B, T, D, dtype=dt), rand(g, D, W), rand(g, D), rand(g, B, W - 1, D, dtype=dt)
    X, Wt, Bt, S = map(d64, (x, w, b, state))
    full = torch.cat([S, X], 1)

    def want(full):
        p = Bt + sum(Wt[:, j] * full[:, j:j + T] for j in range(W))
        M = Bt.abs() + sum((Wt[:, j] * full[:, j:j + T]).abs() for j in range(W))
        return (p * torch.sigmoid(p)).cpu(), ref.conv_bound(p, M, W, True).cpu()

    y, so, kept = ssm.conv_forward(x, w, b, state, return_state=True, save8=True)
    yr, bound = want(full)
    check(y, yr, bound, "y")
    assert torch.equal(so, x[:, T - W + 1:])
    q, scale = ref.act8(X)
    assert torch.equal(kept.scales.double(), scale) and torch.equal(ssm.act8_load(kept, F32).double(), q)
    check(ssm.conv_forward(x, w, b, state), yr, bound, "y alone")
    y8 = ssm.conv_forward(kept, w, b, state, y_dtype=dt)
    check(y8, *want(torch.cat([S, q], 1)), "y from codes")
    n = torch.randint(0, T + 1, (B,), generator=g).tolist()
    n[0], n[1], n[2] = 0, 1, T
    out = torch.full((B, T, D), 7.0, dtype=dt, device="cuda")
    _, so = ssm.conv_forward(x, w, b, state, lens=torch.tensor(n, dtype=torch.int32, device="cuda"), y=out, return_state=True)
    for i in range(B):
        check(out[i, :n[i]], yr[i, :n[i]], bound[i, :n[i]], f"y[{i}]")
        assert (out[i, n[i]:] == 7.0).all()
        assert torch.equal(so[i].double(), full[i, n[i]:n[i] + W - 1])


@pytest.mark.parametrize("D", [132, 37])
@pytest.mark.parametrize("dtype,out", [("f32", "bf16"), ("bf16", "f32")])
def test_conv_output_of_another_type(cuda_device, D, dtype, out):
    B, T, W = 2, 70, 4
    g = gen(D)
    x, w, b, state = rand(g, B, T, D, dtype=DT[dtype]), rand(g, D, W), rand(g, D), rand(g, B, W - 1, D, dtype=DT[dtype])
    yr, sr, p, M = ref.conv(f64(x), f64(w), f64(b), f64(state), True)
    y, so, kept = ssm.conv_forward(x, w, b, state, y_dtype=DT[out], return_state=True, save8=True)
    assert y.dtype == DT[out] and so.dtype == DT[dtype]
    check(y, yr, ref.conv_bound(p, M, W, True), "y")
    assert torch.equal(f64(so), sr)
    assert torch.equal(f64(ssm.act8_load(kept, F32)), ref.act8(f64(x))[0])
    check(ssm.conv_forward(x, w, b, state, y_dtype=DT[out]), yr, ref.conv_bound(p, M, W, True), "y alone")
    st = state.clone()
    y1, _, p, M = ref.conv(f64(x[:, :1]), f64(w), f64(b), f64(state), True)
    check(ssm.conv_step(x[:, 0], w, b, st, y_dtype=DT[out]), y1[:, 0], ref.conv_bound(p, M, W, True)[:, 0], "step")


@pytest.mark.parametrize("D", [132, 37])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("dyt", ["f32", "bf16"])
@pytest.mark.parametrize("src", ["f32", "bf16", "act8"])
def test_conv_gradients_of_mixed_types(cuda_device, D, grad, dyt, src):
    B, T, W = 2, 150, 4
    g = gen(D)
    x = rand(g, B, T, D, dtype=F32 if src == "f32" else BF16)
    w, b, dy, dso = rand(g, D, W), rand(g, D), rand(g, B, T, D, dtype=DT[dyt]), rand(g, B, W - 1, D)
    state = rand(g, B, W - 1, D, dtype=DT[grad] if src == "act8" else DT[src])
    xr = f64(x)
    if src == "act8":
        x, xr = ssm.act8_save(x), ref.act8(f64(x))[0]
    dx, dw, db, ds = ssm.conv_backward(x, w, b, dy, state, dso, grad_dtype=DT[grad])
    assert dx.dtype == DT[grad]
    want = ref.conv_grads(xr, f64(w), f64(b), f64(state), f64(dy), f64(dso), True)
    _, _, p, M = ref.conv(xr, f64(w), f64(b), f64(state), True)
    # as for equal types: dp moves by 0.5 a unit of p, whose own roundings are W + 1; the activation's below 14 + 2 |p|
    edp = f64(dy).abs() * (0.5 * (W + 1) * M + 14 + 2 * p.abs()) * U32
    adp = 1.1 * f64(dy).abs()
    full = torch.cat([f64(state), xr], 1)
    ex = torch.zeros(B, T + W - 1, D, dtype=torch.float64)
    for j in range(W):
        ex[:, j:j + T] += f64(w)[:, j].abs() * (edp + (W + 1) * U32 * adp)
    ex[:, T:] += 2 * U32 * f64(dso).abs()
    check(dx, want[0], ex[:, W - 1:], "dx")
    n = 64 + 8 + B * ((T + 255) // 256) + 2
    check(dw, want[1], torch.stack([((edp + n * U32 * adp) * full[:, j:j + T].abs()).sum((0, 1)) for j in range(W)], 1), "dweight")
    check(db, want[2], (edp + n * U32 * adp).sum((0, 1)), "dbias")
    check(ds, want[3], ex[:, :W - 1], "dstate")


# ---- RMS norm ------------------------------------------------------------------------

def norm_slots(D):
    """Blocks that walk the rows."""
    nblk = (D + 127) // 128
    mb = nblk if nblk <= 2 else 4 if nblk <= 64 else 8
    threads = 32 * ((nblk + mb - 1) // mb)
    return sm_count() * max(1, (1024 if mb <= 2 else 512) // threads)


WIDE = [(3, 128), (3, 131), (3, 256), (5, 640), (5, 2048), (4, 2050), (3, 4096), (4, 9000), (3, 9001), (3, 16384)]


def norm_rows(per, D):
    return per * norm_slots(D) + 3


@pytest.mark.parametrize("per,D", WIDE)
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("f32", "f32"), ("bf16", None), ("bf16", "f32")])
def test_rmsnorm_forward_walks_rows(cuda_device, per, D, dtype, res):
    """Several rows a block, and three blocks with one more."""
    rows = norm_rows(per, D)
    g = gen(D)
    x, w = rand(g, rows, D, dtype=DT[dtype]), rand(g, D)
    r = None if res is None else rand(g, rows, D, dtype=DT[res], std=3.0)
    s, rstd, y = norm_ref(d64(x), d64(r), d64(w), 1e-5)
    o = ssm.rmsnorm_forward(x, w, r, eps=1e-5, save8=True)
    check(o.rstd, rstd[:, 0].cpu(), (4 * U32 * rstd[:, 0]).cpu(), "rstd")
    check(o.y, y.cpu(), (8 * U32 * y.abs()).cpu(), "y")
    if res is not None:
        check(o.residual, s.cpu(), 0 * s.cpu(), "residual")
    assert torch.equal(ssm.act8_load(o.saved, F32).double(), ref.act8(s)[0])
    q = ssm.rmsnorm_forward(x, w, r, eps=1e-5, out8=True).y
    each = q.scales.double().repeat_interleave(128, -1)[..., :D]
    code = ssm.act8_load(q, F32).double() / each
    # the code of the exact y, or its neighbour where y is within 2^-22 of the border between two
    a, b = (ref.e4m3_round(y * (1 + e) / each) for e in (-2.0 ** -22, 2.0 ** -22))
    assert ((code == a) | (code == b)).all()
    top = torch.nn.functional.pad(y, (0, -D % 128)).unflatten(-1, (-1, 128)).abs().amax(-1)
    sc = q.scales.double()
    assert ((sc == ref.act8_scale(top * (1 - 2.0 ** -22))) | (sc == ref.act8_scale(top * (1 + 2.0 ** -22)))).all()


def check_norm_backward(rows, D, src, dyt, grad, extra):
    g = gen(rows + D)
    s = rand(g, rows, D, dtype=F32 if src == "f32" else BF16)
    w, dy = rand(g, D), rand(g, rows, D, dtype=DT[dyt])
    rstd = torch.rsqrt(s.double().square().mean(-1)).float()
    dres = rand(g, rows, D, dtype=DT[grad]) if extra else None
    S = d64(s)
    if src == "act8":
        s, S = ssm.act8_save(s), ref.act8(S)[0]
    dx, dw = ssm.rmsnorm_backward(dy, s, rstd, w, dresidual=dres, grad_dtype=DT[grad])
    assert dx.dtype == DT[grad]
    rs, W, G = d64(rstd)[:, None], d64(w), d64(dy)
    xh = S * rs
    d = d64(dres) if extra else torch.zeros_like(xh)
    c, cM = (W * G * xh).mean(-1, keepdim=True), (W * G * xh).abs().mean(-1, keepdim=True)
    M = d.abs() + rs * ((W * G).abs() + cM * xh.abs())
    check(dx, (d + rs * (W * G - xh * c)).cpu(), (64 * U32 * M).cpu(), "dx")
    check(dw, (G * xh).sum(0).cpu(), ((rows + 16) * U32 * (G * xh).abs().sum(0)).cpu(), "dw")


@pytest.mark.parametrize("per,D", WIDE)
@pytest.mark.parametrize("src,dtype,extra", [("act8", "bf16", True), ("bf16", "bf16", False), ("f32", "f32", True), ("act8", "f32", False)])
def test_rmsnorm_backward_walks_rows(cuda_device, per, D, src, dtype, extra):
    check_norm_backward(norm_rows(per, D), D, src, dtype, dtype, extra)


@pytest.mark.parametrize("D", [256, 131, 640])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("dyt", ["f32", "bf16"])
@pytest.mark.parametrize("src", ["f32", "bf16", "act8"])
@pytest.mark.parametrize("extra", [True, False])
def test_rmsnorm_gradients_of_mixed_types(cuda_device, D, grad, dyt, src, extra):
    check_norm_backward(19, D, src, dyt, grad, extra)


@pytest.mark.parametrize("D", [256, 131, 2052])
@pytest.mark.parametrize("dtype,out", [("f32", "bf16"), ("bf16", "f32")])
def test_rmsnorm_output_of_another_type(cuda_device, D, dtype, out):
    g = gen(D)
    x, r, w = rand(g, 9, D, dtype=DT[dtype]), rand(g, 9, D, dtype=DT[dtype]), rand(g, D)
    _, _, y = norm_ref(f64(x), f64(r), f64(w), 1e-5)
    o = ssm.rmsnorm_forward(x, w, r, eps=1e-5, y_dtype=DT[out])
    assert o.y.dtype == DT[out] and o.residual.dtype == DT[dtype]
    check(o.y, y, 8 * U32 * y.abs(), "y")
