"""Calls of the state-space mixer's operators at the edges of what their header
allows, against the formulas in 64 bits (tests/_mixer.py)."""
import threading

import pytest
import torch

from linear_rnn_sequence_wkv7_b200 import ssm
from tests import _mixer as ref
from tests._mixer import U32, check, f64
from tests.test_gpu_mixer import DT, gen, norm_ref, rand

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


# ---- RMS norm ----------------------------------------------------------------------

@pytest.mark.parametrize("D", [256, 131, 2048, 9000])
@pytest.mark.parametrize("dtype,kept", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_rmsnorm_keeps_the_sum_without_a_residual(cuda_device, D, dtype, kept):
    """The C call with residual NULL and a residual_out: s = x in residual_out's type."""
    rows = 5
    x, w = rand(gen(D), rows, D, dtype=DT[dtype]), torch.ones(D, device="cuda")
    y = torch.empty_like(x)
    out = torch.full((rows, D), float("nan"), dtype=DT[kept], device="cuda")
    code = {F32: ssm.F32, BF16: ssm.BF16}
    st = ssm.load_library().wkv7_rmsnorm_forward(
        rows, D, code[x.dtype], code[out.dtype], code[x.dtype], x.data_ptr(), D, None, w.data_ptr(), 1e-6, out.data_ptr(),
        y.data_ptr(), None, None, None, None, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(out, x.to(DT[kept]))
    assert torch.equal(y, ssm.rmsnorm_forward(x, w, eps=1e-6).y)


def test_norms_of_two_widths_from_two_threads(cuda_device):
    """Widths of one kernel that take different amounts of shared memory, launched by two host threads at once
    through the C calls: none is refused."""
    fwd = ssm.load_library().wkv7_rmsnorm_forward
    bwd = ssm.load_library().wkv7_rmsnorm_backward
    stream = torch.cuda.current_stream().cuda_stream
    failed, go = [], threading.Barrier(2)

    def calls(D):
        x, w = rand(gen(D), 4, D, dtype=BF16), torch.ones(D, device="cuda")
        y, r, dx, dw = torch.empty_like(x), torch.empty(4, device="cuda"), torch.empty_like(x), torch.empty(D, device="cuda")
        ws = torch.empty(ssm.rmsnorm_backward_workspace_size(4, D), dtype=torch.uint8, device="cuda")
        keep = (x, w, y, r, dx, dw, ws)
        b = ssm.BF16
        a = (4, D, b, b, b, x.data_ptr(), D, None, w.data_ptr(), 1e-6, None, y.data_ptr(), None, None, None, r.data_ptr(), stream)
        g = (4, D, b, b, b, x.data_ptr(), None, r.data_ptr(), w.data_ptr(), x.data_ptr(), None, dx.data_ptr(), dw.data_ptr(),
             ws.data_ptr(), ws.numel(), stream)
        return keep, a, g

    def work(a, g):
        go.wait()
        for _ in range(10000):
            if fwd(*a) != 0:
                failed.append("forward")
            if bwd(*g) != 0:
                failed.append("backward")

    sets = [calls(D) for D in (8192, 4096)]
    threads = [threading.Thread(target=work, args=s[1:]) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, f"{len(failed)} calls refused"
    for (x, w, y, *_), *_ in sets:
        assert torch.equal(y, ssm.rmsnorm_forward(x, w).y)


@pytest.mark.parametrize("D", [128, 131, 256, 640, 2048, 9000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("residual", [True, False])
def test_rmsnorm_rows_whose_squares_leave_fp32(cuda_device, D, dtype, residual):
    """|s| from 1e-37 to 2e38 with eps = 0: the mean square is between 1e-75 and 1e76."""
    size = torch.tensor([1.0, 1e25, 1e19, 4e37, 1e-19, 1e-25, 1e-37, 1e-30], dtype=torch.float64)
    g = gen(D)
    # a row's values span a factor of 4, so that the smallest are no subnormals
    x = ((torch.rand(8, D, generator=g, dtype=torch.float64) + 0.5) * size[:, None]).to(DT[dtype]).cuda()
    r = ((torch.rand(8, D, generator=g, dtype=torch.float64) + 0.5) * size[:, None]).to(DT[dtype]).cuda() if residual else None
    w = rand(g, D)
    s, rstd, y = norm_ref(f64(x), f64(r), f64(w), 0.0)
    o = ssm.rmsnorm_forward(x, w, r, eps=0.0, save8=True)
    # rstd as for ordinary rows, or half a step of a subnormal (2^-150) where the row's size is above 2^126
    sub = 2.0 ** -150
    check(o.rstd, rstd[:, 0], 4 * U32 * rstd[:, 0] + sub, "rstd")
    check(o.y, y, (8 * U32 + sub / rstd) * y.abs(), "y")
    assert torch.equal(f64(ssm.act8_load(o.saved, F32)), ref.act8(s)[0])
    q = ssm.rmsnorm_forward(x, w, r, eps=0.0, out8=True).y
    each = f64(q.scales).repeat_interleave(128, -1)[..., :D]
    code = f64(ssm.act8_load(q, F32)) / each
    a, b = (ref.e4m3_round(y * (1 + e) / each) for e in (-2.0 ** -22, 2.0 ** -22))
    assert ((code == a) | (code == b)).all()
    # the gradient from what was kept
    dy = rand(g, 8, D, dtype=DT[dtype])
    dx, dw = ssm.rmsnorm_backward(dy, o.saved, o.rstd, w)
    rs, W, G = f64(o.rstd)[:, None], f64(w), f64(dy)
    xh = f64(ssm.act8_load(o.saved, F32)) * rs
    c, cM = (W * G * xh).mean(-1, keepdim=True), (W * G * xh).abs().mean(-1, keepdim=True)
    check(dx, rs * (W * G - xh * c), 64 * U32 * rs * ((W * G).abs() + cM * xh.abs()), "dx")
    check(dw, (G * xh).sum(0), 24 * U32 * (G * xh).abs().sum(0), "dw")


@pytest.mark.parametrize("D", [128, 131, 640, 2048, 9000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rmsnorm_row_with_an_infinity(cuda_device, D, dtype):
    """1 / sqrt(inf) = 0: the finite elements give 0, the infinite one inf * 0 = NaN; NaN takes its whole row;
    other rows are as they were."""
    x, w = rand(gen(D), 4, D, dtype=DT[dtype]), torch.ones(D, device="cuda")
    x[1, D // 3] = float("inf")
    x[2, D // 2] = float("nan")
    o = ssm.rmsnorm_forward(x, w, eps=1e-6)
    q = ssm.act8_load(ssm.rmsnorm_forward(x, w, eps=1e-6, out8=True).y, F32)
    assert o.rstd[1] == 0 and torch.isnan(o.rstd[2])
    for y in (o.y, q):
        assert torch.isnan(y[1, D // 3]) and int(torch.isnan(y[1]).sum()) == 1 and int((y[1] == 0).sum()) == D - 1
        assert torch.isnan(y[2]).all()
    plain = ssm.rmsnorm_forward(x[0::3].contiguous(), w, eps=1e-6)
    assert torch.equal(o.y[0::3], plain.y) and torch.equal(o.rstd[0::3], plain.rstd)


@pytest.mark.parametrize("D", [384, 640, 700])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rmsnorm_8_bit_blocks_of_zeros_and_nan(cuda_device, D, dtype):
    """Blocks that are all zero or all NaN, by the weight, beside ordinary ones."""
    x, w = rand(gen(D), 7, D, dtype=DT[dtype]), torch.ones(D, device="cuda")
    w[:128], w[128:256] = 0.0, float("nan")
    q = ssm.rmsnorm_forward(x, w, eps=1e-6, out8=True).y
    v = ssm.act8_load(q, F32)
    assert (v[:, :128] == 0).all() and torch.isnan(v[:, 128:256]).all()
    assert (q.scales[:, :2] == 2.0 ** -117).all()
    one = ssm.rmsnorm_forward(x, torch.ones(D, device="cuda"), eps=1e-6, out8=True).y
    assert torch.equal(v[:, 256:], ssm.act8_load(one, F32)[:, 256:]) and torch.equal(q.scales[:, 2:], one.scales[:, 2:])


# ---- scan ----------------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 67])
@pytest.mark.parametrize("N", [4, 16, 40])
def test_fp32_results_of_bf16_inputs(cuda_device, D, N):
    """The gate and its gradients in fp32's precision for every z: with B = C = 0 and u = D = dy = 1 they are
    all that is left; prompt and step alike."""
    T = 3
    z = torch.linspace(-60, 60, T * D).view(1, T, D).to(BF16).cuda()
    one = torch.ones(1, T, D, dtype=BF16, device="cuda")
    none = torch.zeros(1, T, 1, N, dtype=BF16, device="cuda")
    A, skip = torch.full((D, N), -1.0, device="cuda"), torch.ones(D, device="cuda")
    Z = f64(z)
    sg = torch.sigmoid(Z)
    # exp (2 steps, 4 roundings), sum, reciprocal (1 step), products: below 12 roundings, as conv_bound counts
    gate, e = Z * sg, 12 * U32 * (Z * sg).abs()
    y, _ = ssm.ssm_forward(one, one, A, none, none, skip, z, y_dtype=F32)
    check(y, gate, e, "y")
    for t in range(T):
        st = torch.zeros(1, D, N, device="cuda")
        yt = ssm.ssm_step(one[:, t], one[:, t], A, none[:, t], none[:, t], st, skip, z[:, t], y_dtype=F32)
        check(yt, gate[:, t], e[:, t], "step")
    g = ssm.ssm_backward(one, one, A, none, none, one, skip, z)
    check(g.u, gate, e, "du")
    check(g.z, sg * (1 + Z * (1 - sg)), 16 * U32 * sg * (1 + Z.abs() * (1 - sg)), "dz")
    check(g.D, gate.sum((0, 1)), (e + T * U32 * gate.abs()).sum((0, 1)), "dD")


@pytest.mark.parametrize("D", [64, 67])
def test_fp32_step_size_gradients_of_bf16_inputs(cuda_device, D):
    """One token, B = C = u = dy = 1 and no gate: ddelta is N sigmoid(delta)."""
    N = 16
    delta = torch.linspace(-60, 60, D).view(1, 1, D).to(BF16).cuda()
    one = torch.ones(1, 1, D, dtype=BF16, device="cuda")
    bc = torch.ones(1, 1, 1, N, dtype=BF16, device="cuda")
    g = ssm.ssm_backward(one, delta, torch.full((D, N), -1.0, device="cuda"), bc, bc, one)
    want = N * torch.sigmoid(f64(delta))
    check(g.delta, want, 12 * U32 * want, "ddelta")


# ---- in place ------------------------------------------------------------------------

@pytest.mark.parametrize("D", [131, 2050, 9000, 9001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rmsnorm_in_place_without_rows_ahead(cuda_device, D, dtype):
    """residual_out over residual and dx over dresidual where rows are read straight from memory: the same as
    into other tensors, with several rows a block and neighbouring rows in one cache line."""
    rows = 3 * 148 + 5 if D >= 9000 else 3 * 592 + 5
    g, dt = gen(D), DT[dtype]
    x, r, w = rand(g, rows, D, dtype=dt), rand(g, rows, D, dtype=dt, std=1e4), rand(g, D)
    x[::7] *= 2.0 ** -20            # sums that are not exact in fp32
    want = ssm.rmsnorm_forward(x, w, r, save8=True)
    over = r.clone()
    got = ssm.rmsnorm_forward(x, w, over, save8=True, residual_out=over)
    assert got.residual is over and torch.equal(over, want.residual) and torch.equal(got.y, want.y)
    assert torch.equal(got.saved.codes.view(torch.uint8), want.saved.codes.view(torch.uint8))
    dy = rand(g, rows, D, dtype=dt)
    a = ssm.rmsnorm_backward(dy, want.saved, want.rstd, w, dresidual=r, grad_dtype=dt)
    b = ssm.rmsnorm_backward(dy, want.saved, want.rstd, w, dresidual=(over := r.clone()), grad_dtype=dt, dx=over)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---- refusals --------------------------------------------------------------------------

def test_output_type_beside_an_output_has_to_agree(cuda_device):
    """y decides its own type; a y_dtype that differs, or a y of the wrong form, is refused by every call."""
    B, T, D, N = 2, 3, 16, 8
    one = lambda *s, dt=BF16: torch.zeros(s, dtype=dt, device="cuda")
    x, w, cw, A = one(B, T, D), one(D, dt=F32), one(D, 4, dt=F32), one(D, N, dt=F32)
    bc, st, cs = one(B, T, 1, N), one(B, D, N, dt=F32), one(B, 3, D)
    calls = [lambda **k: ssm.rmsnorm_forward(x, w, **k).y, lambda **k: ssm.conv_forward(x, cw, **k),
             lambda **k: ssm.ssm_forward(x, x, A, bc, bc, **k)[0], lambda **k: ssm.ssm_forward_train(x, x, A, bc, bc, **k)[0]]
    steps = [lambda **k: ssm.conv_step(x[:, 0], cw, None, cs, **k),
             lambda **k: ssm.ssm_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], st, **k)]
    for f, shape in [(f, (B, T, D)) for f in calls] + [(f, (B, D)) for f in steps]:
        for dt in (F32, BF16):
            y = one(*shape, dt=dt)
            assert f(y=y) is y and f(y=y, y_dtype=dt) is y
            with pytest.raises(ValueError):
                f(y=y, y_dtype=F32 if dt is BF16 else BF16)
    with pytest.raises(ValueError):
        ssm.rmsnorm_forward(x, w, out8=True, y=one(B, T, D))
    with pytest.raises(ValueError):
        ssm.rmsnorm_forward(x, w, y=ssm.act8_save(x))
