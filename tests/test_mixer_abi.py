"""The state-space mixer's entry points refuse what they cannot do, on the host
and before any CUDA call; runs without a GPU."""
import ctypes

import pytest
import torch

from linear_rnn_sequence_wkv7_b200 import build as libbuild
from linear_rnn_sequence_wkv7_b200 import ssm, wkv7
from tests.test_abi import declared_symbols

P = ctypes.c_void_p(4096)       # aligned, never dereferenced: a check fails first, or nothing is to do
ODD = ctypes.c_void_p(4097)
INVALID, UNSUPPORTED, OK = wkv7.ERR_INVALID_ARG, wkv7.ERR_UNSUPPORTED, wkv7.OK
F32, BF16, E4M3 = ssm.F32, ssm.BF16, ssm.E4M3


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return ssm.load_library()


def test_symbols(lib):
    assert set(ssm.EXPORTED_SYMBOLS) <= declared_symbols()
    for name in ssm.EXPORTED_SYMBOLS:
        assert hasattr(lib, name)


def test_package_exports():
    import linear_rnn_sequence_wkv7_b200 as pkg
    for name in pkg._SSM_EXPORTS:
        assert getattr(pkg, name) is getattr(ssm, name)
    with pytest.raises(AttributeError):
        pkg.no_such_operator


def test_act8_refusals(lib):
    def save(rows=2, D=128, dt=BF16, x=P, ld=128, codes=P, scales=P):
        return lib.wkv7_act8_save(rows, D, dt, x, ld, codes, scales, None)

    def load(rows=2, D=128, codes=P, scales=P, dt=BF16, out=P):
        return lib.wkv7_act8_load(rows, D, codes, scales, dt, out, None)

    assert save(rows=-1) == INVALID and save(D=-1) == INVALID and save(ld=-1) == INVALID
    assert save(dt=E4M3) == INVALID and save(dt=9) == INVALID
    assert save(x=None) == INVALID and save(x=ODD) == INVALID and save(codes=None) == INVALID
    assert save(scales=None) == INVALID and save(scales=ctypes.c_void_p(4098)) == INVALID
    assert save(D=1 << 21) == UNSUPPORTED and save(rows=1 << 40) == UNSUPPORTED
    assert save(rows=0, x=None) == OK and save(D=0, x=None) == OK
    assert load(rows=-1) == INVALID and load(dt=E4M3) == INVALID and load(out=None) == INVALID
    assert load(out=ODD) == INVALID and load(codes=None) == INVALID and load(scales=None) == INVALID
    assert load(rows=0, out=None) == OK


def test_rmsnorm_refusals(lib):
    def fwd(rows=2, D=64, x=BF16, r=BF16, y=BF16, xp=P, ld=64, res=P, w=P, eps=1e-6, ro=P, yp=P, ys=None, sc=None,
            ss=None, rstd=P):
        return lib.wkv7_rmsnorm_forward(rows, D, x, r, y, xp, ld, res, w, eps, ro, yp, ys, sc, ss, rstd, None)

    assert fwd(rows=-1) == INVALID and fwd(D=-2) == INVALID and fwd(ld=-1) == INVALID
    assert fwd(x=E4M3) == INVALID and fwd(r=E4M3) == INVALID and fwd(y=3) == INVALID
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID and fwd(eps=float("inf")) == INVALID
    assert fwd(xp=None) == INVALID and fwd(w=None) == INVALID and fwd(yp=None) == INVALID
    assert fwd(res=ODD) == INVALID and fwd(ro=ODD) == INVALID and fwd(rstd=ODD) == INVALID
    assert fwd(y=E4M3) == INVALID               # codes without scales
    assert fwd(ys=P) == INVALID                 # scales without codes
    assert fwd(sc=P) == INVALID and fwd(ss=P) == INVALID
    assert fwd(D=20000) == UNSUPPORTED
    assert fwd(rows=0) == OK and fwd(D=0) == OK

    def bwd(rows=2, D=64, s=BF16, dy=BF16, g=F32, sp=P, ss=None, rstd=P, w=P, dyp=P, dres=None, dx=P, dw=P, ws=P,
            n=1 << 40):
        return lib.wkv7_rmsnorm_backward(rows, D, s, dy, g, sp, ss, rstd, w, dyp, dres, dx, dw, ws, n, None)

    assert bwd(rows=-1) == INVALID and bwd(dy=E4M3) == INVALID and bwd(g=E4M3) == INVALID
    assert bwd(s=E4M3) == INVALID and bwd(ss=P) == INVALID
    assert bwd(sp=None) == INVALID and bwd(rstd=None) == INVALID and bwd(dx=ODD) == INVALID and bwd(dw=None) == INVALID
    assert bwd(D=20000) == UNSUPPORTED and bwd(D=0) == OK


def test_conv_refusals(lib):
    def fwd(B=1, T=4, D=8, W=4, x=BF16, y=BF16, xp=P, xb=32, xt=8, xs=None, w=P, b=P, st=None, lens=None, yp=P, so=None,
            c=None, s=None):
        return lib.wkv7_conv_forward(B, T, D, W, x, y, xp, xb, xt, xs, w, b, st, lens, 1, yp, so, c, s, None)

    assert fwd(B=-1) == INVALID and fwd(T=-1) == INVALID and fwd(W=0) == INVALID and fwd(xt=-8) == INVALID
    assert fwd(W=1) == UNSUPPORTED and fwd(W=5) == UNSUPPORTED and fwd(D=1 << 21) == UNSUPPORTED
    assert fwd(x=5) == INVALID and fwd(y=E4M3) == INVALID
    assert fwd(xp=None) == INVALID and fwd(xp=ODD) == INVALID and fwd(w=None) == INVALID and fwd(yp=None) == INVALID
    assert fwd(x=E4M3) == INVALID and fwd(xs=P) == INVALID              # codes and scales come together
    assert fwd(x=E4M3, xs=P, so=P) == INVALID                           # the raw inputs are not known
    assert fwd(c=P) == INVALID and fwd(s=P) == INVALID
    assert fwd(c=P, s=P, lens=P) == INVALID and fwd(x=E4M3, xs=P, c=P, s=P) == INVALID
    assert fwd(st=P, so=P) == INVALID                                   # a block may read what another wrote
    assert fwd(st=ODD) == INVALID and fwd(lens=ctypes.c_void_p(4098)) == INVALID
    assert fwd(B=0) == OK and fwd(D=0) == OK and fwd(T=0) == OK

    def step(B=1, D=8, W=4, x=BF16, y=BF16, xp=P, xb=8, w=P, b=None, st=P, yp=P):
        return lib.wkv7_conv_step(B, D, W, x, y, xp, xb, w, b, st, 1, yp, None)

    assert step(x=E4M3) == INVALID and step(st=None) == INVALID and step(W=7) == UNSUPPORTED and step(xb=-1) == INVALID
    assert step(B=0, st=None) == OK

    def bwd(B=1, T=4, D=8, W=4, x=BF16, dy=BF16, g=F32, xp=P, xs=None, st=None, dso=None, ds=None, dw=P, dx=P, ws=P,
            n=1 << 40):
        return lib.wkv7_conv_backward(B, T, D, W, x, dy, g, xp, 32, 8, xs, P, P, st, P, dso, 1, dx, dw, P, ds, ws, n, None)

    assert bwd(W=1) == UNSUPPORTED and bwd(dy=E4M3) == INVALID and bwd(x=E4M3) == INVALID and bwd(xs=P) == INVALID
    assert bwd(dw=None) == INVALID and bwd(dx=None) == INVALID and bwd(ds=P, dso=P) == INVALID
    assert bwd(ws=None) == INVALID and bwd(n=16) == INVALID and bwd(D=0) == OK
    assert lib.wkv7_conv_backward_workspace_size(0, 4, 8, 4) == 0
    assert lib.wkv7_conv_backward_workspace_size(2, 600, 8, 4) >= (2 * 2 + 1) * 8 * 5 * 4


def _fwd(lib, B=1, T=4, D=8, N=16, G=1, dt=BF16, y=BF16, u=P, de=P, A=P, Bm=P, z=P, ts=8, lens=None, st0=None, sT=None,
         states=None, yp=P):
    return lib.wkv7_ssm_forward(B, T, D, N, G, dt, y, u, 32, ts, de, 32, 8, A, Bm, 64, 16, P, 64, 16, P, z, 32, 8, P, st0,
                                1, lens, yp, sT, states, None, 0, None)


def test_ssm_refusals(lib):
    fwd = lambda **k: _fwd(lib, **k)
    assert fwd(B=-1) == INVALID and fwd(N=0) == INVALID and fwd(G=0) == INVALID and fwd(G=3) == INVALID
    assert fwd(N=65) == UNSUPPORTED and fwd(D=1 << 21) == UNSUPPORTED
    assert fwd(dt=E4M3) == INVALID and fwd(y=4) == INVALID and fwd(ts=-8) == INVALID
    assert fwd(u=None) == INVALID and fwd(de=ODD) == INVALID and fwd(A=None) == INVALID and fwd(Bm=None) == INVALID
    assert fwd(z=ODD) == INVALID and fwd(yp=None) == INVALID
    assert fwd(st0=ctypes.c_void_p(4100)) == INVALID and fwd(sT=ctypes.c_void_p(4100)) == INVALID
    assert fwd(lens=P, states=P) == INVALID
    assert fwd(B=0) == OK and fwd(D=0) == OK and fwd(T=0) == OK
    step = lambda N=16, G=1, st=P, u=P, dt=BF16, B=1: lib.wkv7_ssm_step(
        B, 8, N, G, dt, BF16, u, 8, P, 8, P, P, 16, P, 16, P, P, 8, P, st, 1, P, None)
    assert step(N=80) == UNSUPPORTED and step(G=3) == INVALID and step(st=None) == INVALID and step(u=ODD) == INVALID
    assert step(dt=E4M3) == INVALID and step(B=0) == OK
    bwd = lambda N=16, g=F32, du=P, dz=P, z=P, dA=P, n=1 << 45, ws=P, T=4: lib.wkv7_ssm_backward(
        1, T, 8, N, 1, BF16, g, P, 32, 8, P, 32, 8, P, P, 64, 16, P, 64, 16, P, z, 32, 8, P, None, 1, P, P, None, du, P,
        dA, P, P, P, dz, P, P, ws, n, None)
    assert bwd(N=65) == UNSUPPORTED and bwd(g=E4M3) == INVALID and bwd(du=None) == INVALID and bwd(dA=None) == INVALID
    assert bwd(dz=None) == INVALID and bwd(z=None) == INVALID           # a gate and its gradient come together
    assert bwd(ws=None) == INVALID
    assert lib.wkv7_ssm_saved_states_size(2, 33, 8, 16) == 2 * 3 * 8 * 16 * 4
    assert lib.wkv7_ssm_saved_states_size(2, 33, 8, 65) == 0


def test_binding_refuses_cpu_tensors_and_wrong_types():
    libbuild.build()
    x = torch.zeros(2, 3, 8)
    w = torch.zeros(8, 4)
    with pytest.raises(ValueError):
        ssm.conv_forward(x, w)
    with pytest.raises(ValueError):
        ssm.act8_save(x)
    with pytest.raises(TypeError):
        ssm.act8_save(x.half())
    with pytest.raises(TypeError):
        ssm.act8_load(ssm.Act8(x, x), torch.float16)


def test_conv_refuses_its_input_as_output(lib):
    """Runs read tokens of their neighbours: y = x, dx = dy and dx = x would be a race.  Other pointers differ, so
    nothing else is refused, and no GPU is needed for the refusal."""
    x, w, dy, dw, ws = (ctypes.c_void_p(4096 * k) for k in range(1, 6))

    def fwd(y):
        return lib.wkv7_conv_forward(1, 4, 8, 4, BF16, BF16, x, 32, 8, None, w, None, None, None, 1, y, None, None, None, None)

    def bwd(dx):
        return lib.wkv7_conv_backward(1, 4, 8, 4, BF16, BF16, BF16, x, 32, 8, None, w, None, None, dy, None, 1, dx, dw, None,
                                      None, ws, 1 << 40, None)

    assert fwd(x) == INVALID
    assert bwd(dy) == INVALID and bwd(x) == INVALID
    # a call on no token writes nothing
    assert lib.wkv7_conv_forward(1, 0, 8, 4, BF16, BF16, x, 0, 8, None, w, None, None, None, 1, x, None, None, None, None) == OK
