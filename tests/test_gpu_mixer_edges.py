"""Calls of the state-space mixer's operators at the edges of what their header
allows, against the formulas in 64 bits (tests/_mixer.py)."""
import threading

import pytest
import torch

from linear_rnn_sequence_wkv7_b200 import ssm
from tests.test_gpu_mixer import DT, gen, rand

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
