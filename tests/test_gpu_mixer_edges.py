"""Calls of the state-space mixer's operators at the edges of what their header
allows, against the formulas in 64 bits (tests/_mixer.py)."""
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
