"""WKV7 (RWKV-7 time-mix recurrence) on B200: a C-ABI CUDA library (libwkv7.so,
sm_100a) with a thin Python binding.

    from linear_rnn_sequence_wkv7_b200 import forward, step, backward

``forward``/``step``/``backward`` live in ``wkv7.py``, the state-space mixer's
operators (``conv_*``, ``ssm_*``, ``rmsnorm_*``, ``act8_*``) in ``ssm.py``; both
are imported lazily so that ``inputs`` (the seeded workload generator) can be
used without torch.
"""
_EXPORTS = ("forward", "step", "backward", "forward_workspace_size", "backward_workspace_size",
            "device_status", "load_library", "WKV7Error")
_SSM_EXPORTS = ("conv_forward", "conv_step", "conv_backward", "ssm_forward", "ssm_forward_train", "ssm_step",
                "ssm_backward", "rmsnorm_forward", "rmsnorm_backward", "act8_save", "act8_load", "Act8")


def __getattr__(name):
    if name in _EXPORTS:
        from . import wkv7
        return getattr(wkv7, name)
    if name in _SSM_EXPORTS:
        from . import ssm
        return getattr(ssm, name)
    raise AttributeError(name)
