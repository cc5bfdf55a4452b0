"""The Python calls whose tensors are looked at in C++: what they raise, and
that they are the ones that run."""

import pytest
import torch

import mamba_selective_scan_core_b200 as mm
from gdr_ref import BF, F32, gdr_inputs, q4_inputs, to_cuda

pytestmark = pytest.mark.gpu


def test_out_of_memory_is_torchs():
    """An output that no device holds (2^48 bytes): the error that torch's own
    calls raise, which callers catch by its name."""
    x = torch.zeros(1 << 22, 32, dtype=BF, device="cuda")
    W, scales = torch.zeros(1 << 24, 16, dtype=torch.uint8, device="cuda"), torch.zeros(1 << 24, 1, dtype=BF, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        mm.proj_q4(x, W, scales, group=32)


class NoLibrary:
    """Stands for the library that the ctypes way calls."""

    def __getattr__(self, name):
        raise AssertionError(f"{name} is called again through ctypes")


def operands():
    d = to_cuda(gdr_inputs(2, 100, 1, 2, 64, 64, seed=1))
    one = to_cuda(gdr_inputs(2, None, 1, 2, 64, 64, seed=2))
    q4 = {k: t.cuda() for k, t in q4_inputs(3, 100, 512, 64, seed=3).items()}
    return d, one, q4


def calls_of(d, one, q4):
    def args(t, state):
        return (t["q"], t["k"], t["v"], t["dt"], t["beta"], t["dt_bias"], t["A"], state)

    return {"mamba_gdr_fwd": lambda: mm.gdr_fwd(*args(d, d["h0"])),
            "mamba_gdr_state_update": lambda: mm.gdr_state_update(*args(one, one["h0"])),
            "mamba_proj_q4": lambda: mm.proj_q4(q4["x"], q4["W"], q4["scales"], q4["zeros"], group=64)}


def test_a_failed_launch_is_raised_at_once(monkeypatch):
    """Not taken for a call that does not fit and made a second time."""
    for name, call in calls_of(*operands()).items():
        call()
        with monkeypatch.context() as m:
            m.setenv("MAMBA_MIXER_TEST_LAUNCH_FAIL", "1")
            m.setattr(mm._names(), "lib", NoLibrary())
            with pytest.raises(mm.MixerError, match=name) as e:
                call()
            assert e.value.status == 7
        call()
    torch.cuda.synchronize()
