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


class Counting:
    """names.calls, with how often each call gave a result."""

    def __init__(self, calls):
        self.calls, self.answered = calls, 0

    def __getattr__(self, name):
        call = getattr(self.calls, name)

        def run(*args):
            out = call(*args)
            self.answered += out is not None
            return out
        return run


def layouts(L):
    """q, k, v of a call of L tokens in the layouts that programs have them in:
    dense, parts of one packed tensor, a prompt cut from a longer buffer, one
    key head."""
    for B, G, packed in ((1, 2, False), (2, 2, True), (3, 1, True), (1, 1, False)):
        yield to_cuda(gdr_inputs(B, L, G, 2, 64, 64, seed=L + B, packed=packed))
    d = to_cuda(gdr_inputs(1, L + 5, 2, 2, 64, 64, seed=L, packed=True))
    yield {k: t if k in ("A", "dt_bias", "h0") else t[:, :L] for k, t in d.items()}


@pytest.mark.parametrize("L", [1, 2, 30, 200])
def test_prefills_are_looked_at_in_c(monkeypatch, L):
    names = mm._names()
    counting = Counting(names.calls)
    for n, d in enumerate(layouts(L)):
        args = (d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"])
        monkeypatch.setattr(names, "calls", counting)
        y, h = mm.gdr_fwd(*args)
        assert counting.answered == n + 1, f"layout {n}: left to ctypes"
        monkeypatch.setattr(names, "calls", None)
        y2, h2 = mm.gdr_fwd(*args)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(h, h2)


def test_steps_and_projections_are_looked_at_in_c(monkeypatch):
    counting = Counting(mm._names().calls)
    monkeypatch.setattr(mm._names(), "calls", counting)
    _, one, q4 = operands()
    n = 0
    for B in (1, 3):
        d = to_cuda(gdr_inputs(B, None, 1, 2, 64, 64, F32, seed=5, packed=True))
        mm.gdr_state_update(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"])
        n += 1
        assert counting.answered == n
    for zeros, dtype in ((q4["zeros"], BF), (None, F32)):
        mm.proj_q4(q4["x"], q4["W"], q4["scales"], zeros, group=64, out_dtype=dtype)
        n += 1
        assert counting.answered == n
    torch.cuda.synchronize()
