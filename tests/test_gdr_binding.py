"""What the Python calls of the gated delta rule let through to the library,
on the CPU: tensors that say they are on a device, and a library that counts
its calls and runs nothing."""

import pytest
import torch

import mamba_selective_scan_core_b200 as mm
from gdr_ref import BF, F32, gdr_inputs
from mamba_selective_scan_core_b200 import build as mmbuild


class OnDevice(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda", 0)

    def get_device(self):
        return 0


class CountingLibrary:
    def __init__(self):
        self.calls = []

    def mamba_gdr_workspace_size(self, *args):
        return 256

    def mamba_gdr_fwd(self, *args):
        self.calls.append("fwd")
        return 0

    def mamba_gdr_state_update(self, *args):
        self.calls.append("step")
        return 0


@pytest.fixture
def library(monkeypatch):
    mmbuild.build()
    names = mm._names()
    counting = CountingLibrary()
    monkeypatch.setattr(names, "calls", None)
    monkeypatch.setattr(names, "lib", counting)
    monkeypatch.setattr(names, "current_device", lambda: 0)
    monkeypatch.setattr(names, "raw_stream", lambda i: 0)
    return counting


def on_device(inp):
    return {k: None if t is None else t.as_subclass(OnDevice) for k, t in inp.items()}


def fwd(d, **kw):
    return mm.gdr_fwd(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"], **kw)


def step(d):
    return mm.gdr_state_update(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"])


@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("name", ["q", "k"])
def test_sizes_of_q_and_k(library, act, name):
    """q or k with fewer sequences or tokens than v, which the kernels would read past."""
    d = on_device(gdr_inputs(3, 20, 1, 2, 64, 64, act))
    fwd(d)
    assert library.calls == ["fwd"]
    for t in (d[name][:1], d[name][:2], d[name][:, :7], d[name][:1, :7].contiguous(), d[name][:, :7].contiguous(), d[name][:0]):
        with pytest.raises(ValueError, match=name):
            fwd(dict(d, **{name: t}))
    one = on_device(gdr_inputs(3, None, 1, 2, 64, 64, act))
    step(one)
    for n in (0, 1, 2):
        with pytest.raises(ValueError, match=name):
            step(dict(one, **{name: one[name][:n]}))
    single = on_device(gdr_inputs(1, 1, 1, 2, 64, 64, act))
    fwd(single)
    with pytest.raises(ValueError, match=name):
        fwd(dict(single, **{name: single[name][:, :0]}))
    assert library.calls == ["fwd", "step", "fwd"]


def test_workspace_in_one_piece(library):
    """A workspace whose bytes are not one block of memory (one byte expanded,
    every other byte) is refused: its nbytes is not what lies behind its address."""
    d = on_device(gdr_inputs(1, 20, 1, 2, 64, 64))
    ws = torch.empty(4096, dtype=torch.uint8).as_subclass(OnDevice)
    fwd(d, workspace=ws)
    for bad in (ws[:1].expand(4096), ws[::2], ws.view(64, 64)[:, :32]):
        with pytest.raises(ValueError, match="workspace"):
            fwd(d, workspace=bad)
    assert library.calls == ["fwd"]


@pytest.mark.parametrize("B,L,H,P,N", [(1024, 64, 128, 64, 64), (65535, 100, 16, 64, 64), (300, 4096, 64, 128, 128), (8, 70, 65535, 64, 64),
                                       (1, 1 << 20, 4096, 64, 128)])
def test_workspace_is_bounded(B, L, H, P, N):
    """However many sequences: 50 KB for each of 16384 chunks of a head (or one
    of each head, where a sequence has more), two states of the heads at work
    where their chunks take several rounds, and a segment's states and
    transitions for the few heads of calls that have segments."""
    units = max(16384, H)
    bound = 256 + units * (5 * 64 * 4 + 6 * 64 * 128) + 2 * units * P * N * 4 + 32 * 256 * (2 * P + N) * N * 4
    assert 256 < mm.gdr_workspace_size(B, L, H, P, N, 1) <= bound
    assert mm.gdr_workspace_size(B, L, H, P, N, 1) <= mm.gdr_workspace_size(B, 4 * L, H, P, N, 1)


@pytest.mark.parametrize("B,L,H,P,N,chunks", [
    (1, 48, 2, 64, 64, False), (1, 64, 16, 128, 64, False), (1, 24, 32, 128, 128, False), (32, 16, 32, 64, 64, False),
    (16, 16, 64, 128, 64, False), (64, 16, 64, 64, 64, False), (32, 16, 32, 64, 128, False),
    (1, 128, 2, 64, 64, True), (1, 128, 16, 128, 128, True), (4, 48, 32, 128, 64, True), (4, 32, 32, 128, 128, True),
    (8, 48, 64, 128, 64, True), (16, 48, 64, 128, 128, True), (64, 64, 64, 64, 128, True), (1, 129, 1, 64, 64, True)])
def test_which_calls_run_in_chunks(B, L, H, P, N, chunks):
    """Sizes at which the other form took 1.25 to 2.2 times as long; a call that
    is not in chunks has no workspace but its status."""
    mmbuild.build()
    assert (mm.gdr_workspace_size(B, L, H, P, N, 1) > 256) == chunks
    assert mm.gdr_workspace_size(B, L, H, P, N, 1, act=mm.MM_F32) == 256
