"""Calls of the gated delta rule and of the 4-bit projection on a stream other
than the current one, with outputs that they allocate: the memory is not some
that work on the current stream still writes, nor handed out again while the
current stream still reads the result."""

import pytest
import torch

import mamba_selective_scan_core_b200 as mm
from gdr_ref import BF, F32, gdr_inputs, q4_inputs, to_cuda

pytestmark = pytest.mark.gpu

CYCLES = 20_000_000           # some 10 ms on the current stream


def prefill(seed, L):
    d = to_cuda(gdr_inputs(2, L, 1, 4, 64, 64, seed=seed))
    return lambda **kw: mm.gdr_fwd(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"], **kw)


def step(seed):
    d = to_cuda(gdr_inputs(64, None, 1, 4, 64, 64, seed=seed))
    return lambda **kw: (mm.gdr_state_update(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"].clone(), **kw),)


def project(seed):
    d = {k: t.cuda() for k, t in q4_inputs(16, 1000, 256, 64, seed=seed).items()}
    return lambda **kw: (mm.proj_q4(d["x"], d["W"], d["scales"], d["zeros"], group=64, out_dtype=BF, **kw),)


@pytest.mark.parametrize("make", [lambda s: prefill(s, 30), lambda s: prefill(s, 300), project], ids=["tokens", "chunks", "q4"])
def test_memory_of_another_stream(make):
    call, other = make(1), make(2)
    want, want2 = [t.clone() for t in call()], [t.clone() for t in other()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    # memory freed on the current stream, whose work there is still to come
    busy = [torch.empty_like(t) for t in want for _ in range(4)]
    taken = {t.data_ptr() for t in busy}
    torch.cuda._sleep(CYCLES)
    for t in busy:
        t.fill_(7)
    del t, busy
    got = call(stream=s)
    assert not taken & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # results still read on the current stream when they are freed
    torch.cuda._sleep(CYCLES)
    read = [t.clone() for t in got]
    held = {t.data_ptr() for t in got}
    del got
    got2 = other(stream=s)
    assert not held & {t.data_ptr() for t in got2}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, want)) and all(torch.equal(a, b) for a, b in zip(got2, want2))


def test_step_on_another_stream():
    call = step(3)
    want = call()[0].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    got = call(stream=torch.cuda.current_stream())[0]
    assert got.dtype == BF and torch.equal(got, want)
    d = to_cuda(gdr_inputs(64, None, 1, 4, 64, 64, F32, seed=3))
    torch.cuda.synchronize()
    busy = torch.empty(64, 4, 64, device="cuda")
    at = busy.data_ptr()
    torch.cuda._sleep(CYCLES)
    busy.fill_(7)
    del busy
    y = mm.gdr_state_update(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"], stream=s)
    assert y.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and not (y == 7).all()
