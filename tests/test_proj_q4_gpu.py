"""The projection with 4-bit weights (mamba_proj_q4) against its definition in
64 bits.

Tolerance.  c - 8, 8 - z and x enter exactly; a sum over K inputs in fp32, in
whatever order, is off by at most the number of additions on a path times
2^-24 of the sum of the terms' magnitudes.  A path runs through K / 32 / 2
accumulations of mma products (16 inputs each, counted as 16), the group's
scaling and the joins of at most 16 parts: the bound below takes K / 4 + 32
roundings, and the output's own: 2^-24 or, for bf16, half a step, 2^-8."""

import pytest
import torch

import mamba_selective_scan_core_b200 as mm
from gdr_ref import BF, F32, q4_inputs, q4_reference

pytestmark = pytest.mark.gpu


def check(inp, group, dtype):
    d = {k: None if t is None else t.cuda() for k, t in inp.items()}
    out = mm.proj_q4(d["x"], d["W"], d["scales"], d["zeros"], group=group, out_dtype=dtype)
    torch.cuda.synchronize()
    ref, mag = q4_reference(inp, group)
    K = inp["x"].shape[1]
    bound = (K / 4 + 32) * 2.0 ** -24 * mag + (2.0 ** -8 if dtype == BF else 2.0 ** -24) * ref.abs()
    err = (out.cpu().double() - ref).abs()
    assert (err <= bound).all(), f"{(err / bound.clamp_min(1e-300)).max().item():.3g} of the bound"
    # and in the norm: fp32 sums are far better than their worst case
    if dtype == F32:
        assert err.norm() <= 2e-6 * ref.norm() + 1e-30
    return out


@pytest.mark.parametrize("M,N,K,group", [(1, 1, 32, 32), (1, 8, 64, 64), (2, 63, 128, 128), (3, 64, 256, 64),
                                         (8, 65, 288, 32), (9, 1000, 544, 32), (16, 128, 1024, 128), (17, 72, 640, 128),
                                         (32, 257, 2048, 64), (33, 40, 384, 128), (64, 100, 4096, 128), (65, 33, 96, 32),
                                         (130, 66, 320, 64), (1, 288, 8192, 64), (5, 4097, 1056, 32)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_projection(M, N, K, group, zeros, dtype):
    check(q4_inputs(M, N, K, group, seed=M + N + K, zeros=zeros), group, dtype)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_zero_points_between_the_numbers(group):
    check(q4_inputs(4, 130, 512, group, seed=3, fractional=True), group, F32)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_where_each_number_stands(group):
    """One input at a time: out[k, n] is weight n's k-th number (minus 8) times
    its group's scale, exactly."""
    K, N = 256, 70
    inp = q4_inputs(K, N, K, group, seed=7, zeros=False)
    inp["x"] = torch.eye(K, dtype=BF)
    out = check(inp, group, F32).cpu()
    W = inp["W"]
    c = torch.stack([W & 15, W >> 4], -1).reshape(N, K).float() - 8
    assert torch.equal(out.T, c * inp["scales"].float().repeat_interleave(group, -1))


def test_nothing_to_do():
    d = q4_inputs(0, 16, 128, 128)
    out = mm.proj_q4(*(d[k].cuda() for k in ("x", "W", "scales", "zeros")))
    assert out.shape == (0, 16)


def test_rows_around_the_output_are_left():
    d = {k: t.cuda() for k, t in q4_inputs(3, 65, 512, 64, seed=11).items()}
    buf = torch.full((5 * 65 + 16,), 7.0, dtype=F32, device="cuda")
    out = buf[8:8 + 3 * 65].view(3, 65)
    mm.proj_q4(d["x"], d["W"], d["scales"], d["zeros"], group=64, out=out)
    torch.cuda.synchronize()
    assert (buf[:8] == 7).all() and (buf[8 + 3 * 65:] == 7).all() and not (out == 7).any()


def test_streams_and_graph():
    """Calls side by side on two streams, and a captured one replayed on new
    rows, give the same bits as a call alone (no sum depends on an order)."""
    d = {k: t.cuda() for k, t in q4_inputs(5, 288, 8192, 64, seed=13).items()}
    args = (d["x"], d["W"], d["scales"], d["zeros"])
    want = mm.proj_q4(*args, group=64)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [mm.proj_q4(*args, group=64, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.empty_like(want)
    x = d["x"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mm.proj_q4(x, *args[1:], group=64, out=out)
    for rows in (d["x"], -d["x"], d["x"]):
        x.copy_(rows)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want if rows is d["x"] else -want)


def test_reported_failures(monkeypatch):
    d = {k: t.cuda() for k, t in q4_inputs(2, 70, 1024, 128, seed=17).items()}
    args = (d["x"], d["W"], d["scales"], d["zeros"])
    want = mm.proj_q4(*args)
    torch.cuda.synchronize()
    monkeypatch.setenv("MAMBA_MIXER_TEST_LAUNCH_FAIL", "1")
    with pytest.raises(mm.MixerError):
        mm.proj_q4(*args)
    monkeypatch.delenv("MAMBA_MIXER_TEST_LAUNCH_FAIL")
    assert mm.fault_status(reset=True) == 0
    monkeypatch.setenv("MAMBA_MIXER_WAIT_LIMIT", "0")
    mm.proj_q4(*args)
    torch.cuda.synchronize()
    assert mm.fault_status(reset=True) == 11
    monkeypatch.delenv("MAMBA_MIXER_WAIT_LIMIT")
    out = mm.proj_q4(*args)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and mm.fault_status() == 0


def test_binding_refuses():
    d = {k: t.cuda() for k, t in q4_inputs(2, 64, 256, 64).items()}
    with pytest.raises(TypeError):
        mm.proj_q4(d["x"].float(), d["W"], d["scales"], group=64)
    with pytest.raises(ValueError):
        mm.proj_q4(d["x"], d["W"], d["scales"], group=32)          # scales are for groups of 64
    with pytest.raises(ValueError):
        mm.proj_q4(d["x"][:, ::2], d["W"][:, :64], d["scales"][:, :2], group=64)
    with pytest.raises(TypeError):
        mm.proj_q4(d["x"], d["W"], d["scales"], group=64, out_dtype=torch.float16)


def test_forced_wait_timeout_is_reported_and_recoverable(monkeypatch):
    inp = q4_inputs(3, 200, 2048, 128, seed=11)
    d = {k: t.cuda() for k, t in inp.items()}
    assert mm.fault_status(reset=True) == 0
    monkeypatch.setenv("MAMBA_MIXER_WAIT_LIMIT", "0")
    mm.proj_q4(d["x"], d["W"], d["scales"], d["zeros"], group=128)
    torch.cuda.synchronize()
    assert mm.fault_status(reset=True) == 11
    monkeypatch.delenv("MAMBA_MIXER_WAIT_LIMIT")
    check(inp, 128, F32)
    assert mm.fault_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF])
def test_both_ways_into_the_library(monkeypatch, dtype):
    """The C++ call and the ctypes one: the same bits, a given output or not."""
    names = mm._names()
    assert names.calls is not None
    d = {k: t.cuda() for k, t in q4_inputs(3, 100, 512, 64, seed=12).items()}
    got = []
    for calls in (names.calls, None):
        monkeypatch.setattr(names, "calls", calls)
        out = torch.empty(3, 100, dtype=dtype, device="cuda")
        assert mm.proj_q4(d["x"], d["W"], d["scales"], d["zeros"], group=64, out=out) is out
        got += [out, mm.proj_q4(d["x"], d["W"], d["scales"], d["zeros"], group=64, out_dtype=dtype)]
    torch.cuda.synchronize()
    assert all(torch.equal(got[0], t) for t in got)
