"""The projection with 4-bit weights where its calls end: waits that give up
part of the way, the longest rows, inputs that are not finite."""

import pytest
import torch

import mamba_selective_scan_core_b200 as mm
from gdr_ref import BF, F32, q4_inputs, q4_reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,group,zeros", [(1, 1000, 8192, 128, False), (20, 300, 4096, 32, True)])
def test_waits_that_give_up_part_of_the_way(monkeypatch, M, N, K, group, zeros):
    """Waits of a few tries, which some warps get through and others do not: a
    call is either right or reported, and the next one is right."""
    d = {k: None if t is None else t.cuda() for k, t in q4_inputs(M, N, K, group, seed=M, zeros=zeros).items()}
    args = (d["x"], d["W"], d["scales"], d["zeros"])
    want = mm.proj_q4(*args, group=group)
    torch.cuda.synchronize()
    assert mm.fault_status(reset=True) == 0
    for limit in (1, 2, 3, 4, 6, 8, 12, 16, 32):
        for _ in range(20):
            monkeypatch.setenv("MAMBA_MIXER_WAIT_LIMIT", str(limit))
            got = mm.proj_q4(*args, group=group)
            torch.cuda.synchronize()
            monkeypatch.delenv("MAMBA_MIXER_WAIT_LIMIT")
            status = mm.fault_status(reset=True)
            assert status in (0, 11)
            if status == 0:
                assert torch.equal(got, want)
    assert torch.equal(mm.proj_q4(*args, group=group), want) and mm.fault_status() == 0


def test_the_longest_row():
    """K = 2^31 - 32, the largest that the call takes: a few inputs of one row,
    the last among them, whose sum is exact."""
    K = 2 ** 31 - 32
    x = torch.zeros(1, K, dtype=BF, device="cuda")
    W = torch.zeros(1, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.ones(1, K // 32, dtype=BF, device="cuda")
    want = 0.0
    for k, v, c in ((0, 1.0, 15), (255, 0.5, 3), (2 ** 30 + 5, 2.0, 11), (K - 33, -4.0, 1), (K - 1, 8.0, 13)):
        x[0, k] = v
        W[0, k // 2] = c << 4 if k % 2 else c
        want += v * (c - 8)
    out = mm.proj_q4(x, W, scales, group=32)
    torch.cuda.synchronize()
    assert out.item() == want


@pytest.mark.parametrize("M", [1, 3, 12, 20, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros,fractional", [(False, False), (True, False), (True, True)])
def test_inputs_that_are_not_finite(M, group, zeros, fractional):
    """Infinities and NaN in some rows of x: what the formula gives, infinity
    times c - z of either sign and NaN where that is 0; the other rows as ever."""
    K, N = 640, 70
    inp = q4_inputs(M, N, K, group, seed=M + group, zeros=zeros, fractional=fractional)
    inp["scales"] = inp["scales"].abs() + 0.01
    x, inf = inp["x"], float("inf")
    x[0, 5] = inf
    if M > 1:
        x[2, 300], x[2, K - 1] = -inf, -inf
    if M > 8:
        x[8, 7], x[8, 70], x[M - 1, 33], x[M - 2, 0], x[M - 2, 1] = inf, -inf, float("nan"), inf, -inf
    d = {k: None if t is None else t.cuda() for k, t in inp.items()}
    out = mm.proj_q4(d["x"], d["W"], d["scales"], d["zeros"], group=group).cpu().double()
    W = inp["W"].to(torch.int64)
    c = torch.stack([W & 15, W >> 4], -1).reshape(N, -1, group).double()
    z = 8.0 if inp["zeros"] is None else inp["zeros"].double()[..., None]
    w = ((c - z) * inp["scales"].double()[..., None]).reshape(N, K)
    ref = (x.double()[:, None, :] * w).sum(-1)
    odd = [m for m in range(M) if not torch.isfinite(x[m]).all()]
    assert torch.equal(out[odd].isnan(), ref[odd].isnan())
    assert torch.equal(out[odd].nan_to_num(nan=0.0), ref[odd].nan_to_num(nan=0.0))
    if M > 1:
        rest = [m for m in range(M) if m not in odd]
        clean, mag = q4_reference(dict(inp, x=x[rest]), group)
        assert ((out[rest] - clean).abs() <= (K / 4 + 32) * 2.0 ** -24 * mag + 2.0 ** -24 * clean.abs()).all()
