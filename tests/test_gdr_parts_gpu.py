"""The gated delta rule for more sequences than its workspace holds at once:
they go in parts, and each is what it is by itself."""

import pytest
import torch

import mamba_selective_scan_core_b200 as mm
from gdr_ref import BF

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,L,H,given", [(600, 140, 64, True), (260, 200, 65, False)])
def test_many_sequences(B, L, H, given):
    P, N = 64, 64
    g = torch.Generator(device="cuda").manual_seed(B)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    d = {"q": normal(B, L, 1, N).to(BF), "k": normal(B, L, 1, N).to(BF), "v": normal(B, L, H, P).to(BF),
         "dt": normal(B, L, H).to(BF), "beta": normal(B, L, H).to(BF)}
    A, h0 = -torch.rand(H, device="cuda") - 0.1, normal(B, H, P, N) if given else None
    ws = torch.full((mm.gdr_workspace_size(B, L, H, P, N, 1),), 255, dtype=torch.uint8, device="cuda")
    y, h = mm.gdr_fwd(*d.values(), None, A, h0, workspace=ws)
    assert mm.check_status(ws) == 0
    for lo, hi in ((0, 3), (B // 3 - 2, B // 3 + 3), (B // 2 - 2, B // 2 + 2), (B - 2, B)):
        y1, h1 = mm.gdr_fwd(*(t[lo:hi].contiguous() for t in d.values()), None, A, h0[lo:hi] if given else None)
        assert torch.equal(y[lo:hi], y1) and torch.equal(h[lo:hi], h1)
