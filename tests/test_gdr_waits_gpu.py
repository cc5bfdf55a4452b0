"""The gated delta rule's prefill with waits of a few tries, which some of a
call's warps get through and others do not: a call is either right or reported
as failed, by its workspace and by the device, and the next one is right."""

import pytest
import torch

import mamba_selective_scan_core_b200 as mm
from gdr_ref import BF, F32, gdr_inputs, to_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,B,L,H,P,N", [(F32, 1, 100, 8, 64, 128), (BF, 2, 300, 4, 128, 64), (BF, 1, 2500, 2, 64, 128)],
                         ids=["tokens", "chunks", "segments"])
def test_waits_that_give_up_part_of_the_way(monkeypatch, act, B, L, H, P, N):
    d = to_cuda(gdr_inputs(B, L, 1, H, P, N, act, seed=L))
    ws = torch.empty(mm.gdr_workspace_size(B, L, H, P, N, 1, mm.MM_F32 if act == F32 else mm.MM_BF16), dtype=torch.uint8, device="cuda")

    def fwd():
        return mm.gdr_fwd(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"], workspace=ws)

    want = fwd()
    torch.cuda.synchronize()
    assert mm.fault_status(reset=True) == 0
    for limit in (1, 2, 3, 4, 6, 8, 12, 16, 32):
        for _ in range(5):
            monkeypatch.setenv("MAMBA_MIXER_WAIT_LIMIT", str(limit))
            got = fwd()
            monkeypatch.delenv("MAMBA_MIXER_WAIT_LIMIT")
            status = mm.check_status(ws)
            assert status in (0, 11) and mm.fault_status(reset=True) == status
            if status == 0:
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = fwd()
    assert mm.check_status(ws) == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
