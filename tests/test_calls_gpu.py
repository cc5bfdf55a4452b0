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
