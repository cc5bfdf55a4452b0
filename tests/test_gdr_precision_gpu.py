"""How exact the gated delta rule's chunked calls are: as exact as fp32.

Tolerances.  The products' operands are sums of three bf16 parts, each off by
at most half a step of what is left, 2^-9: 2^-27 of an operand stays out, less
than an fp32 rounding.  What a chunk rounds in fp32, in units of 2^-24: a
norm's rsqrt and a decay's exponential, 4 each, the 12 additions of a product
of up to 128 inputs taken 16 at a time and of its parts, and the state's own
update.  Of either sign they come to sqrt(4^2 + 4^2 + 13) = 6.7; decays take an
error along with the value that has it.  8 x 2^-24 of the norm for the state.

y has the same error before it is rounded to bf16.  Rounding then gives another
value than that of the exact result for a share |error| / step of the values,
one step off each; a step is at most 2^-7 of the value, so in the norm they
differ by at most sqrt(2^-7 x 8 x 2^-24) = 6.1e-5.  (Two parts of each operand
would leave 3e-7 to 1e-6 of the state and 1.3e-4 of y.)"""

import pytest
import torch

import mamba_selective_scan_core_b200 as mm
from gdr_ref import BF, gdr_inputs, gdr_reference, to_cuda

pytestmark = pytest.mark.gpu

NORM = 8 * 2.0 ** -24
ROUNDED = (2.0 ** -7 * NORM) ** 0.5


def off(got, ref):
    return ((got.double().cpu() - ref.double()).norm() / ref.double().norm()).item()


def check(y, h, ry, rh):
    assert off(h, rh) <= NORM, f"h_last: {off(h, rh):.3g} of the norm"
    assert off(y, ry.to(BF)) <= ROUNDED, f"y: {off(y, ry.to(BF)):.3g} of the norm"


@pytest.mark.parametrize("B,L,G,H,P,N,eps,h0", [
    (1, 1001, 2, 4, 64, 64, 1e-6, True), (2, 500, 1, 2, 128, 128, 1e-6, False), (1, 700, 2, 2, 64, 128, 0.0, True),
    (1, 4096, 1, 2, 64, 128, 1e-6, False), (1, 3000, 1, 1, 128, 64, 0.0, True)])
def test_chunks_are_as_exact_as_fp32(B, L, G, H, P, N, eps, h0):
    """In one pass and, the longer ones, in segments."""
    inp = gdr_inputs(B, L, G, H, P, N, seed=L, h0=h0, unit=eps == 0)
    d = to_cuda(inp)
    y, h = mm.gdr_fwd(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"], norm_eps=eps)
    torch.cuda.synchronize()
    check(y, h, *gdr_reference(inp, N ** -0.5, eps))


def test_rounds_are_as_exact_as_fp32():
    """A call whose chunks run in several rounds, two of its heads."""
    B, L, H, P, N = 8, 64 * 130 + 5, 16, 64, 64
    g = torch.Generator(device="cuda").manual_seed(101)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(BF)

    q, k, v = normal(B, L, 1, N), normal(B, L, 1, N), normal(B, L, H, P)
    dt, beta, A = normal(B, L, H) - 4, normal(B, L, H), -torch.ones(H, device="cuda")
    y, h = mm.gdr_fwd(q, k, v, dt, beta, None, A)
    torch.cuda.synchronize()
    for b, n in ((0, 0), (7, 14)):
        one = {"q": q[b:b + 1], "k": k[b:b + 1], "v": v[b:b + 1, :, n:n + 2], "dt": dt[b:b + 1, :, n:n + 2],
               "beta": beta[b:b + 1, :, n:n + 2], "A": A[n:n + 2]}
        ry, rh = gdr_reference({**{name: t.cpu() for name, t in one.items()}, "dt_bias": None, "h0": None}, N ** -0.5, 1e-6)
        check(y[b:b + 1, :, n:n + 2], h[b:b + 1, n:n + 2], ry, rh)
