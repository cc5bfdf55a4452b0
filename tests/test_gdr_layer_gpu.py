"""A layer of the gated delta rule as a serving program runs it: projections
with 4-bit weights on either side, a prompt's prefill, then single tokens in
place on its state, eagerly and from a captured graph.

Every stage is compared with its definition in 64 bits on the values that the
stage before it left on the GPU, so each has its own tolerance: those of
test_gdr_gpu.py and of test_proj_q4_gpu.py."""

import pytest
import torch

import mamba_selective_scan_core_b200 as mm
from gdr_ref import BF, F32, gdr_reference, q4_inputs, q4_reference
from test_gdr_gpu import close

pytestmark = pytest.mark.gpu

HIDDEN, G, H, P, N, GROUP = 256, 2, 4, 64, 64, 64
WIDTHS = (G * N, G * N, H * P, H, H)


class Layer:
    def __init__(self, seed):
        pad = -sum(WIDTHS) % 8                    # rows of the projection a multiple of 16 bytes
        self.inp = q4_inputs(1, sum(WIDTHS) + pad, HIDDEN, GROUP, seed=seed)
        self.out = q4_inputs(1, HIDDEN, H * P, GROUP, seed=seed + 1, zeros=False)
        g = torch.Generator().manual_seed(seed + 2)
        self.dt_bias, self.A = torch.randn(H, generator=g) - 3, -torch.rand(H, generator=g) * 4 - 0.1
        self.dev = {k: v.cuda() for k, v in (("Wi", self.inp["W"]), ("si", self.inp["scales"]), ("zi", self.inp["zeros"]),
                                             ("Wo", self.out["W"]), ("so", self.out["scales"]), ("b", self.dt_bias), ("A", self.A))}

    def project_in(self, x):
        """[..., HIDDEN] -> q, k, v as parts of one tensor, dt and beta."""
        d = self.dev
        row = mm.proj_q4(x.flatten(0, -2), d["Wi"], d["si"], d["zi"], group=GROUP, out_dtype=BF)
        q, k, v, dt, beta = row[:, :sum(WIDTHS)].unflatten(0, x.shape[:-1]).split(WIDTHS, -1)
        return (row, q.unflatten(-1, (G, N)), k.unflatten(-1, (G, N)), v.unflatten(-1, (H, P)), dt.contiguous(), beta.contiguous())

    def project_out(self, y):
        return mm.proj_q4(y.flatten(-2).flatten(0, -2), self.dev["Wo"], self.dev["so"], group=GROUP)

    def prefill(self, x):
        row, q, k, v, dt, beta = self.project_in(x)
        y, h = mm.gdr_fwd(q, k, v, dt, beta, self.dev["b"], self.dev["A"])
        return row, (q, k, v, dt, beta), y, h, self.project_out(y)

    def step(self, x, h):
        row, q, k, v, dt, beta = self.project_in(x)
        y = mm.gdr_state_update(q, k, v, dt, beta, self.dev["b"], self.dev["A"], h)
        return row, (q, k, v, dt, beta), y, self.project_out(y)

    def check(self, x, row, parts, h0, y, h, out):
        for rows, w, group, got in ((x, self.inp, GROUP, row), (y.flatten(-2), self.out, GROUP, out)):
            rows = rows.flatten(0, -2).cpu()
            ref, mag = q4_reference(dict(w, x=rows), group)
            bound = (rows.shape[1] / 4 + 32) * 2.0 ** -24 * mag + (2.0 ** -8 if got.dtype == BF else 2.0 ** -24) * ref.abs()
            assert ((got.cpu().double() - ref).abs() <= bound).all()
        q, k, v, dt, beta = (t.cpu() for t in parts)
        ry, rh = gdr_reference({"q": q, "k": k, "v": v, "dt": dt, "beta": beta, "dt_bias": self.dt_bias, "A": self.A, "h0": h0},
                               N ** -0.5, 1e-6)
        close(y, ry, "y")
        close(h, rh, "state")


@pytest.mark.parametrize("L", [30, 150])
def test_prefill_then_tokens(L):
    layer = Layer(300 + L)
    g = torch.Generator().manual_seed(L)
    x = torch.randn(2, L, HIDDEN, generator=g).to(BF).cuda()
    row, parts, y, h, out = layer.prefill(x)
    layer.check(x, row, parts, None, y, h, out)
    for _ in range(3):
        x1 = torch.randn(2, HIDDEN, generator=g).to(BF).cuda()
        before = h.cpu().clone()
        row, parts, y, out = layer.step(x1, h)
        layer.check(x1, row, parts, before, y, h, out)


def test_tokens_from_a_graph():
    layer = Layer(400)
    g = torch.Generator().manual_seed(1)
    xs = [torch.randn(3, HIDDEN, generator=g).to(BF).cuda() for _ in range(4)]
    h0 = torch.randn(3, H, P, N, generator=g).cuda()
    h, want = h0.clone(), []
    for x in xs:
        want.append(layer.step(x, h)[3].clone())
    x, state = xs[0].clone(), h0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(x, state)[3]
    state.copy_(h0)
    for src, ref in zip(xs, want):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert out.dtype == F32 and torch.equal(out, ref)
    assert torch.equal(state, h)
