"""The gated delta rule with a token that is not finite: what the formulas
make of it is not finite (its own output and, but for a query, the state and
the outputs that follow: of one state row where it is a value, of the whole
head otherwise), and everything else is bit for bit what it is without it.
One token at a time, in groups, in chunks and in segments of chunks."""

import pytest
import torch

import mamba_selective_scan_core_b200 as mm
from gdr_ref import BF, F32, gdr_inputs, to_cuda

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
G, H, P, N = 2, 4, 64, 64


def fwd(inp, eps):
    d = to_cuda(inp)
    y, h = mm.gdr_fwd(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"], norm_eps=eps)
    torch.cuda.synchronize()
    return y.cpu(), h.cpu()


def spoil(inp, name, value, b, t, at):
    """One input of token t of sequence b; returns the masks of the outputs and
    of the state that it reaches."""
    inp = dict(inp, **{name: inp[name].clone()})
    B, L = inp["v"].shape[:2]
    ys, hs = torch.zeros(B, L, H, P, dtype=torch.bool), torch.zeros(B, H, P, N, dtype=torch.bool)
    if name == "v":
        h, p = at % H, at % P
        inp[name][b, t, h, p] = value
        ys[b, t:, h, p] = hs[b, h, p] = True
    elif name in ("q", "k"):
        g = at % G
        inp[name][b, t, g, at % N] = value
        heads = slice(g * (H // G), (g + 1) * (H // G))
        if name == "q":
            ys[b, t, heads] = True
        else:
            ys[b, t:, heads] = hs[b, heads] = True
    else:
        h = at % H
        inp[name][b, t, h] = value
        ys[b, t:, h] = hs[b, h] = True
    return inp, ys, hs


@pytest.mark.parametrize("act,L,eps", [(BF, 30, 1e-6), (F32, 40, 0.0), (BF, 200, 1e-6), (BF, 200, 0.0), (BF, 2500, 1e-6)])
@pytest.mark.parametrize("name,value", [("v", NAN), ("v", INF), ("v", -INF), ("k", NAN), ("k", INF), ("q", NAN), ("q", -INF),
                                        ("dt", NAN), ("beta", NAN)])
def test_no_token_before_it_changes(act, L, eps, name, value):
    inp = gdr_inputs(2, L, G, H, P, N, act, seed=L, unit=eps == 0)
    y0, h0 = fwd(inp, eps)
    assert torch.isfinite(y0).all() and torch.isfinite(h0).all()
    for b, t, at in ((0, 0, 0), (1, 5, 7), (0, L // 2 + 1, 62), (1, L - 3, 33), (0, L - 1, 3)):
        bad, ys, hs = spoil(inp, name, value, b, t, at)
        y, h = fwd(bad, eps)
        assert torch.equal(y[~ys], y0[~ys]), f"token {t}: an output it does not reach"
        assert torch.equal(h[~hs], h0[~hs]), f"token {t}: a state it does not reach"
        assert not torch.isfinite(y[ys]).any(), f"token {t}: a finite output behind it"
        assert not torch.isfinite(h[hs]).any(), f"token {t}: a finite state behind it"


@pytest.mark.parametrize("act", [BF, F32])
def test_one_token(act):
    inp = gdr_inputs(2, 1, G, H, P, N, act, seed=9)
    one = lambda d: {k: t if k in ("A", "dt_bias", "h0") else t[:, 0].contiguous() for k, t in d.items()}  # noqa: E731

    def step(inp):
        d = to_cuda(one(inp))
        y = mm.gdr_state_update(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"])
        torch.cuda.synchronize()
        return y.cpu(), d["h0"].cpu()

    y0, h0 = step(inp)
    for name, value in (("v", NAN), ("v", INF), ("k", NAN), ("k", INF), ("q", NAN), ("dt", NAN), ("beta", NAN)):
        bad, ys, hs = spoil(inp, name, value, 1, 0, 5)
        y, h = step(bad)
        assert torch.equal(y[~ys[:, 0]], y0[~ys[:, 0]]) and torch.equal(h[~hs], h0[~hs])
        assert not torch.isfinite(y[ys[:, 0]]).any() and not torch.isfinite(h[hs]).any()
