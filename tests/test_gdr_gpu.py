"""The gated delta rule (mamba_gdr_fwd, mamba_gdr_state_update) against its
definition in 64 bits.

Tolerances.  Token by token (fp32 activations, short calls, the one-token
step) a step's sums are of N <= 128 products in fp32, some 30 roundings of
2^-24 on a path, and the state's own two: 32 x 2^-24 = 2e-6 of the state's
norm, which the recurrence carries on with factors below 1; 1e-5 of the norm
leaves room for the steps that the decays keep.  In chunks the products'
operands are sums of two bf16 parts: a part is off by at most half a step,
2^-9 of what is split (bf16 keeps 8 bits), so two leave 2^-18, and a product
of two split factors leaves out lo x lo, another 2^-18: three split operands
a chunk (the solved rows, the state, the new values) make 6 x 2^-18 = 2.3e-5
at the very worst and, with rounding errors of either sign, about a quarter
of it in the norm: 1e-5 again.  A single element may be off by 40 times that
of the tensor's rms or its own size, whichever is larger.  bf16 outputs add
their own rounding, half a step, 2^-8 of the value."""

import pytest
import torch

import mamba_selective_scan_core_b200 as mm
from gdr_ref import BF, F32, gdr_inputs, gdr_reference, to_cuda

pytestmark = pytest.mark.gpu

NORM, MOST = 1e-5, 4e-4


def close(got, ref, name):
    got, stored = got.cpu().double(), got.dtype
    assert got.shape == ref.shape
    assert torch.isfinite(got).all(), f"{name}: not finite"
    if not ref.numel():
        return
    err = (got - ref).abs()
    if stored == BF:
        err = (err - 2.0 ** -8 * ref.abs()).clamp_min(0)
    rms = ref.square().mean().sqrt()
    assert err.square().mean().sqrt() <= NORM * rms, f"{name}: {(err.square().mean().sqrt() / rms).item():.3g} of the norm"
    assert (err <= MOST * torch.maximum(ref.abs(), rms)).all(), \
        f"{name}: an element off by {(err / torch.maximum(ref.abs(), rms)).max().item():.3g}"


def fwd(d, scale=None, eps=1e-6, **kw):
    return mm.gdr_fwd(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], d["h0"], scale=scale,
                      norm_eps=eps, **kw)


def step(d, state, scale=None, eps=1e-6, **kw):
    return mm.gdr_state_update(d["q"], d["k"], d["v"], d["dt"], d["beta"], d["dt_bias"], d["A"], state, scale=scale,
                               norm_eps=eps, **kw)


def check(inp, scale=None, eps=1e-6):
    N = inp["q"].shape[-1]
    y, h = fwd(to_cuda(inp), scale, eps)
    torch.cuda.synchronize()
    ry, rh = gdr_reference(inp, N ** -0.5 if scale is None else scale, eps)
    close(y, ry, "y")
    close(h, rh, "h_last")


@pytest.mark.parametrize("B,L,G,H,P,N", [
    (1, 1, 1, 1, 64, 64), (2, 2, 1, 2, 128, 128), (1, 7, 3, 3, 192, 64), (1, 63, 2, 4, 64, 128),
    (2, 64, 1, 1, 128, 128), (1, 65, 2, 2, 256, 64), (1, 127, 1, 4, 128, 128), (3, 128, 2, 2, 64, 64),
    (1, 129, 4, 4, 192, 128), (2, 300, 2, 6, 128, 128), (1, 515, 1, 2, 256, 128), (1, 1000, 2, 2, 64, 64)])
@pytest.mark.parametrize("act", [BF, F32])
def test_prefill(B, L, G, H, P, N, act):
    check(gdr_inputs(B, L, G, H, P, N, act, seed=B * 1000 + L + H))


@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("L", [5, 200])
@pytest.mark.parametrize("eps,unit,h0,bias,packed,scale", [
    (0.0, True, False, True, False, None), (1e-6, False, False, False, True, 1.0), (0.25, False, True, True, True, -0.3)])
def test_prefill_options(act, L, eps, unit, h0, bias, packed, scale):
    """Keys used as they are, a large eps, no initial state, no dt_bias, parts
    of a packed tensor, a given scale."""
    inp = gdr_inputs(2, L, 2, 4, 128, 128, act, seed=17 + L, h0=h0, packed=packed, unit=unit)
    if not bias:
        inp["dt_bias"] = None
        inp["dt"] -= 3
    check(inp, scale, eps)


@pytest.mark.parametrize("L", [33, 200])
def test_row_strides(L):
    """q, k and v with spare elements between their rows; what lies there is
    not read into the result."""
    inp = gdr_inputs(2, L, 1, 2, 64, 64, seed=5)
    d = to_cuda(inp)
    for name, pad in (("q", 8), ("k", 16), ("v", 24)):
        t = d[name]
        wide = torch.full((2, L, t.shape[2] * t.shape[3] + pad), float("nan"), dtype=BF, device="cuda")
        wide[..., :t.shape[2] * t.shape[3]] = t.flatten(2)
        d[name] = wide[..., :t.shape[2] * t.shape[3]].unflatten(-1, t.shape[2:])
    y, h = fwd(d)
    y0, h0 = fwd(to_cuda(inp))
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and torch.equal(h, h0)


@pytest.mark.parametrize("L", [20, 333])
@pytest.mark.parametrize("dt_mean", [-8.0, 5.0, 40.0])
def test_decays(L, dt_mean):
    """Almost no decay, a state forgotten within a few tokens, and decays that
    underflow to zero at each token."""
    check(gdr_inputs(1, L, 2, 2, 64, 128, seed=23, dt_mean=dt_mean))


@pytest.mark.parametrize("L", [20, 200])
def test_one_key_for_every_token(L):
    """The chunk's triangular system at its worst: every key the same, so each
    token takes out all that the ones before wrote."""
    inp = gdr_inputs(1, L, 1, 2, 64, 128, seed=29, same_key=True, dt_mean=-8.0)
    inp["beta"] += 4
    check(inp)


@pytest.mark.parametrize("L", [9, 100, 300])
def test_padded_batch(L):
    """Tokens with dt = beta = -inf leave the state as it is: sequences of
    different lengths, padded at the end, have the states of their own runs."""
    inp = gdr_inputs(3, L, 1, 2, 64, 64, seed=31)
    lens = (L, L // 2, 1)
    for b, n in enumerate(lens):
        inp["dt"][b, n:] = inp["beta"][b, n:] = float("-inf")
    y, h = fwd(to_cuda(inp))
    torch.cuda.synchronize()
    assert torch.isfinite(y).all()
    for b, n in enumerate(lens):
        one = {k: (t if k in ("A", "dt_bias") else t[b:b + 1] if k == "h0" else t[b:b + 1, :n]) for k, t in inp.items()}
        ry, rh = gdr_reference(one, 64 ** -0.5, 1e-6)
        close(y[b:b + 1, :n], ry, "y")
        close(h[b:b + 1], rh, "h_last")


@pytest.mark.parametrize("B,L,G,H,P,N", [(1, 2500, 1, 1, 64, 64), (1, 2049, 1, 2, 192, 128), (2, 1600, 1, 2, 128, 64),
                                         (1, 1985, 2, 2, 256, 128)])
@pytest.mark.parametrize("dt_mean", [0.0, -8.0])
def test_long_sequences_of_few_heads(B, L, G, H, P, N, dt_mean):
    """Sequences whose chunks run in segments at once, each from the state that
    the transitions of those before it give."""
    check(gdr_inputs(B, L, G, H, P, N, seed=L, dt_mean=dt_mean, h0=B == 1))


@pytest.mark.parametrize("B,L,H,cut", [(8, 64 * 130 + 5, 16, 4096), (1, 64 * 8192 + 1000, 2, 300000)])
def test_more_chunks_than_one_round(B, L, H, cut):
    """Chunks whose workspace is kept for part of the sequence at a time, of
    many heads and (in segments) of few: as two calls, the second from the
    first one's state."""
    P, N = 64, 64
    g = torch.Generator(device="cuda").manual_seed(97)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(BF)

    d = {"q": normal(B, L, 1, N), "k": normal(B, L, 1, N), "v": normal(B, L, H, P), "dt": normal(B, L, H) - 4,
         "beta": normal(B, L, H), "dt_bias": None, "A": -torch.ones(H, device="cuda"), "h0": None}
    y, h = fwd(d)

    def part(lo, hi, h0):
        return {n: t if n == "A" or t is None else t[:, lo:hi].contiguous() for n, t in d.items() if n != "h0"} | {"h0": h0}

    y1, h1 = fwd(part(0, cut, None))
    y2, h2 = fwd(part(cut, L, h1))
    torch.cuda.synchronize()
    # both are within NORM of the exact values, and the rounded y within its last bit
    assert (h - h2).norm() <= 2 * NORM * h.norm()
    ref = torch.cat([y1, y2], 1).double()
    err = ((y.double() - ref).abs() - 2.0 ** -7 * ref.abs()).clamp_min(0)
    assert err.norm() <= 2 * NORM * ref.norm()


@pytest.mark.parametrize("L", [40, 130])
def test_all_tokens_masked(L):
    """A sequence of padding alone: the state comes back bit for bit."""
    inp = gdr_inputs(2, L, 1, 1, 64, 128, seed=37)
    inp["dt"].fill_(float("-inf"))
    inp["beta"].fill_(float("-inf"))
    d = to_cuda(inp)
    _, h = fwd(d)
    torch.cuda.synchronize()
    assert torch.equal(h, d["h0"])


@pytest.mark.parametrize("L", [12, 150])
def test_zero_keys_and_queries(L):
    """Keys and queries of zeros (a masked token's): normalised, they stay zero."""
    inp = gdr_inputs(1, L, 1, 1, 64, 64, seed=41)
    inp["k"][:, 3:9] = 0
    inp["q"][:, 5:12] = 0
    check(inp)


def test_nothing_to_do():
    """seqlen 0 passes the state on (zeros without one); batch 0 does nothing."""
    for act in (BF, F32):
        d = to_cuda(gdr_inputs(2, 0, 1, 2, 64, 64, act, seed=43))
        y, h = fwd(d)
        torch.cuda.synchronize()
        assert y.shape == (2, 0, 2, 64) and torch.equal(h, d["h0"])
        _, h = fwd(dict(d, h0=None))
        torch.cuda.synchronize()
        assert torch.count_nonzero(h) == 0
        d = to_cuda(gdr_inputs(0, 5, 1, 2, 64, 64, act))
        y, h = fwd(d)
        assert y.numel() == h.numel() == 0
        d = to_cuda(gdr_inputs(0, None, 1, 2, 64, 64, act))
        assert step(d, d["h0"]).numel() == 0


@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("B,G,H,P,N,eps", [(1, 1, 1, 64, 64, 1e-6), (3, 2, 6, 192, 128, 1e-6), (5, 4, 4, 128, 64, 0.0),
                                           (2, 16, 32, 128, 128, 1e-6), (64, 8, 16, 256, 128, 1e-6)])
def test_step(act, B, G, H, P, N, eps):
    """One token, in place; small batches and one that takes the wide rows."""
    inp = gdr_inputs(B, None, G, H, P, N, act, seed=B + H, unit=eps == 0, packed=B % 2 == 0)
    d = to_cuda(inp)
    state = d["h0"].clone()
    y = step(d, state, eps=eps)
    torch.cuda.synchronize()
    ry, rh = gdr_reference(inp, N ** -0.5, eps)
    close(y, ry, "y")
    close(state, rh, "state")


@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("L", [2, 3, 4, 6, 8, 9, 16, 17, 31])
def test_few_tokens(act, L):
    """Groups of four tokens and blocks of eight that the sequence does not fill."""
    check(gdr_inputs(2, L, 2, 4, 64, 128 if L % 2 else 64, act, seed=200 + L, h0=L % 3 != 0, packed=L % 2 == 0))


@pytest.mark.parametrize("act,L", [(F32, 11), (BF, 7)])
def test_few_tokens_of_many_rows(act, L):
    """Enough state rows that a lane holds two of them."""
    check(gdr_inputs(10, L, 4, 16, 256, 64, act, seed=211))


@pytest.mark.parametrize("act,B,L,H,P", [(BF, 2, 20, 2, 64), (F32, 1, 30, 2, 64), (BF, 2, 200, 2, 128), (BF, 1, 2500, 1, 64)])
def test_forced_wait_timeout_is_reported_and_recoverable(monkeypatch, act, B, L, H, P):
    """Waits that give up at once, token by token, in chunks and in segments:
    the call's status and the device's say so, and the next call is right."""
    inp = gdr_inputs(B, L, 1, H, P, 64, act, seed=220)
    d = to_cuda(inp)
    ws = torch.full((mm.gdr_workspace_size(B, L, H, P, 64, 1, mm.MM_F32 if act == F32 else mm.MM_BF16),), 255, dtype=torch.uint8,
                    device="cuda")
    assert mm.fault_status(reset=True) == 0
    monkeypatch.setenv("MAMBA_MIXER_WAIT_LIMIT", "0")
    fwd(d, workspace=ws)
    assert mm.check_status(ws) == 11
    assert mm.fault_status(reset=True) == 11
    monkeypatch.delenv("MAMBA_MIXER_WAIT_LIMIT")
    y, h = fwd(d, workspace=ws)
    assert mm.check_status(ws) == 0 and mm.fault_status() == 0
    ry, rh = gdr_reference(inp, 64 ** -0.5, 1e-6)
    close(y, ry, "y")
    close(h, rh, "h_last")


@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("L", [1, 30, 200])
def test_both_ways_into_the_library(monkeypatch, act, L):
    """The C++ calls and the ctypes ones: the same bits, given outputs or not."""
    names = mm._names()
    assert names.calls is not None
    d = to_cuda(gdr_inputs(2, L, 1, 2, 64, 64, act, seed=230, packed=True))
    one = to_cuda(gdr_inputs(2, None, 1, 2, 64, 64, act, seed=231, packed=True))
    got = []
    for calls in (names.calls, None):
        monkeypatch.setattr(names, "calls", calls)
        y, h = fwd(d)
        out = torch.empty_like(y)
        y2, h2 = fwd(d, y=out, h_last=torch.empty_like(h), scale=64 ** -0.5)
        assert y2.data_ptr() == out.data_ptr()
        s = h.clone()
        got.append((y, h, y2, h2, step(one, s), s))
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.equal(got[0][0], got[0][2]) and torch.equal(got[0][1], got[0][3])


def test_workspace_given():
    """One that is too small is not used; one on the host is refused."""
    d = to_cuda(gdr_inputs(1, 300, 1, 2, 64, 64, seed=240))
    want = fwd(d)
    small = torch.full((256,), 7, dtype=torch.uint8, device="cuda")
    got = fwd(d, workspace=small)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (small == 7).all()
    with pytest.raises(ValueError):
        fwd(d, workspace=torch.empty(1 << 20, dtype=torch.uint8))


def test_calls_in_a_chain_without_waiting():
    """Prefills of three lengths, each from the state of the one before and on
    one workspace, and steps after them, queued at once: what the same calls
    give one by one."""
    lens = (300, 20, 2100)
    parts = [to_cuda(gdr_inputs(1, n, 1, 2, 128, 128, seed=250 + n)) for n in lens]
    one = to_cuda(gdr_inputs(1, None, 1, 2, 128, 128, seed=251))
    ws = torch.empty(max(mm.gdr_workspace_size(1, n, 2, 128, 128, 1) for n in lens), dtype=torch.uint8, device="cuda")

    def chain(wait):
        h, ys = torch.zeros(1, 2, 128, 128, device="cuda"), []
        for d in parts:
            y, h = fwd(dict(d, h0=h), workspace=ws)
            ys.append(y)
            if wait:
                torch.cuda.synchronize()
        for _ in range(3):
            ys.append(step(one, h))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return ys + [h]

    for a, b in zip(chain(True), chain(False)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("cut", [1, 64, 100])
def test_calls_continue_one_another(act, cut):
    """A prefill, a second one from its state, then single tokens: the whole
    sequence's values and state."""
    L = 200
    inp = gdr_inputs(2, L, 2, 4, 128, 128, act, seed=47)
    d = to_cuda(inp)

    def part(lo, hi, h0):
        return {k: (t if k in ("A", "dt_bias") else h0 if k == "h0" else t[:, lo:hi].contiguous()) for k, t in d.items()}

    y1, h = fwd(part(0, cut, d["h0"]))
    y2, h = fwd(part(cut, L - 3, h))
    ys = [y1, y2]
    for t in range(L - 3, L):
        c = {k: (t_ if k in ("A", "dt_bias", "h0") else t_[:, t].contiguous()) for k, t_ in d.items()}
        ys.append(step(c, h)[:, None])
    torch.cuda.synchronize()
    ry, rh = gdr_reference(inp, 128 ** -0.5, 1e-6)
    close(torch.cat(ys, 1), ry, "y")
    close(h, rh, "state")


@pytest.mark.parametrize("L", [30, 300])
def test_repeatable_with_a_dirty_workspace(L):
    """Two calls give the same bits whatever the workspace holds, and leave
    the rows around their outputs alone."""
    d = to_cuda(gdr_inputs(2, L, 1, 3, 64, 128, seed=53))
    n = mm.gdr_workspace_size(2, L, 3, 64, 128, 1)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    buf = torch.full((4, L, 3, 64), 7.0, dtype=BF, device="cuda")
    y1, h1 = fwd(d, workspace=ws, y=buf[1:3])
    assert mm.check_status(ws) == 0
    y2, h2 = fwd(d, workspace=torch.zeros_like(ws))
    torch.cuda.synchronize()
    assert torch.equal(y1, y2) and torch.equal(h1, h2)
    assert (buf[0] == 7).all() and (buf[3] == 7).all()


@pytest.mark.parametrize("L", [30, 300])
def test_two_streams_at_once(L):
    """Two calls side by side on two streams, each with a workspace of its own."""
    ds = [to_cuda(gdr_inputs(1, L, 2, 4, 128, 128, seed=s)) for s in (59, 61)]
    want = [fwd(d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = []
    for d, s in zip(ds, streams):
        got.append([fwd(d, stream=s) for _ in range(5)])
    torch.cuda.synchronize()
    for rs, (y, h) in zip(got, want):
        for y1, h1 in rs:
            assert torch.equal(y, y1) and torch.equal(h, h1)


@pytest.mark.parametrize("L", [30, 300])
def test_graph_replay(L):
    """Captured prefill and step, replayed with new inputs in the same buffers."""
    a, b = (to_cuda(gdr_inputs(2, L, 1, 2, 128, 128, seed=s)) for s in (67, 71))
    one = to_cuda(gdr_inputs(2, None, 1, 2, 128, 128, seed=73))
    want = []
    for d in (a, b):
        y, h = fwd(d)
        want.append((y, step(one, h), h))
    torch.cuda.synchronize()
    ws = torch.empty(mm.gdr_workspace_size(2, L, 2, 128, 128, 1), dtype=torch.uint8, device="cuda")
    cur = {k: v.clone() for k, v in a.items()}
    y, h, y1 = (torch.empty_like(t) for t in (want[0][0], want[0][2], want[0][1]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fwd(cur, workspace=ws, y=y, h_last=h)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd(cur, workspace=ws, y=y, h_last=h)
        step(one, h, y=y1)
    for d, (wy, w1, wh) in ((b, want[1]), (a, want[0]), (a, want[0])):
        for k in cur:
            cur[k].copy_(d[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, wy) and torch.equal(y1, w1) and torch.equal(h, wh)
    assert mm.check_status(ws) == 0


def test_launch_failure_is_reported(monkeypatch):
    d = to_cuda(gdr_inputs(1, 100, 1, 1, 64, 64, seed=79))
    monkeypatch.setenv("MAMBA_MIXER_TEST_LAUNCH_FAIL", "1")
    with pytest.raises(mm.MixerError):
        fwd(d)
    with pytest.raises(mm.MixerError):
        step({k: (v if k in ("A", "dt_bias", "h0") else v[:, 0].contiguous()) for k, v in d.items()}, d["h0"].clone())
    monkeypatch.delenv("MAMBA_MIXER_TEST_LAUNCH_FAIL")
    fwd(d)
    torch.cuda.synchronize()


def test_binding_refuses():
    d = to_cuda(gdr_inputs(2, 8, 1, 2, 64, 64, seed=83))
    with pytest.raises(TypeError):
        fwd(dict(d, q=d["q"].float()))
    with pytest.raises(ValueError):
        fwd(dict(d, k=d["k"].transpose(0, 1).contiguous().transpose(0, 1)))       # tokens not evenly spaced
    with pytest.raises(ValueError):
        fwd(dict(d, v=d["v"][..., ::2]))                        # rows not dense (and the wrong width)
    with pytest.raises(ValueError):
        fwd(dict(d, k=d["k"][:1].expand(2, 8, 1, 64)))          # both sequences the same rows: no row stride says that
    with pytest.raises(ValueError):
        fwd(dict(d, h0=d["h0"].cpu()))
    with pytest.raises(mm.MixerError) as e:
        fwd(d, eps=float("nan"))
    assert e.value.status == 12
    with pytest.raises(mm.MixerError) as e:
        fwd(d, h_last=d["h0"])
    assert e.value.status == 5
