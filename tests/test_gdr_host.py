"""Argument checks of the gated delta rule and of the 4-bit projection, on the
host: every call runs in a child process that sees no CUDA device, so one that
passes them ends at the device check with MM_ERR_DEVICE."""

import pytest

import mamba_selective_scan_core_b200 as mm
from abi_nodevice import NoDeviceLib
from mamba_selective_scan_core_b200 import build as mmbuild

OK, ENULL, ESHAPE, EALIGN, EDTYPE, EALIAS, EUNSUP, ECUDA, EDEVICE, EWORKSPACE, ESCRATCH, ETIMEOUT, EARG = range(13)
BASE = 1 << 40
AT = {name: BASE + (i << 33) for i, name in enumerate(
    ("q", "k", "v", "dt", "beta", "dt_bias", "A", "h0", "y", "h_last", "ws"))}
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def L():
    mmbuild.build()
    mm.lib()
    worker = NoDeviceLib()
    yield worker
    worker.close()


def fwd_args(B=2, Lq=300, G=2, H=4, P=128, N=64, qs=None, ks=None, vs=None, scale=0.1, eps=1e-6, act=BF16,
             ws_bytes=None, **over):
    p = dict(AT, **over)
    if ws_bytes is None:
        ws_bytes = mm.gdr_workspace_size(B, Lq, H, P, N, G, act)
    return [p[k] for k in ("q", "k", "v", "dt", "beta", "dt_bias", "A", "h0", "y", "h_last")] + [
        B, Lq, G, H, P, N, G * N if qs is None else qs, G * N if ks is None else ks, H * P if vs is None else vs,
        scale, eps, act, p["ws"], ws_bytes, None]


def step_args(B=2, G=2, H=4, P=128, N=64, qs=None, ks=None, vs=None, scale=0.1, eps=1e-6, act=BF16, **over):
    p = dict(AT, **over)
    return [p[k] for k in ("q", "k", "v", "dt", "beta", "dt_bias", "A", "h0", "y")] + [
        B, G, H, P, N, G * N if qs is None else qs, G * N if ks is None else ks, H * P if vs is None else vs,
        scale, eps, act, None]


def q4_args(M=3, N=100, K=1024, group=128, dtype=BF16, **over):
    p = dict({k: BASE + (i << 36) for i, k in enumerate(("x", "W", "scales", "zeros", "out"))}, **over)
    return [p[k] for k in ("x", "W", "scales", "zeros", "out")] + [M, N, K, group, dtype, None]


@pytest.mark.parametrize("act", [F32, BF16])
@pytest.mark.parametrize("which", ["fwd", "step"])
def test_gdr_sizes(L, which, act):
    call, args = (L.mamba_gdr_fwd, fwd_args) if which == "fwd" else (L.mamba_gdr_state_update, step_args)
    run = lambda **kw: call(*args(act=act, **kw))  # noqa: E731
    assert run() == EDEVICE
    assert run(dt_bias=None) == EDEVICE
    for P in (64, 128, 192, 256):
        for N in (64, 128):
            assert run(P=P, N=N) == EDEVICE
    for over in (dict(P=32), dict(P=96), dict(P=320), dict(N=32), dict(N=96), dict(N=256)):
        assert run(**over) == EUNSUP, over
    for over in (dict(H=5), dict(G=0), dict(H=0), dict(B=-1), dict(G=3), dict(B=65536), dict(qs=64), dict(ks=127),
                 dict(vs=511), dict(qs=-128), dict(vs=1 << 40)):
        assert run(**over) == ESHAPE, over
    # rows that are no multiple of 16 bytes apart
    assert run(qs=130) == run(ks=2 * 64 + 2) == run(vs=513) == EALIGN
    assert run(qs=136, ks=144, vs=520) == EDEVICE
    for over in (dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(scale=float("nan")),
                 dict(scale=float("-inf"))):
        assert run(**over) == EARG, over
    assert run(eps=0.0, scale=0.0) == EDEVICE
    assert call(*args(act=2)) == EDTYPE
    assert run(B=0) == OK


def test_gdr_fwd_pointers(L):
    f = L.mamba_gdr_fwd
    assert f(*fwd_args(h0=None)) == EDEVICE
    for name in ("q", "k", "v", "dt", "beta", "A", "y", "h_last"):
        assert f(*fwd_args(**{name: None})) == ENULL, name
    assert f(*fwd_args(Lq=0, q=None, k=None, v=None, dt=None, beta=None, y=None)) == EDEVICE
    assert f(*fwd_args(Lq=-1, ws_bytes=0)) == ESHAPE
    assert f(*fwd_args(Lq=(1 << 30) + 1, ws_bytes=0)) == ESHAPE
    for name in ("q", "k", "v", "dt", "beta", "dt_bias", "A", "h0", "y", "h_last", "ws"):
        assert f(*fwd_args(**{name: AT[name] + 8})) == EALIGN, name
    for out in ("y", "h_last"):
        for name in ("q", "k", "v", "dt", "beta", "dt_bias", "A", "h0"):
            assert f(*fwd_args(**{out: AT[name]})) == EALIAS, (out, name)
    assert f(*fwd_args(y=AT["h_last"])) == EALIAS
    for name in ("q", "v", "h0", "y", "h_last"):
        assert f(*fwd_args(ws=AT[name])) == EALIAS, name
    need = mm.gdr_workspace_size(2, 300, 4, 128, 64, 2)
    assert f(*fwd_args(ws_bytes=need - 16)) == EWORKSPACE
    assert f(*fwd_args(ws=None)) == EWORKSPACE
    # parts of one packed tensor: rows of q | k | v, 256 + 512 elements
    packed = dict(q=BASE, k=BASE + 128 * 2, v=BASE + 256 * 2, qs=768, ks=768, vs=768)
    assert f(*fwd_args(**packed)) == EDEVICE
    # y in the gap behind v's last row but one still lies inside v's span
    assert f(*fwd_args(**dict(packed, y=BASE + 599 * 768 * 2))) == EALIAS
    assert f(*fwd_args(**dict(packed, y=BASE + 600 * 768 * 2))) == EDEVICE


def test_gdr_step_pointers(L):
    f = L.mamba_gdr_state_update
    for name in ("q", "k", "v", "dt", "beta", "A", "h0", "y"):
        assert f(*step_args(**{name: None})) == ENULL, name
    for name in ("q", "k", "v", "dt", "beta", "dt_bias", "A", "h0", "y"):
        assert f(*step_args(**{name: AT[name] + 8})) == EALIGN, name
    for name in ("q", "k", "v", "dt", "beta", "dt_bias", "A"):
        assert f(*step_args(h0=AT[name])) == EALIAS, name
        assert f(*step_args(y=AT[name])) == EALIAS, name
    assert f(*step_args(y=AT["h0"])) == EALIAS


def test_gdr_workspace_size():
    assert mm.gdr_workspace_size(2, 0, 4, 128, 64, 2) == 256
    assert mm.gdr_workspace_size(2, 4096, 4, 128, 64, 2, act=mm.MM_F32) == 256      # token by token
    for bad in (dict(headdim=96), dict(d_state=32), dict(groups=3), dict(batch=0), dict(seqlen=-1), dict(act=5)):
        assert mm.gdr_workspace_size(**dict(dict(batch=2, seqlen=64, heads=4, headdim=128, d_state=64, groups=2), **bad)) == 0


def test_q4(L):
    f = L.mamba_proj_q4
    assert f(*q4_args()) == f(*q4_args(zeros=None)) == f(*q4_args(dtype=F32)) == EDEVICE
    for group in (32, 64, 128):
        assert f(*q4_args(group=group)) == EDEVICE
    assert f(*q4_args(N=1, M=1, K=32, group=32)) == EDEVICE
    for group in (0, 16, 256, -32):
        assert f(*q4_args(group=group)) == EUNSUP
    for over in (dict(K=1000), dict(K=1024 + 64), dict(K=0), dict(N=0), dict(M=-1), dict(M=65535 * 64 + 1), dict(N=1 << 31)):
        assert f(*q4_args(**over)) == ESHAPE, over
    assert f(*q4_args(dtype=2)) == EDTYPE
    assert f(*q4_args(M=0)) == OK
    for i, name in enumerate(("x", "W", "scales", "zeros", "out")):
        if name != "zeros":
            assert f(*q4_args(**{name: None})) == ENULL, name
        assert f(*q4_args(**{name: BASE + (i << 36) + 8})) == EALIGN, name
        if name != "out":
            assert f(*q4_args(out=BASE + (i << 36))) == EALIAS, name
