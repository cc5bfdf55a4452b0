"""Inputs and 64-bit results of the gated delta rule and of the 4-bit
projection, from their definitions, on the CPU."""

from __future__ import annotations

import math

import torch

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def gdr_inputs(B, L, G, H, P, N, act=BF, seed=0, h0=True, packed=False, unit=False, dt_mean=0.0, same_key=False):
    """One call's inputs on the CPU (L None: one token, no time axis).  q, k, v
    as a convolution with SiLU leaves them; unit: q and k of norm 1."""
    g = torch.Generator().manual_seed(seed)
    lead = (B,) if L is None else (B, L)

    def normal(*shape):
        return torch.randn(shape, generator=g)

    silu = torch.nn.functional.silu
    q, k, v = silu(normal(*lead, G, N)), silu(normal(*lead, G, N)), silu(normal(*lead, H, P))
    if same_key:
        k = k[..., :1, :, :].expand_as(k) if L is None else k[:, :1].expand_as(k)
    if unit:
        q, k = (t / t.norm(dim=-1, keepdim=True) for t in (q, k))
    q, k, v = (t.to(act).contiguous() for t in (q, k, v))
    if packed:
        qkv = torch.cat([t.flatten(-2) for t in (q, k, v)], -1)
        q, k, v = (t.unflatten(-1, s) for t, s in zip(qkv.split([G * N, G * N, H * P], -1), ((G, N), (G, N), (H, P))))
    step = torch.exp(torch.rand(H, generator=g) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
    return {"q": q, "k": k, "v": v, "dt": (normal(*lead, H) + dt_mean).to(act), "beta": normal(*lead, H).to(act),
            "dt_bias": step + torch.log(-torch.expm1(-step)), "A": -(torch.rand(H, generator=g) * 15 + 1),
            "h0": normal(B, H, P, N) * 0.1 if h0 else None}


def to_cuda(inp):
    """The inputs on the device; the parts of a packed tensor stay parts of one."""
    out = {}
    for name, t in inp.items():
        if t is None or t.is_contiguous() or name not in ("q", "k", "v"):
            out[name] = None if t is None else t.cuda()
        else:
            base = t._base
            out.setdefault("_base", base.cuda())
            out[name] = out["_base"].as_strided(t.shape, t.stride(), t.storage_offset())
    out.pop("_base", None)
    return out


def gdr_reference(inp, scale, eps):
    """(y, state) in 64 bits, token by token."""
    v = inp["v"].to(F64)
    one = v.dim() == 3
    q, k, dt, beta = (inp[n].to(F64) for n in ("q", "k", "dt", "beta"))
    if one:
        q, k, v, dt, beta = (t.unsqueeze(1) for t in (q, k, v, dt, beta))
    B, L, H, P = v.shape
    G, N = q.shape[2:]
    if eps > 0:
        q, k = (t / (t.square().sum(-1, keepdim=True) + eps).sqrt() for t in (q, k))
    q, k = (t.repeat_interleave(H // G, 2) for t in (q, k))
    if inp["dt_bias"] is not None:
        dt = dt + inp["dt_bias"].to(F64)
    a = torch.exp(torch.logaddexp(dt, torch.zeros_like(dt)) * inp["A"].to(F64))
    b = torch.sigmoid(beta)
    S = inp["h0"].to(F64).clone() if inp["h0"] is not None else torch.zeros(B, H, P, N, dtype=F64)
    y = torch.zeros(B, L, H, P, dtype=F64)
    for t in range(L):
        S = a[:, t, :, None, None] * S
        u = b[:, t, :, None] * (v[:, t] - (S * k[:, t, :, None, :]).sum(-1))
        S = S + u[..., None] * k[:, t, :, None, :]
        y[:, t] = scale * (S * q[:, t, :, None, :]).sum(-1)
    return (y[:, 0] if one else y), S


def q4_inputs(M, N, K, group, seed=0, zeros=True, fractional=False):
    g = torch.Generator().manual_seed(seed)
    z = None
    if zeros:
        z = torch.randint(0, 16, (N, K // group), generator=g).to(BF)
        if fractional:
            z = z + 0.5
    return {"x": torch.randn(M, K, generator=g).to(BF), "W": torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8),
            "scales": ((torch.rand(N, K // group, generator=g) - 0.3) * 0.1).to(BF), "zeros": z}


def q4_reference(inp, group):
    """(out, sum of the terms' magnitudes) in 64 bits."""
    W = inp["W"].to(torch.int64)
    N = W.shape[0]
    c = torch.stack([W & 15, W >> 4], -1).reshape(N, -1, group).to(F64)
    z = 8.0 if inp["zeros"] is None else inp["zeros"].to(F64)[..., None]
    w = ((c - z) * inp["scales"].to(F64)[..., None]).reshape(N, -1)
    x = inp["x"].to(F64)
    # the kernel adds the terms of c - 8 and of 8 - z separately
    mag = ((c - 8).abs() + (torch.as_tensor(z) - 8).abs()) * inp["scales"].to(F64).abs()[..., None]
    return x @ w.T, x.abs() @ mag.reshape(N, -1).T
