"""Workloads of the gated delta rule (prefill and one-token step) and of the
projection with 4-bit weights, in their plain form and through the library.

Per sequence and value head h (key head g = h / (H / G)), state S [P, N]:

    a_t = exp(softplus(dt_t + dt_bias) A)        b_t = sigmoid(beta_t)
    q^, k^ = q_t, k_t over sqrt(sum of squares + norm_eps)   (as they are when norm_eps is 0)
    S_t = a_t S_{t-1} + b_t (v_t - a_t S_{t-1} k^_t) k^_t^T
    y_t = scale S_t q^_t

and, for a weight of 4-bit numbers c with a scale s and a zero point z per
`group` inputs of a row,

    out[m, n] = sum_k x[m, k] s[n, k / group] (c[n, k] - z[n, k / group])
"""

import math

import torch

own = False

_EPS = 1e-6
_CHUNK = 64
_BF16 = torch.bfloat16


# ---------------------------------------------------------------- cases
def _prefill(name, batch, seqlen, groups, heads, headdim, d_state, act="bf16", carried=False, packed=True, norm=True):
    c = {"op": "prefill", "batch": batch, "seqlen": seqlen, "groups": groups, "heads": heads, "headdim": headdim,
         "d_state": d_state, "act": act, "carried": carried, "packed": packed, "norm": norm}
    return dict(c, name=name) if name else c


def _step(name, batch, groups, heads, headdim, d_state, act="bf16", norm=True):
    c = {"op": "step", "batch": batch, "groups": groups, "heads": heads, "headdim": headdim, "d_state": d_state,
         "act": act, "norm": norm}
    return dict(c, name=name) if name else c


def _q4(name, rows, outputs, inputs, group, zeros=False, out="bf16"):
    c = {"op": "q4", "rows": rows, "outputs": outputs, "inputs": inputs, "group": group, "zeros": zeros, "out": out}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short prompt, or a few speculated tokens continuing a sequence: latency
        _prefill("prefill 1x29 8 heads", 1, 29, 4, 8, 64, 64, carried=True),
        # the layer whose value width is the 8192 channels of the other forms' prefill
        _prefill("prefill 1x4096 64 heads", 1, 4096, 32, 64, 128, 128),
        # several prompts of an odd length, continued from carried states
        _prefill("prefill 4x1001 16 heads", 4, 1001, 16, 16, 128, 64, carried=True, packed=False, norm=False),
        # a long document on one of several GPUs that share the heads: few heads, many tokens
        _prefill("prefill 1x16384 8 heads", 1, 16384, 4, 8, 256, 128),
        # fp32 activations (a reference run, a small model)
        _prefill("prefill 2x200 f32", 2, 200, 8, 16, 128, 64, act="f32"),
        # one sequence being decoded: latency
        _step("step 1x32 heads", 1, 16, 32, 128, 128),
        # a full serving batch: the state's traffic
        _step("step 128x64 heads", 128, 32, 64, 128, 128),
        # an odd batch of fp32 activations, a head width that is no power of two
        _step("step 17x24 heads f32", 17, 8, 24, 192, 64, act="f32"),
        # a decoded token's input projection: hidden 4096 to x and z of 8192 channels
        _q4("q4 1x16384x4096", 1, 16384, 4096, 128),
        # its low-rank step and B, C projection: few outputs, many inputs
        _q4("q4 1x288x8192", 1, 288, 8192, 64, zeros=True, out="f32"),
        # the output projection of a batch of 16 sequences
        _q4("q4 16x4096x8192", 16, 4096, 8192, 128, zeros=True),
        # odd sizes
        _q4("q4 5x1003x1056", 5, 1003, 1056, 32, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "q4"])
    if op == "q4":
        group = rng.choice([32, 64, 128])
        inputs = group * _log_int(rng, 1, 16384 // group)
        return _q4(None, _log_int(rng, 1, 64), _log_int(rng, 8, 16384), inputs, group, rng.random() < 0.5,
                   rng.choice(["bf16", "f32"]))
    groups = rng.choice([1, 2, 3, 4, 8, 16])
    heads = groups * rng.choice([1, 2, 4])
    headdim, d_state = rng.choice([64, 128, 192, 256]), rng.choice([64, 128])
    act = "f32" if rng.random() < 0.2 else "bf16"
    if op == "step":
        return _step(None, _log_int(rng, 1, max(1, 128 * 64 * 128 // (heads * headdim))), groups, heads, headdim, d_state, act,
                     rng.random() < 0.7)
    # no more state rows x tokens than the largest listed prefill
    batch = _log_int(rng, 1, 8)
    most = 4096 * 64 * 128 // (batch * heads * headdim)
    seqlen = _log_int(rng, 1, max(1, min(16384 if act == "bf16" else 512, most)))
    return _prefill(None, batch, seqlen, groups, heads, headdim, d_state, act, rng.random() < 0.5, rng.random() < 0.5,
                    rng.random() < 0.7)


# ---------------------------------------------------------------- inputs
def _act(t, act):
    return t.to(_BF16) if act == "bf16" else t


def _unit(t):
    return t * torch.rsqrt((t * t).sum(-1, keepdim=True) + _EPS)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, device="cuda", generator=g) * (hi - lo) + lo

    if case["op"] == "q4":
        M, N, K, G = case["rows"], case["outputs"], case["inputs"], case["group"]
        out = {"x": normal(M, K).to(_BF16), "group": G, "out": torch.float32 if case["out"] == "f32" else _BF16,
               "W": torch.randint(0, 256, (N, K // 2), device="cuda", generator=g, dtype=torch.uint8),
               "scales": (uniform(0.5, 1.5, N, K // G) * (0.25 / math.sqrt(K))).to(_BF16), "zeros": None}
        if case["zeros"]:
            out["zeros"] = torch.randint(0, 16, (N, K // G), device="cuda", generator=g).to(_BF16)
        return out

    B, G, H, P, N, act = (case[k] for k in ("batch", "groups", "heads", "headdim", "d_state", "act"))
    lead = (B, case["seqlen"]) if case["op"] == "prefill" else (B,)
    # q, k and v as a convolution with SiLU leaves them; unit q and k where the call does not normalise
    silu = torch.nn.functional.silu
    q, k, v = silu(normal(*lead, G, N)), silu(normal(*lead, G, N)), silu(normal(*lead, H, P))
    if not case["norm"]:
        q, k = _unit(q), _unit(k)
    q, k, v = _act(q, act), _act(k, act), _act(v, act)
    if case.get("packed", True):    # one tensor [q | k | v], as the convolution writes it
        qkv = torch.cat([t.flatten(-2) for t in (q, k, v)], -1)
        q, k, v = (t.unflatten(-1, s) for t, s in zip(qkv.split([G * N, G * N, H * P], -1), ((G, N), (G, N), (H, P))))
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), H))
    return {"q": q, "k": k, "v": v, "dt": _act(normal(*lead, H), act), "beta": _act(normal(*lead, H), act),
            "dt_bias": step + torch.log(-torch.expm1(-step)), "A": -uniform(1.0, 16.0, H),
            "h0": normal(B, H, P, N) * 0.1 if case["op"] == "step" or case["carried"] else None,
            "eps": _EPS if case["norm"] else 0.0, "scale": N ** -0.5}


# ---------------------------------------------------------------- one pass
def run(state):
    if "W" in state:
        return _own_q4(state) if own else _plain_q4(state)
    if state["q"].dim() == 3:
        return _own_step(state) if own else _plain_step(state)
    return _own_prefill(state) if own else _plain_prefill(state)


def _own_prefill(s):
    import mamba_selective_scan_core_b200 as mm

    B, L, H, P = s["v"].shape
    G, N = s["q"].shape[2:]
    if "workspace" not in s:    # scratch that a program keeps from call to call
        s["workspace"] = torch.empty(mm.gdr_workspace_size(B, L, H, P, N, G, act=mm.MM_F32 if s["v"].dtype == torch.float32 else mm.MM_BF16),
                                     dtype=torch.uint8, device="cuda")
    return mm.gdr_fwd(s["q"], s["k"], s["v"], s["dt"], s["beta"], s["dt_bias"], s["A"], s["h0"], scale=s["scale"],
                      norm_eps=s["eps"], workspace=s["workspace"])


def _own_step(s):
    import mamba_selective_scan_core_b200 as mm

    y = mm.gdr_state_update(s["q"], s["k"], s["v"], s["dt"], s["beta"], s["dt_bias"], s["A"], s["h0"],
                            scale=s["scale"], norm_eps=s["eps"])
    return y, s["h0"]


def _own_q4(s):
    import mamba_selective_scan_core_b200 as mm

    return mm.proj_q4(s["x"], s["W"], s["scales"], s["zeros"], group=s["group"], out_dtype=s["out"])


def _gates(s):
    v = s["dt"].float() + s["dt_bias"]
    step = v.clamp_min(0) + torch.log1p(torch.exp(-v.abs()))
    return step * s["A"], 1 / (1 + torch.exp(-s["beta"].float()))


def _keys(s):
    H, G = s["v"].shape[-2], s["q"].shape[-2]
    q, k = s["q"].float(), s["k"].float()
    if s["eps"] > 0:
        q, k = (t * torch.rsqrt((t * t).sum(-1, keepdim=True) + s["eps"]) for t in (q, k))
    return q.repeat_interleave(H // G, -2) * s["scale"], k.repeat_interleave(H // G, -2)


def _plain_step(s):
    log_a, b = _gates(s)
    q, k = _keys(s)
    S = s["h0"].mul_(torch.exp(log_a)[..., None, None])
    S += (b[..., None] * (s["v"].float() - (S * k[..., None, :]).sum(-1)))[..., None] * k[..., None, :]
    return (S * q[..., None, :]).sum(-1).to(s["v"].dtype), S


def _plain_prefill(s):
    # chunks of 64 tokens: the tokens of a chunk at once, the chunks in order
    B, L, H, P = s["v"].shape
    C = min(_CHUNK, L)
    n = -(-L // C)

    def chunks(t):      # [B, L, H, ...] -> [B, H, n, C, ...], zeros behind the last token
        t = torch.nn.functional.pad(t, [0, 0] * (t.dim() - 2) + [0, n * C - L])
        return t.unflatten(1, (n, C)).movedim(3, 1)

    log_a, b = (chunks(t) for t in _gates(s))
    q, k = (chunks(t) for t in _keys(s))
    v = chunks(s["v"].float())
    cum = log_a.double().cumsum(-1)     # differences of long sums
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).tril()).float()
    into, out_of = torch.exp(cum).float(), torch.exp(cum[..., -1:] - cum).float()
    rank = torch.arange(C, device="cuda")
    T = -(b[..., None] * (k @ k.mT) * decay).where(rank[:, None] > rank, 0)
    for i in range(1, C):               # (I + the strict lower part)^-1 by substitution
        T[..., i, :i] += (T[..., i, :i, None] * T[..., :i, :i]).sum(-2)
    T = (T + (rank[:, None] == rank)) * b[..., None, :]
    U, W = T @ v, (T * into[..., None, :]) @ k
    M = ((q @ k.mT) * decay).where(rank[:, None] >= rank, 0)
    q, k = q * into[..., None], k * out_of[..., None]
    S = s["h0"].mT.clone() if s["h0"] is not None else v.new_zeros(B, H, k.shape[-1], P)
    y = torch.empty_like(U)
    for c in range(n):
        new = U[:, :, c] - W[:, :, c] @ S
        y[:, :, c] = q[:, :, c] @ S + M[:, :, c] @ new
        S = into[:, :, c, -1, None, None] * S + k[:, :, c].mT @ new
    y = y.movedim(1, 3).flatten(1, 2)[:, :L]
    return y.to(s["v"].dtype).contiguous(), S.mT.contiguous()


def _plain_q4(s):
    c = torch.stack([s["W"] & 15, s["W"] >> 4], -1).flatten(-2).float()     # the low four bits come first
    z = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(s["group"], -1)
    w = (c - z) * s["scales"].float().repeat_interleave(s["group"], -1)
    return (s["x"].float() @ w.T).to(s["out"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "q4":
        M, N, K, G = case["rows"], case["outputs"], case["inputs"], case["group"]
        bytes_ = N * K // 2 + N * (K // G) * (4 if case["zeros"] else 2) + M * K * 2 + M * N * (4 if case["out"] == "f32" else 2)
        return {"bytes": bytes_, "flops": 2 * M * N * K}
    B, G, H, P, N = (case[k] for k in ("batch", "groups", "heads", "headdim", "d_state"))
    es = 4 if case["act"] == "f32" else 2
    tokens = B * case.get("seqlen", 1)
    states = (2 if case["op"] == "step" or case["carried"] else 1) * B * H * P * N * 4
    # a token: decay, S k, the rank-one update, S q (2 P N each but the decay)
    return {"bytes": tokens * (2 * G * N + 2 * H * P + 2 * H) * es + states + 8 * H, "flops": tokens * H * P * N * 7}


# ---------------------------------------------------------------- in 64 bits, from the definition
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "q4":
        M, N, K, G = case["rows"], case["outputs"], case["inputs"], case["group"]
        w = torch.empty(N, K, dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = (s["W"] % 16).double(), (s["W"] // 16).double()
        w = w.view(N, K // G, G)
        w = (w - (8 if s["zeros"] is None else s["zeros"].double()[..., None])) * s["scales"].double()[..., None]
        return s["x"].double() @ w.view(N, K).T
    B, G, H, P, N = (case[k] for k in ("batch", "groups", "heads", "headdim", "d_state"))
    L = case.get("seqlen", 1)
    q, k, v = s["q"].double().reshape(B, L, G, N), s["k"].double().reshape(B, L, G, N), s["v"].double().reshape(B, L, H, P)
    if s["eps"] > 0:
        q, k = q / (q.square().sum(-1, keepdim=True) + s["eps"]).sqrt(), k / (k.square().sum(-1, keepdim=True) + s["eps"]).sqrt()
    dt = torch.nn.functional.softplus(s["dt"].double().reshape(B, L, H) + s["dt_bias"].double(), threshold=60.0)
    a, b = torch.exp(dt * s["A"].double()), torch.sigmoid(s["beta"].double().reshape(B, L, H))
    S = s["h0"].double() if s["h0"] is not None else torch.zeros(B, H, P, N, dtype=torch.float64, device="cuda")
    S = S.view(B, G, H // G, P, N).clone()
    y = torch.empty(B, L, G, H // G, P, dtype=torch.float64, device="cuda")
    v, a, b = (t.unflatten(2, (G, H // G)) for t in (v, a, b))
    for t in range(L):
        S *= a[:, t, ..., None, None]
        miss = v[:, t] - torch.einsum("bghpn,bgn->bghp", S, k[:, t])
        S += (b[:, t, ..., None] * miss)[..., None] * k[:, t, :, None, None, :]
        y[:, t] = torch.einsum("bghpn,bgn->bghp", S, q[:, t])
    y = (y * s["scale"]).reshape(s["v"].shape)
    return y, S.reshape(B, H, P, N)
