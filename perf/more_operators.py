"""Operators of a block with a gated delta-rule mixer, as a user calls them, beside their plain forms.

The gated delta rule (delta_fwd, delta_bwd: whole sequences, blocks and single tokens, one direction a call), the norm /
gate / residual step with an 8-bit output and its scales (adaln_fp8), and the projection that reads this output
(proj_fp8: a product in 8-bit floating point with one scale per 128 inputs of a row and per 128 x 128 weights).

`own` False: the operators written out in elementary torch operations, 32-bit arithmetic, one rounding at the end.
`own` True: the library's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
LEAST = 2.0 ** -100  # a block's largest magnitude counts as at least this
GROUP = 128
EPS = 1e-5

# The largest listed sizes; draw() stays below them.
FWD_MOST = 65536 * 32          # batch * tokens * heads, of 128 x 128 states
BWD_MOST = 8192 * 32
NORM_MOST = 8 * 8192 * 2048    # rows * model width
PROJ_MOST = 16384 * 8192 * 4096  # rows * outputs * inputs


def listed():
    return [
        # one new token for each of 16 sequences: every head's state is read and written once
        {"name": "delta_step_token", "op": "delta_fwd", "batch": 16, "seqlen": 1, "hk": 16, "heads": 32, "dk": 128,
         "dv": 128, "dir": "fwd", "state": True},
        # the reverse layer on a ragged batch with narrow keys and shared key heads
        {"name": "delta_fwd_ragged_rev", "op": "delta_fwd", "batch": 3, "seqlen": 1001, "hk": 4, "heads": 8, "dk": 64,
         "dv": 128, "dir": "rev", "state": False},
        # the long sequence through a layer of 4096 channels, its end state kept
        {"name": "delta_fwd_long_64k", "op": "delta_fwd", "batch": 1, "seqlen": 65536, "hk": 32, "heads": 32, "dk": 128,
         "dv": 128, "dir": "fwd", "state": True},
        # gradients of a short sequence through a narrow layer
        {"name": "delta_bwd_short_256", "op": "delta_bwd", "batch": 1, "seqlen": 256, "hk": 2, "heads": 4, "dk": 64,
         "dv": 64, "dir": "fwd", "state": True},
        # gradients of the layer's training sequence, two value heads to a key head
        {"name": "delta_bwd_layer_2k", "op": "delta_bwd", "batch": 2, "seqlen": 2048, "hk": 16, "heads": 32, "dk": 128,
         "dv": 128, "dir": "fwd", "state": False},
        # gradients of a long sequence, reverse layer
        {"name": "delta_bwd_long_8k", "op": "delta_bwd", "batch": 1, "seqlen": 8192, "hk": 32, "heads": 32, "dk": 128,
         "dv": 128, "dir": "rev", "state": False},
        # one active block of 32 tokens ahead of its projection
        {"name": "adaln_fp8_step_32", "op": "adaln_fp8", "batch": 1, "seqlen": 32, "d_model": 2048, "dtype": "bf16",
         "norm": "rms", "post": False, "gate": True, "shared": False},
        # a batch of whole sequences: post-norm of the branch, gate, residual, modulated norm
        {"name": "adaln_fp8_batch_8k", "op": "adaln_fp8", "batch": 8, "seqlen": 8192, "d_model": 2048, "dtype": "bf16",
         "norm": "layer", "post": True, "gate": True, "shared": False},
        # fp32 rows of the paper's width under one weight vector
        {"name": "adaln_fp8_ragged_f32", "op": "adaln_fp8", "batch": 3, "seqlen": 1001, "d_model": 1920,
         "dtype": "f32", "norm": "rms", "post": False, "gate": False, "shared": True},
        # the input projection (gate, step, B, C and x of the paper's layer) of one block of 32 tokens
        {"name": "proj_fp8_step_32", "op": "proj_fp8", "rows": 32, "n": 8056, "k": 1920, "out": "bf16"},
        # the output projection of an odd number of rows, kept in fp32
        {"name": "proj_fp8_ragged", "op": "proj_fp8", "rows": 1001, "n": 1920, "k": 3840, "out": "f32"},
        # a batch of sequences into a wide layer
        {"name": "proj_fp8_batch_16k", "op": "proj_fp8", "rows": 16384, "n": 8192, "k": 4096, "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "adaln_fp8", "proj_fp8", "proj_fp8"])
    if op in ("delta_fwd", "delta_bwd"):
        hk = _log_int(rng, 1, 32)
        heads = hk * rng.choice([1, 1, 2, 3])
        batch = _log_int(rng, 1, 16)
        most = max(1, (FWD_MOST if op == "delta_fwd" else BWD_MOST) // 2 // (batch * heads))
        return {"op": op, "batch": batch, "seqlen": _log_int(rng, 1, min(32768 if op == "delta_fwd" else 8192, most)),
                "hk": hk, "heads": heads, "dk": rng.choice([64, 128]), "dv": rng.choice([64, 128]),
                "dir": rng.choice(["fwd", "fwd", "rev"]), "state": rng.random() < 0.5}
    if op == "adaln_fp8":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        d_model = GROUP * _log_int(rng, 1, 64)
        batch = rng.randint(1, 8)
        seqlen = _log_int(rng, 1, min(16384, NORM_MOST // (2 if dtype == "f32" else 1) // (batch * d_model)))
        return {"op": op, "batch": batch, "seqlen": seqlen, "d_model": d_model, "dtype": dtype,
                "norm": rng.choice(["layer", "rms", "rms"]), "post": rng.random() < 0.6, "gate": rng.random() < 0.7,
                "shared": rng.random() < 0.3}
    n, k = 8 * _log_int(rng, 8, 1024), GROUP * _log_int(rng, 1, 64)
    return {"op": op, "rows": _log_int(rng, 1, min(16384, PROJ_MOST // (n * k))), "n": n, "k": k,
            "out": rng.choice(["bf16", "bf16", "f32"])}


def _e4m3(y, amax):
    """(y over its scale, rounded to 8 bits; the scale) for the largest magnitude of y's block."""
    s = amax.clamp(min=LEAST) / F8_MAX
    return (y / s).to(F8), s


def prepare(case, seed):
    """What a program holds before the call: activations N(0, 1) in the I/O type, keys and queries of unit length, steps
    by the layer's initialisation, fp32 parameters; for the projection 8-bit rows and weights with their scales."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)

    def normal(*shape, scale=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale + mean).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV, dtype=torch.float32)

    def unit(*shape):
        v = normal(*shape)
        return (v / v.square().sum(-1, keepdim=True).sqrt()).to(torch.bfloat16)

    s = {"case": dict(case)}
    if case["op"] in ("delta_fwd", "delta_bwd"):
        nb, L, hk, nh, dk, dv = (case[n] for n in ("batch", "seqlen", "hk", "heads", "dk", "dv"))
        bf = torch.bfloat16
        step = torch.exp(uniform(nh) * (math.log(1e-1) - math.log(1e-3)) + math.log(1e-3))
        s.update(q=unit(nb, L, hk, dk), k=unit(nb, L, hk, dk), v=normal(nb, L, nh, dv, dtype=bf),
                 dt=normal(nb, L, nh, scale=0.5, dtype=bf), A=-1.0 - 15.0 * uniform(nh), b=normal(nb, L, nh, dtype=bf),
                 dt_bias=torch.log(torch.expm1(step)),
                 h_in=normal(nb, nh, dk, dv, scale=0.3) if case["state"] else None, scale=dk ** -0.5)
        if case["op"] == "delta_fwd":
            s["h_out"] = torch.empty(nb, nh, dk, dv, device=DEV) if case["state"] else None
        else:
            s["dout"] = normal(nb, L, nh, dv, dtype=bf)
            s["dh_out"] = normal(nb, nh, dk, dv, scale=0.1) if case["state"] else None
    elif case["op"] == "adaln_fp8":
        nb, L, nd = case["batch"], case["seqlen"], case["d_model"]
        io = DTYPES[case["dtype"]]
        rows = 1 if case["shared"] else nb
        # the residual stream has grown over the blocks before; the branch's scale is its own
        s.update(gamma=normal(rows, nd, scale=0.2, mean=1.0),
                 beta=normal(rows, nd, scale=0.2) if case["norm"] == "layer" else None,
                 gate=normal(rows, nd, scale=0.3, mean=0.5) if case["gate"] else None,
                 post_weight=normal(nd, scale=0.2, mean=1.0) if case["post"] else None,
                 branch=normal(nb, L, nd, scale=1.5, dtype=io), x=normal(nb, L, nd, scale=3.0, mean=0.2, dtype=io))
    else:
        m, n, k = case["rows"], case["n"], case["k"]
        x, w = normal(m, k), normal(n, k, scale=k ** -0.5)
        x = x.view(m, k // GROUP, GROUP)
        x, sx = _e4m3(x, x.abs().amax(-1, keepdim=True))
        blocks = -(-n // GROUP)
        amax = torch.zeros(blocks * GROUP, k, device=DEV)
        amax[:n] = w.abs()
        amax = amax.view(blocks, GROUP, k // GROUP, GROUP).amax((1, 3))
        w, _ = _e4m3(w, _spread(amax, n))
        s.update(x=x.view(1, m, k), x_scales=sx.view(1, m, k // GROUP).contiguous(), w=w,
                 w_scales=(amax.clamp(min=LEAST) / F8_MAX).contiguous())
    return s


def _spread(v, n):
    """One value per 128 x 128 block to one per weight."""
    return v.repeat_interleave(GROUP, 0)[:n].repeat_interleave(GROUP, 1)


# ---- the library's calls ----


def _own_run(s):
    import bidirectional_mamba_selective_amd as bm

    c = s["case"]
    if c["op"] == "proj_fp8":
        return bm.bimamba_proj_fp8(s["x"], s["x_scales"], s["w"], s["w_scales"], out_dtype=DTYPES[c["out"]])
    if c["op"] == "adaln_fp8":
        return bm.bimamba_adaln_fwd_fp8(s["x"], s["gamma"], s["beta"], s["branch"], s["post_weight"], s["gate"],
                                        eps=EPS, flags=bm.FLAG_RMS_NORM if c["norm"] == "rms" else 0)
    flags = bm.FLAG_FWD_ONLY if c["dir"] == "fwd" else bm.FLAG_REV_ONLY
    if c["op"] == "delta_fwd":
        out = bm.bimamba_delta_fwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["b"], s["dt_bias"], h_in=s["h_in"],
                                   h_out=s["h_out"], scale=s["scale"], flags=flags)
        return out, s["h_out"]
    return bm.bimamba_delta_bwd(s["dout"], s["q"], s["k"], s["v"], s["dt"], s["A"], s["b"], s["dt_bias"],
                                h_in=s["h_in"], dh_out=s["dh_out"], scale=s["scale"], flags=flags)


# ---- plain forms ----


def _unit_lower_inverse(n):
    """(I + n)^-1 for strictly lower triangular n [..., C, C], C a power of two: blocks of 1, 2, 4, ... joined two by
    two, [[a, 0], [c, d]]^-1 = [[a', 0], [-d' c a', d']]."""
    C = n.shape[-1]
    t = torch.ones(*n.shape[:-2], C, 1, 1, device=n.device, dtype=n.dtype)
    size = 1
    while size < C:
        m = C // (2 * size)
        cells = n.reshape(*n.shape[:-2], m, 2 * size, m, 2 * size)
        low = torch.diagonal(cells, dim1=-4, dim2=-2)[..., size:, :size, :].movedim(-1, -3)
        a, d = t[..., 0::2, :, :], t[..., 1::2, :, :]
        left = torch.cat([a, -(d @ low @ a)], -2)
        right = torch.cat([torch.zeros_like(a), d], -2)
        t = torch.cat([left, right], -1)
        size *= 2
    return t[..., 0, :, :]


def _plain_delta(q, k, v, dt, A, b, dt_bias, h, scale):
    """Forward direction, fp32: chunks of up to 64 tokens, their states one after the other.  [batch, tokens, heads, .]
    in and out; (out, end state)."""
    L, nh = v.shape[1], v.shape[2]
    C = 1
    while C < min(64, L):
        C *= 2
    pad = -L % C

    def cut(t):  # [B, L, H, ...] -> [B, H, chunks, C, ...]
        t = torch.nn.functional.pad(t, (0, 0) * (t.dim() - 2) + (0, pad)) if pad else t
        return t.movedim(2, 1).unflatten(2, (-1, C))

    x = dt + dt_bias
    delta = x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))
    q, k = (t.repeat_interleave(nh // t.shape[2], 2) for t in (q, k))
    q, k, v, g, beta = cut(q), cut(k), cut(v), cut(delta * A), cut(1 / (1 + torch.exp(-b)))
    if pad:
        real = (torch.arange(L + pad, device=v.device) < L).view(-1, C)
        g, beta = torch.where(real, g, 0.0), torch.where(real, beta, 0.0)
    gam = g.double().cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=v.device).tril()
    decay = torch.exp(torch.where(low, gam[..., :, None] - gam[..., None, :], -math.inf).float())
    kt = k.transpose(-1, -2).contiguous()
    t = _unit_lower_inverse((k @ kt * decay * beta[..., None]).tril(-1)) * beta[..., None, :]
    attn = q @ kt * decay * scale
    eg = torch.exp(gam).float()[..., None]
    last = gam[..., -1:]
    keep = torch.exp(last - gam).float()[..., None]
    last = torch.exp(last).float()[..., None]
    tv, tk, qs, kd = t @ v, t @ (k * eg), q * eg * scale, (k * keep).transpose(-1, -2).contiguous()
    del t, decay
    out = []
    for n in range(v.shape[2]):
        u = tv[:, :, n] - tk[:, :, n] @ h
        out.append(qs[:, :, n] @ h + attn[:, :, n] @ u)
        h = last[:, :, n] * h + kd[:, :, n] @ u
    return torch.cat(out, 2)[:, :, :L].movedim(1, 2), h


_SEQ = ("q", "k", "v", "dt", "b")


def _delta_inputs(s, wide):
    """The call's inputs in 32 or 64 bits, tokens in the order in which the direction meets them."""
    rev = s["case"]["dir"] == "rev"
    t = {n: s[n].to(wide).flip(1) if rev else s[n].to(wide) for n in _SEQ}
    t.update(A=s["A"].to(wide), dt_bias=s["dt_bias"].to(wide))
    nb, nh = s["v"].shape[0], s["v"].shape[2]
    t["h"] = torch.zeros(nb, nh, s["q"].shape[3], s["v"].shape[3], device=DEV, dtype=wide) if s["h_in"] is None \
        else s["h_in"].to(wide)
    return t


_ARGS = ("q", "k", "v", "dt", "A", "b", "dt_bias", "h")


def _plain_delta_fwd(s):
    t = _delta_inputs(s, torch.float32)
    out, h = _plain_delta(*[t[n] for n in _ARGS], s["scale"])
    out = out.flip(1) if s["case"]["dir"] == "rev" else out
    return out.to(torch.bfloat16).contiguous(), (h if s["h_out"] is not None else None)


def _delta_grads(s, got):
    """Gradients by input name, in the inputs' types and token order."""
    rev = s["case"]["dir"] == "rev"
    g = {n: (v.flip(1) if rev else v).to(s[n].dtype).contiguous() if n in _SEQ else v for n, v in got.items()}
    h = g.pop("h")
    g["h_in"] = None if s["h_in"] is None else h
    return g


def _plain_delta_bwd(s):
    t = {n: v.requires_grad_() for n, v in _delta_inputs(s, torch.float32).items()}
    out, h = _plain_delta(*[t[n] for n in _ARGS], s["scale"])
    dout = s["dout"].float()
    dout = dout.flip(1) if s["case"]["dir"] == "rev" else dout
    dh = torch.zeros_like(h) if s["dh_out"] is None else s["dh_out"]
    return _delta_grads(s, dict(zip(_ARGS, torch.autograd.grad([out, h], [t[n] for n in _ARGS], [dout, dh]))))


def _rows(p):
    return None if p is None else p[:, None, :]


def _plain_adaln_fp8(s):
    c = s["case"]
    io = s["x"].dtype
    gamma, beta, gate = _rows(s["gamma"]), _rows(s["beta"]), _rows(s["gate"])
    m = s["branch"].float()
    if c["post"]:
        m = m * torch.rsqrt((m * m).mean(-1, keepdim=True) + EPS) * s["post_weight"]
    h = s["x"].float() + (m if gate is None else gate * m)
    hc = h - h.mean(-1, keepdim=True) if c["norm"] == "layer" else h
    out = hc * torch.rsqrt((hc * hc).mean(-1, keepdim=True) + EPS) * gamma
    out = (out if beta is None else out + beta).unflatten(-1, (-1, GROUP))
    out, scales = _e4m3(out, out.abs().amax(-1, keepdim=True))
    return h.to(io), out.flatten(-2), scales.squeeze(-1)


def _plain_proj_fp8(s):
    x = s["x"][0].float() * s["x_scales"][0].repeat_interleave(GROUP, 1)
    w = s["w"].float() * _spread(s["w_scales"], s["w"].shape[0])
    return (x @ w.t()).to(DTYPES[s["case"]["out"]])[None]


_PLAIN = {"delta_fwd": _plain_delta_fwd, "delta_bwd": _plain_delta_bwd, "adaln_fp8": _plain_adaln_fp8,
          "proj_fp8": _plain_proj_fp8}


def run(state):
    return _own_run(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ----


def work(case):
    if case["op"] in ("delta_fwd", "delta_bwd"):
        nb, L, hk, nh, dk, dv = (case[n] for n in ("batch", "seqlen", "hk", "heads", "dk", "dv"))
        seq = nb * L * 2 * (2 * hk * dk + nh * dv + 2 * nh)  # q, k, v, dt, b
        io = nb * L * 2 * nh * dv                            # out or its gradient
        st = nb * nh * dk * dv * 4 if case["state"] else 0
        if case["op"] == "delta_fwd":
            # per token, head and state: decay, the read at k, the update, the read at q
            return {"bytes": seq + io + 2 * st + 8 * nh, "flops": nb * L * nh * dk * dv * 7}
        # the states again; the adjoint's decay, its read at k, its two updates; the state read for dq, the adjoint and
        # the state for dk, the decay's gradient
        return {"bytes": 2 * seq + io + 3 * st + 16 * nh, "flops": nb * L * nh * dk * dv * 20}
    if case["op"] == "adaln_fp8":
        n = case["batch"] * case["seqlen"] * case["d_model"]
        rows = 1 if case["shared"] else case["batch"]
        vec = 4 * case["d_model"] * (rows * (1 + (case["norm"] == "layer") + case["gate"]) + case["post"])
        return {"bytes": n * (3 * (4 if case["dtype"] == "f32" else 2) + 1) + n // GROUP * 4 + vec, "flops": n * 15}
    m, n, k = case["rows"], case["n"], case["k"]
    scales = 4 * (k // GROUP) * (m + -(-n // GROUP))
    return {"bytes": m * k + n * k + scales + m * n * (4 if case["out"] == "f32" else 2), "flops": 2 * m * n * k}


# ---- the definitions in 64 bits ----


def _exact_delta(t, scale, heads):
    """Token after token, for the value heads of the slice `heads`."""
    nh = t["v"].shape[2]
    which = torch.arange(nh, device=DEV)[heads]
    share = nh // t["k"].shape[2]
    q, k = (t[n].index_select(2, which // share) for n in ("q", "k"))
    v, dt, b = (t[n][:, :, heads] for n in ("v", "dt", "b"))
    g = torch.logaddexp(dt + t["dt_bias"][heads], torch.zeros((), dtype=torch.float64, device=DEV)) * t["A"][heads]
    a = torch.exp(g)[..., None, None].unbind(1)
    beta = torch.sigmoid(b)[..., None, None].unbind(1)
    q, k, v = (x.unsqueeze(-2).unbind(1) for x in (q, k, v))
    h, out = t["h"][:, heads], []
    for i in range(len(q)):
        h = a[i] * h
        h = h + k[i].transpose(-1, -2) * (beta[i] * (v[i] - torch.matmul(k[i], h)))
        out.append(torch.matmul(q[i], h))
    return scale * torch.cat(out, -2).movedim(1, 2), h


def _exact_delta_fwd(s):
    t = _delta_inputs(s, torch.float64)
    out, h = _exact_delta(t, s["scale"], slice(None))
    return (out.flip(1) if s["case"]["dir"] == "rev" else out), (h if s["h_out"] is not None else None)


def _exact_delta_bwd(s):
    t = {n: v.requires_grad_() for n, v in _delta_inputs(s, torch.float64).items()}
    rev = s["case"]["dir"] == "rev"
    c = s["case"]
    # the states of every token are kept for differentiation: a few heads at a time
    at_once = max(1, int(6e9 // (8 * c["batch"] * c["seqlen"] * c["dk"] * c["dv"])))
    total = dict.fromkeys(_ARGS, 0.0)
    for first in range(0, c["heads"], at_once):
        part = slice(first, min(c["heads"], first + at_once))
        out, h = _exact_delta(t, s["scale"], part)
        dout = s["dout"][:, :, part].double()
        dh = torch.zeros_like(h) if s["dh_out"] is None else s["dh_out"][:, part].double()
        got = torch.autograd.grad([out, h], [t[n] for n in _ARGS], [dout.flip(1) if rev else dout, dh])
        total = {n: total[n] + x for n, x in zip(_ARGS, got)}
    g = {n: x.flip(1) if rev and n in _SEQ else x for n, x in total.items()}
    h = g.pop("h")
    g["h_in"] = None if s["h_in"] is None else h
    return g


def _exact_adaln_fp8(s):
    c = s["case"]
    p = {n: None if s[n] is None else s[n].double() for n in ("x", "branch", "gamma", "beta", "gate", "post_weight")}
    add = p["branch"]
    if p["post_weight"] is not None:
        add = add / torch.sqrt(add.pow(2).mean(2, True) + EPS) * p["post_weight"]
    h = p["x"] + (add if p["gate"] is None else add * p["gate"].unsqueeze(1))
    y = h if c["norm"] == "rms" else h - h.mean(2, True)
    y = y / torch.sqrt(y.pow(2).mean(2, True) + EPS) * p["gamma"].unsqueeze(1)
    y = y if p["beta"] is None else y + p["beta"].unsqueeze(1)
    groups = y.reshape(*y.shape[:2], -1, GROUP)
    scales = torch.maximum(groups.abs().amax(3), torch.tensor(LEAST, dtype=y.dtype, device=DEV)) / F8_MAX
    z = (groups / scales.unsqueeze(3)).reshape(y.shape)
    # e4m3: three bits after the leading one, exponents from -6, below that steps of 2^-9
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return h, torch.round(z / step) * step, scales


def _exact_proj_fp8(s):
    m, k = s["x"].shape[1:]
    n = s["w"].shape[0]
    total = torch.zeros(m, n, dtype=torch.float64, device=DEV)
    col = torch.arange(n, device=DEV) // GROUP
    for j in range(k // GROUP):
        part = slice(j * GROUP, (j + 1) * GROUP)
        # the right factor as a matrix of its own: [128, n]
        dots = s["x"][0, :, part].double() @ s["w"][:, part].double().t().contiguous()
        total += dots * s["x_scales"][0, :, j, None].double() * s["w_scales"][col, j].double()
    return total[None]


def exact(case, seed):
    s = prepare(case, seed)
    return {"delta_fwd": _exact_delta_fwd, "delta_bwd": _exact_delta_bwd, "adaln_fp8": _exact_adaln_fp8,
            "proj_fp8": _exact_proj_fp8}[case["op"]](s)
