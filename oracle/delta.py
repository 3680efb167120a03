"""Gated delta rule in fp64, token by token: the definition, its gradients, and bounds on what fp32 arithmetic may be off.

Per head, in the direction's order (H: the state, dk x dv):
    a = exp(softplus(dt + dt_bias) A),  beta = sigmoid(b)
    H = a H_before,  e = v - H^T k,  H_t = H + beta k e^T,  out = scale H_t^T q
"""
from __future__ import annotations

import numpy as np

_SEQ = ("q", "k", "v", "dt", "b")


def _sigmoid(x):
    x = np.asarray(x, np.float64)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def _prepare(inp, rev):
    """fp64 inputs in the direction's order, keys and queries repeated for the heads that share them, gates."""
    p = {n: np.asarray(inp[n], np.float64) for n in _SEQ}
    if rev:
        p = {n: x[:, ::-1] for n, x in p.items()}
    nh, share = p["v"].shape[2], p["v"].shape[2] // p["k"].shape[2]
    p["q"], p["k"] = np.repeat(p["q"], share, 2), np.repeat(p["k"], share, 2)
    A = np.asarray(inp["A"], np.float64)
    x = p["dt"] + (0.0 if inp.get("dt_bias") is None else np.asarray(inp["dt_bias"], np.float64))
    delta = np.logaddexp(x, 0.0)
    p.update(A=A, x=x, delta=delta, a=np.exp(delta * A), beta=_sigmoid(p["b"]), share=share)
    nb, L = p["v"].shape[:2]
    h = inp.get("h_in")
    p["h"] = np.zeros((nb, nh, p["k"].shape[3], p["v"].shape[3])) if h is None else np.asarray(h, np.float64)
    return p


def delta_fwd(inp, scale=None, rev=False, keep=False):
    """(out, h_out) for inputs q, k, v, dt, A, b and optionally dt_bias, h_in; keep: also what the backward pass needs."""
    p = _prepare(inp, rev)
    scale = p["q"].shape[3] ** -0.5 if scale is None else scale
    H, out, kept = p["h"], np.zeros_like(p["v"]), []
    for t in range(out.shape[1]):
        k, q = p["k"][:, t], p["q"][:, t]
        Hd = p["a"][:, t, :, None, None] * H
        e = p["v"][:, t] - np.einsum("bhk,bhkv->bhv", k, Hd)
        H = Hd + k[..., None] * (p["beta"][:, t, :, None] * e)[:, :, None, :]
        out[:, t] = scale * np.einsum("bhk,bhkv->bhv", q, H)
        if keep:
            kept.append((Hd, e, H))
    out = out[:, ::-1] if rev else out
    return (out, H, p, kept, scale) if keep else (out, H)


def _shared(g, share):
    return g.reshape(*g.shape[:2], -1, share, g.shape[3]).sum(3)


def delta_bwd(dout, inp, dh_out=None, scale=None, rev=False):
    """Gradients of delta_fwd's inputs, by name."""
    _, H, p, kept, scale = delta_fwd(inp, scale, rev, keep=True)
    do = np.asarray(dout, np.float64)
    do = do[:, ::-1] if rev else do
    G = np.zeros_like(H) if dh_out is None else np.asarray(dh_out, np.float64).copy()
    g = {n: np.zeros_like(p[n]) for n in _SEQ}
    dg = np.zeros_like(p["dt"])
    for t in range(do.shape[1] - 1, -1, -1):
        Hd, e, H = kept[t]
        k, q, o, beta = p["k"][:, t], p["q"][:, t], do[:, t], p["beta"][:, t, :, None]
        G = G + scale * q[..., None] * o[:, :, None, :]
        g["q"][:, t] = scale * np.einsum("bhkv,bhv->bhk", H, o)
        du = np.einsum("bhk,bhkv->bhv", k, G)
        g["v"][:, t] = beta * du
        g["k"][:, t] = np.einsum("bhkv,bhv->bhk", G, beta * e) - np.einsum("bhkv,bhv->bhk", Hd, beta * du)
        g["b"][:, t] = (du * e).sum(-1) * p["beta"][:, t] * _sigmoid(-p["b"][:, t])
        G = G - k[..., None] * (beta * du)[:, :, None, :]
        dg[:, t] = (G * Hd).sum((2, 3))
        G = p["a"][:, t, :, None, None] * G
    ddt = dg * p["A"] * _sigmoid(p["x"])
    g["dt"] = ddt
    g["q"], g["k"] = _shared(g["q"], p["share"]), _shared(g["k"], p["share"])
    if rev:
        g = {n: x[:, ::-1] for n, x in g.items()}
    g.update(A=(dg * p["delta"]).sum((0, 1)), dt_bias=ddt.sum((0, 1)), h_in=G)
    return g


def _norm(x, ax=-1):
    return np.sqrt((x * x).sum(ax))


def delta_bounds(inp, dout=None, dh_out=None, scale=None, rev=False, eps=2.0 ** -16, eps16=2.0 ** -15):
    """How far results formed in fp32 may be off, as 2-norms per (token, head), before the outputs' own rounding.

    The map from one state to the next, a (I - beta k k^T), does not enlarge a vector where |k| <= 1 and beta <= 1, so
    errors of the state add up and do not grow.  With every sum and product off by at most eps relative to the norms of
    what goes into it (2^-16: 256 roundings of 2^-24, for sums of 64 and 128 terms, the triangular inverse, whose entries
    are at most 1, and its application),
        E_t = a E_(t-1) + eps (a W_(t-1) (1 + beta |k|^2) + beta |k| |v|)      bounds the state's error,
        F_t = a (F_(t+1) + eps (Y_t (1 + beta |k|^2) + scale |q| |dout|))     that of its gradient G,
    W and Y the norms of the state and of G where a run of 64 tokens begins plus those of the terms that its tokens add
    (a run is worked out as a whole).  eps16 (2^-15) is what bf16 pairs in place
    of fp32 operands leave, on both sides of a product, in results that are rounded to bf16.  The results' bounds follow
    by the product rule."""
    _, H, p, kept, scale = delta_fwd(inp, scale, rev, keep=True)
    k, q, v, a, beta = _norm(p["k"]), _norm(p["q"]), _norm(p["v"]), p["a"], p["beta"]
    E, W = np.zeros_like(v[:, 0]), _norm(p["h"], (2, 3))
    Es, Ws, Ed, Wd, en, ee = [], [], [], [], [], []
    L = v.shape[1]
    begins = [t == 0 or (L - t) % 64 == 0 if rev else t % 64 == 0 for t in range(L)]
    for t in range(L):
        if begins[t] and t:
            W = _norm(kept[t - 1][2], (2, 3))
        Ed.append(a[:, t] * E)
        Wd.append(a[:, t] * W)
        en.append(_norm(kept[t][1]))
        ee.append(k[:, t] * Ed[t] + eps * (v[:, t] + k[:, t] * Wd[t]))
        E = Ed[t] + eps * (Wd[t] * (1 + beta[:, t] * k[:, t] ** 2) + beta[:, t] * k[:, t] * v[:, t])
        W = Wd[t] + beta[:, t] * k[:, t] * en[t]
        Es.append(E)
        Ws.append(W)
    flip = (lambda x: x[:, ::-1]) if rev else (lambda x: x)
    r = {"out": flip(scale * q * (np.stack(Es, 1) + eps16 * np.stack(Ws, 1))), "h_out": E}
    if dout is None:
        return r
    do = np.asarray(dout, np.float64)
    do = do[:, ::-1] if rev else do
    o = _norm(do)
    G = np.zeros_like(H) if dh_out is None else np.asarray(dh_out, np.float64).copy()
    F, Y = np.zeros_like(E), _norm(G, (2, 3))
    g = {n: np.zeros_like(v) for n in _SEQ}
    sA = sb = 0.0
    for t in range(L - 1, -1, -1):
        if t + 1 < L and begins[t + 1]:
            Y = _norm(G, (2, 3))
        be, kt, on = beta[:, t], k[:, t], scale * q[:, t] * o[:, t]
        G = G + scale * p["q"][:, t][..., None] * do[:, t][:, :, None, :]
        F, Y = F + eps * on, Y + on
        du = np.einsum("bhk,bhkv->bhv", p["k"][:, t], G)
        d, ed = _norm(du), kt * (F + eps * Y)
        g["q"][:, t] = scale * o[:, t] * (Es[t] + eps16 * Ws[t])
        g["v"][:, t] = be * ed
        g["k"][:, t] = be * ((F + eps16 * Y) * en[t] + Y * ee[t] + (Ed[t] + eps16 * Wd[t]) * d + Wd[t] * ed)
        g["b"][:, t] = be * _sigmoid(-p["b"][:, t]) * (d * ee[t] + ed * en[t] + eps * d * en[t])
        G = G - p["k"][:, t][..., None] * (be[..., None] * du)[:, :, None, :]
        F, Y = F + eps * Y * (1 + be * kt * kt) + be * kt * ed, Y + be * kt * d
        dg = F * Wd[t] + Y * Ed[t] + eps * Y * Wd[t]
        g["dt"][:, t] = dg * np.abs(p["A"]) * _sigmoid(p["x"][:, t])
        sA = sA + (dg * p["delta"][:, t]).sum(0)
        sb = sb + g["dt"][:, t].sum(0)
        G = a[:, t, :, None, None] * G
        F, Y = a[:, t] * F, a[:, t] * Y
    for n in ("q", "k"):
        g[n] = g[n].reshape(*g[n].shape[:2], -1, p["share"]).sum(3)
    r.update({n: flip(x) for n, x in g.items()}, A=sA, dt_bias=sb, h_in=F)
    return r
