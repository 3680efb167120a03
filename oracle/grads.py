"""Gradients of the mixer's operators in fp64: the selective scan's, the short convolution's, and the
norm / gate / residual step between two blocks (with its forward pass).

Plain numpy.  The scan's gradients walk the tokens one by one, every state of every token kept; nothing is
shared with the HIP path.  Sections cite "DiffuMamba: High-Throughput Diffusion LMs with Mamba Backbone"
(arXiv v4): eq. (4)-(6) for the scan, Appendix C Table 12 for the convolution, Appendix A.1 eq. (10)-(12) for
the modulated norm and the residual around the mixer.
"""
from __future__ import annotations

import numpy as np

from .scan import _f64, softplus


def sigmoid(v):
    v = _f64(v)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0.0, 1.0 / (1.0 + e), e / (1.0 + e))


def silu_grad(v):
    s = sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


def _direction_grads(delta, u, A, B, C, dy, reverse):
    """One direction's scan h, its adjoint q and w = d(loss)/d(log abar), walking tokens in the scan's order.

    h_t = abar_t h_{t-1} + u_t B_t; q_t = C_t dy_t + abar_{t+1} q_{t+1}; w_t = abar_t q_t h_{t-1}."""
    nb, L, nd = u.shape
    ns = A.shape[1]
    order = range(L - 1, -1, -1) if reverse else range(L)
    h = np.zeros((nb, L, nd, ns))
    before = np.zeros((nb, L, nd, ns))
    state = np.zeros((nb, nd, ns))
    for t in order:
        before[:, t] = state
        state = np.exp(delta[:, t, :, None] * A) * state + u[:, t, :, None] * B[:, t, None, :]
        h[:, t] = state
    q = np.zeros((nb, L, nd, ns))
    w = np.zeros((nb, L, nd, ns))
    back = np.zeros((nb, nd, ns))  # abar q of the token after this one in the scan's order
    for t in reversed(order):
        q[:, t] = C[:, t, None, :] * dy[:, t, :, None] + back
        back = np.exp(delta[:, t, :, None] * A) * q[:, t]
        w[:, t] = back * before[:, t]
    return h, q, w


def scan_bwd(dout, x, dt, A, B, C, D=None, z=None, dt_bias=None, *, gate=True, fwd=True, rev=True):
    """Gradients of scan_fwd's inputs for the gradient dout of its output, as a dict keyed by input."""
    dout, x, dt, A, B, C, D, z, dt_bias = (_f64(v) for v in (dout, x, dt, A, B, C, D, z, dt_bias))
    v = dt if dt_bias is None else dt + dt_bias
    delta = softplus(v)
    u = delta * x
    skip = 0.0 if D is None else D
    k = int(fwd) + int(rev)
    dy = dout * (z * sigmoid(z)) if gate else dout
    h = q = w = 0.0
    for on, reverse in ((fwd, False), (rev, True)):
        if on:
            hd, qd, wd = _direction_grads(delta, u, A, B, C, dy, reverse)
            h, q, w = h + hd, q + qd, w + wd
    du = np.sum(q * B[:, :, None, :], axis=-1)
    ddt = (x * du + np.sum(w * A, axis=-1)) * sigmoid(v)
    g = {
        "x": delta * du + k * skip * dy,
        "dt": ddt,
        "A": np.sum(w * delta[..., None], axis=(0, 1)),
        "B": np.sum(q * u[..., None], axis=2),
        "C": np.sum(h * dy[..., None], axis=2),
        "D": k * np.sum(x * dy, axis=(0, 1)),
        "dt_bias": np.sum(ddt, axis=(0, 1)),
        "z": None,
    }
    if gate:
        g["z"] = dout * (np.sum(h * C[:, :, None, :], axis=-1) + k * skip * x) * silu_grad(z)
    return g


def scan_bwd_magnitudes(dout, x, dt, A, B, C, D=None, z=None, dt_bias=None, *, gate=True, fwd=True, rev=True):
    """For each element of scan_bwd's result, the sum of the magnitudes of the terms it is made of: the same sums
    on absolute values (every decay and step size is positive), the gate's factors taken as they are."""
    ab = lambda a: None if a is None else np.abs(_f64(a))  # noqa: E731
    z = _f64(z)
    dy = ab(dout) * (np.abs(z * sigmoid(z)) if gate else 1.0)
    g = scan_bwd(dy, ab(x), dt, A, ab(B), ab(C), ab(D), None, dt_bias, gate=False, fwd=fwd, rev=rev)
    v = _f64(dt) if dt_bias is None else _f64(dt) + _f64(dt_bias)
    # the decay's part of ddt carries A < 0; with |A| in its place the two parts add
    delta = softplus(v)
    u = delta * ab(x)
    h = w = 0.0
    for on, reverse in ((fwd, False), (rev, True)):
        if on:
            hd, _, wd = _direction_grads(delta, u, _f64(A), ab(B), ab(C), dy, reverse)
            h, w = h + hd, w + wd
    decay = np.sum(w * ab(A), axis=-1) * sigmoid(v)
    g["dt"] = g["dt"] + 2.0 * decay
    g["dt_bias"] = np.sum(g["dt"], axis=(0, 1))
    if gate:
        k = int(fwd) + int(rev)
        y = np.sum(h * ab(C)[:, :, None, :], axis=-1) + (0.0 if D is None else k * ab(D) * ab(x))
        # silu'(z) = s + z s (1 - s) is itself a sum of two terms, which cancel near z = -1.28: rounding s (2^-24
        # relative) moves each by that much of its own size, whatever is left of their sum
        s = sigmoid(z)
        g["z"] = ab(dout) * y * s * (1.0 + np.abs(z) * (1.0 - s))
    return g


def _taps(u, reverse):
    """The four inputs of each output of the width-4 filter: u[t - 3 + k], or u[t + 3 - k] in reverse."""
    nb, L, nc = u.shape
    pad = np.zeros((nb, L + 6, nc))
    pad[:, 3:3 + L] = u
    return [pad[:, 6 - k:6 - k + L] if reverse else pad[:, k:k + L] for k in range(4)]


def conv_bwd(dout_f, dout_r, u, w_f=None, b_f=None, w_r=None, b_r=None, *, act=True):
    """Gradients of conv_bidir's inputs, as a dict keyed by input (None where a direction is not there)."""
    u = _f64(u)
    nb, L, nc = u.shape
    du = np.zeros((nb, L + 6, nc))
    g = {"w_f": None, "b_f": None, "w_r": None, "b_r": None}
    for d, dout, w, b, reverse in (("f", dout_f, w_f, b_f, False), ("r", dout_r, w_r, b_r, True)):
        if w is None:
            continue
        w = _f64(w)
        taps = _taps(u, reverse)
        p = sum(w[:, k] * taps[k] for k in range(4)) + (0.0 if b is None else _f64(b))
        dp = _f64(dout) * (silu_grad(p) if act else 1.0)
        g["w_" + d] = np.stack([np.sum(dp * taps[k], axis=(0, 1)) for k in range(4)], axis=-1)
        g["b_" + d] = None if b is None else np.sum(dp, axis=(0, 1))
        for k in range(4):
            at = 6 - k if reverse else k
            du[:, at:at + L] += w[:, k] * dp
    g["u"] = du[:, 3:3 + L]
    return g


def _mod(p):
    return None if p is None else _f64(p)[:, None, :]


def adaln_fwd(x, gamma=None, beta=None, branch=None, post_weight=None, gate=None, eps=1e-5, *, rms=False):
    """h = x + gate * (RMSNorm(branch) * post_weight), out = gamma * norm(h) + beta; returns (h, out).

    eq. (10): AdaLN, gamma (h - mean) / sigma + beta, one (gamma, beta) per sequence ([batch, d], or [1, d] for
    all); rms leaves out the mean.  eq. (11)-(12): the residual sum around the mixer.  branch None: h = x; gate
    None: 1; post_weight None: the branch is not normalised."""
    h = _f64(x)
    if branch is not None:
        m = _f64(branch)
        if post_weight is not None:
            m = m / np.sqrt(np.mean(m * m, axis=-1, keepdims=True) + eps) * _f64(post_weight)
        h = h + (m if gate is None else _mod(gate) * m)
    c = h if rms else h - np.mean(h, axis=-1, keepdims=True)
    out = c / np.sqrt(np.mean(c * c, axis=-1, keepdims=True) + eps)
    out = out if gamma is None else out * _mod(gamma)
    return h, out if beta is None else out + _mod(beta)


def adaln_bwd(dout, dres, h, gamma=None, beta=None, branch=None, post_weight=None, gate=None, eps=1e-5, *, rms=False):
    """Gradients of adaln_fwd's inputs, given its h and the gradients of out (dout) and of h (dres or None)."""
    dout, h = _f64(dout), _f64(h)
    nb, _, nd = h.shape

    def over_tokens(v, like):
        s = np.sum(v, axis=1)
        return s if like.shape[0] == nb else np.sum(s, axis=0, keepdims=True)

    c = h if rms else h - np.mean(h, axis=-1, keepdims=True)
    r = 1.0 / np.sqrt(np.mean(c * c, axis=-1, keepdims=True) + eps)
    xhat = c * r
    e = dout if gamma is None else dout * _mod(gamma)
    dh = e - xhat * np.mean(e * xhat, axis=-1, keepdims=True)
    if not rms:
        dh = dh - np.mean(e, axis=-1, keepdims=True)
    dh = r * dh + (0.0 if dres is None else _f64(dres))
    g = {"x": dh, "gamma": None if gamma is None else over_tokens(dout * xhat, gamma),
         "beta": None if beta is None else over_tokens(dout, beta), "branch": None, "post_weight": None, "gate": None}
    if branch is None:
        return g
    m = _f64(branch)
    dm = dh if gate is None else dh * _mod(gate)
    if post_weight is None:
        mp = m
    else:
        q = 1.0 / np.sqrt(np.mean(m * m, axis=-1, keepdims=True) + eps)
        mh = m * q
        mp = mh * _f64(post_weight)
        g["post_weight"] = np.sum(dm * mh, axis=(0, 1))
        f = dm * _f64(post_weight)
        dm = q * (f - mh * np.mean(f * mh, axis=-1, keepdims=True))
    if gate is not None:
        g["gate"] = over_tokens(dh * mp, gate)
    g["branch"] = dm
    return g
