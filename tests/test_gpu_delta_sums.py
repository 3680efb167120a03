"""The delta rule's sums before their last rounding: results in which two terms nearly cancel, so that what an operand of a
product lacks of its 24 bits shows in a bf16 result.

Two unit keys e0 and e1 carry one value each, and a query reads c0 times the one less c1 times the other; values are chosen
so that the difference is 2^-12 to 2^-10 of the terms.  Operands of 24 bits leave: the gates, 2^-22 (an exponential, a
reciprocal, a softplus and a product, at most 4 roundings of 2^-24), and the sum's, 2^-23, of each term; the result's half
step is 2^-8 of it.  Operands of 17 bits would be off by 2^-17 of a term, 2^-7 to 2^-5 of the result."""
import numpy as np
import pytest

from bidirectional_mamba_selective_amd import inputs
from tests.gpu_util import f32_dev, say, to_dev, to_host64, torch_mod

pytestmark = pytest.mark.gpu

T0, T1, TQ = 3, 5, 9  # the tokens of the two keys and of the query


def near(c0, c1, n, seed):
    """n pairs of bf16 values with c0 v0 - c1 v1 between 2^-12 and 2^-10 of c0 v0."""
    r = np.random.default_rng(seed)
    v0, v1 = [], []
    while len(v0) < n:
        a = inputs.round_to(r.uniform(1, 2, 4096).astype(np.float32), "bf16").astype(np.float64)
        b = inputs.round_to((c0 * a / c1).astype(np.float32), "bf16").astype(np.float64)
        d = np.abs(c0 * a - c1 * b) / (c0 * a)
        keep = (d > 2.0 ** -12) & (d < 2.0 ** -10)
        v0 += list(a[keep])
        v1 += list(b[keep])
    return np.array(v0[:n]), np.array(v1[:n])


def tokens(L, dk, dv):
    """Tokens that leave the state as it is and answer 0."""
    z = lambda *s: np.zeros(s, np.float32)  # noqa: E731
    return dict(q=z(1, L, 1, dk), k=z(1, L, 1, dk), v=z(1, L, 1, dv), dt=np.full((1, L, 1), -np.inf, np.float32),
                b=np.full((1, L, 1), -np.inf, np.float32), A=np.full(1, -1.0, np.float32))


def case(kind, L, dk, dv, rev):
    """(inputs, the terms of token TQ's result)"""
    inp = tokens(L, dk, dv)
    t0, t1, tq = (L - 1 - t if rev else t for t in (T0, T1, TQ))
    inp["q"][0, tq, 0, :2] = 1, -1
    if kind == "state":       # both values are in the state already, in all their bits
        r = np.random.default_rng(L)
        h = np.zeros((1, 1, dk, dv), np.float32)
        h[0, 0, 0] = r.uniform(1, 2, dv)
        h[0, 0, 1] = h[0, 0, 0] * (1 + r.uniform(2.0 ** -12, 2.0 ** -10, dv))
        inp["h_in"] = h
        return inp, h[0, 0, :2].astype(np.float64)
    if kind == "correction":  # corrections beta v
        b = np.array([1.0, 0.25])
        c = 1 / (1 + np.exp(-b))
    else:                     # scores that carry a decay, corrections v
        b = np.array([40.0, 40.0])
        dt = 1.78125  # of such steps' decays one of the farthest from 17 bits
        inp["dt"][0, t1] = dt
        c = np.array([np.exp(-np.logaddexp(dt, 0.0)), 1.0])
    v = near(c[0], c[1], dv, L)
    for t, i in ((t0, 0), (t1, 1)):
        inp["k"][0, t, 0, i] = 1
        inp["v"][0, t, 0] = v[i]
        inp["b"][0, t] = b[i]
    return inp, np.stack([c[0] * v[0], c[1] * v[1]])


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("kind", ["state", "correction", "score"])
@pytest.mark.parametrize("L,dk,dv", [(12, 64, 64), (64, 64, 64), (64, 128, 128), (100, 64, 128), (100, 128, 64)])
def test_cancelling_terms_of_out(kind, L, dk, dv, rev):
    import bidirectional_mamba_selective_amd as bm

    inp, terms = case(kind, L, dk, dv, rev)
    dev = {n: to_dev(x, "bf16") if n in ("q", "k", "v", "dt", "b") else f32_dev(x) for n, x in inp.items()}
    scale = 0.125
    out = bm.bimamba_delta_fwd(**dev, scale=scale, flags=bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY)
    got = to_host64(out)[0, L - 1 - TQ if rev else TQ, 0]
    want = scale * (terms[0] - terms[1])
    allow = 2.0 ** -8 * np.abs(want) + 2 * (2.0 ** -22 + 2.0 ** -23) * scale * terms[0]
    worst = float(np.max(np.abs(got - want) / allow))
    say(f"{kind} L {L} {dk} x {dv}: worst element at {worst:.3f} of its bound")
    assert worst <= 1.0


def opposite(a, r):
    """-a, but for one place, where both are about 2^-6 and the other is 2^-7 larger: their sum is about 2^-13."""
    a, c = a.copy(), r.integers(0, a.shape[-1])
    a[..., c] = 2.0 ** -6 * (1 + r.integers(0, 64) / 128)
    b = -a
    b[..., c] *= 1 + 2.0 ** -7
    b = inputs.round_to(b.astype(np.float32), "bf16")
    return a, b


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("L,dk,dv", [(64, 64, 64), (64, 128, 128), (64, 64, 128), (100, 128, 64)])
def test_cancelling_terms_of_the_gradients_of_q_and_k(L, dk, dv, rev):
    """dq of a token whose two terms D1 k nearly cancel (two orthogonal keys with one coordinate alike, values nearly
    opposite); dk of a token whose terms D1 q, two and two, nearly cancel (one query, gradients nearly opposite).  A score
    is a sum of dv products: 2^-22 of their magnitudes, which 24-bit operands keep; 17 bits would be off by 2^-17 of the
    score, some 2^3 half steps of the difference."""
    import bidirectional_mamba_selective_amd as bm
    import oracle

    r, scale = np.random.default_rng(dk + dv), 0.125
    rnd = lambda *s: inputs.round_to(r.standard_normal(s).astype(np.float32), "bf16")  # noqa: E731
    at = (lambda t: L - 1 - t) if rev else (lambda t: t)
    n = 10
    inp = tokens(L, dk, dv)
    dout = np.zeros((1, L, 1, dv), np.float32)
    v0, v1 = opposite(rnd(dv), r)
    for t, key, v in ((T0, (0.5, 0.5), v0), (T1, (0.5, -0.5), v1)):
        inp["k"][0, at(t), 0, :2] = key
        inp["v"][0, at(t), 0] = v
        inp["b"][0, at(t)] = 40
    pairs = [(TQ + 2 * m, TQ + 2 * m + 1) for m in range(n)]
    for m, (t0, t1) in enumerate(pairs):
        dout[0, at(t0), 0], dout[0, at(t1), 0] = opposite(rnd(dv), r)
        inp["q"][0, [at(t0), at(t1)], 0, 2 + m] = 1
    dev = {x: to_dev(y, "bf16") if x in ("q", "k", "v", "dt", "b") else f32_dev(y) for x, y in inp.items()}
    g = bm.bimamba_delta_bwd(to_dev(dout, "bf16"), **dev, scale=scale, flags=bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY)
    want = oracle.delta_bwd(dout, inp, scale=scale, rev=rev)
    for m, (t0, t1) in enumerate(pairs):
        terms = scale * float((np.abs(dout[0, at(t0), 0]) * np.abs(v0)).sum())
        for name, t, c, size in (("q", t0, 0, 0.5), ("q", t1, 0, 0.5), ("k", T0, 2 + m, 1.0), ("k", T1, 2 + m, 1.0)):
            got, w = to_host64(g[name])[0, at(t), 0, c], want[name][0, at(t), 0, c]
            allow = 2.0 ** -8 * abs(w) + 2.0 ** -22 * 2 * size * terms
            assert abs(got - w) <= allow, (name, t, got, w, abs(got - w) / allow)
