"""The gradient oracle (oracle/grads.py) pinned on the CPU: central differences of the forward oracles, closed
forms that do not go through the recurrences, and planted mistakes that a pin has to catch."""
import numpy as np
import pytest

import oracle
import oracle.grads as ograds

RNG = np.random.default_rng


def scan_case(seed, nb=2, L=5, nd=3, ns=2):
    r = RNG(seed)
    n = r.standard_normal
    return dict(x=n((nb, L, nd)), dt=n((nb, L, nd)), A=-np.exp(n((nd, ns))), B=n((nb, L, ns)), C=n((nb, L, ns)),
                D=n(nd), z=n((nb, L, nd)), dt_bias=n(nd)), n((nb, L, nd))


def differences(loss, inp, names, step=1e-6):
    """Central differences of loss(inp) by every element of inp[name]."""
    got = {}
    for name in names:
        g = np.zeros_like(inp[name])
        for i in np.ndindex(g.shape):
            hi, lo = inp[name].copy(), inp[name].copy()
            hi[i] += step
            lo[i] -= step
            g[i] = (loss(dict(inp, **{name: hi})) - loss(dict(inp, **{name: lo}))) / (2 * step)
        got[name] = g
    return got


def assert_grads(got, want):
    # truncation of the differences ~ step^2 = 1e-12 of third derivatives, rounding 1e-16 / 1e-6 = 1e-10 of a loss ~ 1e1
    for k, w in want.items():
        assert np.max(np.abs(got[k] - w)) <= 2e-8 * max(1.0, np.max(np.abs(w))), k


MODES = [dict(), dict(fwd=False), dict(rev=False), dict(gate=False), dict(gate=False, rev=False)]


def pin_scan_differences():
    for seed, mode in enumerate(MODES):
        inp, dout = scan_case(seed)
        got = oracle.grads.scan_bwd(dout, **inp, **mode)
        names = [k for k in inp if mode.get("gate", True) or k != "z"]
        assert_grads(got, differences(lambda v: float(np.sum(oracle.scan_fwd(**v, **mode) * dout)), inp, names))


def pin_scan_flip():
    """The reverse layer's gradients are the forward layer's on the flipped sequence."""
    inp, dout = scan_case(11, L=7)
    flip = {k: (v[:, ::-1] if v.ndim == 3 else v) for k, v in inp.items()}
    f = oracle.grads.scan_bwd(dout[:, ::-1], **flip, rev=False)
    r = oracle.grads.scan_bwd(dout, **inp, fwd=False)
    for k in r:
        want = f[k][:, ::-1] if f[k].ndim == 3 else f[k]
        assert np.allclose(r[k], want, rtol=1e-12, atol=1e-12), k


def pin_scan_one_token():
    """L = 1, no gate: y = k (delta x C.B + D x) has no recurrence; the gradients are the product rule's."""
    inp, dout = scan_case(12, L=1)
    g = oracle.grads.scan_bwd(dout, **inp, gate=False)
    v = inp["dt"] + inp["dt_bias"]
    delta, cb = np.logaddexp(v, 0.0), np.sum(inp["B"] * inp["C"], -1)[..., None]
    assert np.allclose(g["x"], 2 * dout * (delta * cb + inp["D"]))
    assert np.allclose(g["dt"], 2 * dout * inp["x"] * cb / (1 + np.exp(-v)))
    assert np.all(g["A"] == 0)


PINS = [pin_scan_differences, pin_scan_flip, pin_scan_one_token]


@pytest.mark.parametrize("pin", PINS, ids=lambda p: p.__name__)
def test_scan_pins(pin):
    pin()


def _mutant(**change):
    real = ograds._direction_grads

    def planted(delta, u, A, B, C, dy, reverse):
        if change.get("swap"):
            B, C = C, B
        h, q, w = real(delta, u, A, B, C, dy, reverse if not change.get("same_way") else False)
        if change.get("own_decay"):  # w from h_t instead of h_{t-1}
            w = q * h
        if change.get("late"):  # the adjoint of the token after
            q = np.roll(q, 1, axis=1)
        return h, q, w
    return planted


@pytest.mark.parametrize("change", ["swap", "same_way", "own_decay", "late"])
def test_planted_mistakes_fail_a_pin(monkeypatch, change):
    monkeypatch.setattr(ograds, "_direction_grads", _mutant(**{change: True}))
    failed = 0
    for pin in PINS:
        try:
            pin()
        except AssertionError:
            failed += 1
    assert failed


def test_scan_magnitudes_bound_the_gradients():
    inp, dout = scan_case(13, L=9)
    g = oracle.scan_bwd(dout, **inp)
    m = oracle.scan_bwd_magnitudes(dout, **inp)
    for k in g:
        assert np.all(np.abs(g[k]) <= m[k] * (1 + 1e-12)), k


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("dirs", ["both", "f", "r"])
def test_conv_differences(act, dirs):
    r = RNG(3)
    inp = dict(u=r.standard_normal((2, 6, 3)))
    dout = {}
    for d in "fr":
        if dirs in ("both", d):
            inp["w_" + d], inp["b_" + d] = r.standard_normal((3, 4)), r.standard_normal(3)
            dout[d] = r.standard_normal((2, 6, 3))

    def loss(v):
        t = 0.0
        if "w_f" in v:
            t += np.sum(oracle.conv_causal(v["u"], v["w_f"], v["b_f"], act=act) * dout["f"])
        if "w_r" in v:
            t += np.sum(oracle.conv_anticausal(v["u"], v["w_r"], v["b_r"], act=act) * dout["r"])
        return float(t)

    got = oracle.conv_bwd(dout.get("f"), dout.get("r"), inp["u"], inp.get("w_f"), inp.get("b_f"), inp.get("w_r"),
                          inp.get("b_r"), act=act)
    assert_grads(got, differences(loss, inp, list(inp)))


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("rows", [2, 1])
@pytest.mark.parametrize("post,gated", [(True, True), (False, True), (True, False), (False, False)])
def test_adaln_differences(rms, rows, post, gated):
    r = RNG(4)
    n = r.standard_normal
    inp = dict(x=n((2, 3, 5)), gamma=n((rows, 5)), beta=n((rows, 5)), branch=n((2, 3, 5)))
    if post:
        inp["post_weight"] = n(5)
    if gated:
        inp["gate"] = n((rows, 5))
    dout, dres = n((2, 3, 5)), n((2, 3, 5))

    def loss(v):
        h, out = oracle.adaln_fwd(**v, rms=rms)
        return float(np.sum(out * dout) + np.sum(h * dres))

    rest = {k: inp[k] for k in inp if k != "x"}
    got = oracle.adaln_bwd(dout, dres, oracle.adaln_fwd(**inp, rms=rms)[0], **rest, rms=rms)
    assert_grads(got, differences(loss, inp, list(inp)))


def test_adaln_closed_forms():
    """A row of equal values has a zero norm; scaling a branch leaves its post-norm (eps 0) as it is."""
    x = np.full((1, 2, 8), 3.0)
    h, out = oracle.adaln_fwd(x)
    assert np.all(out == 0) and np.all(h == 3.0)
    r = RNG(5)
    b, w = r.standard_normal((1, 2, 8)), r.standard_normal(8)
    one, _ = oracle.adaln_fwd(x, branch=b, post_weight=w, eps=0.0)
    two, _ = oracle.adaln_fwd(x, branch=7 * b, post_weight=w, eps=0.0)
    assert np.allclose(one, two)
    assert np.allclose(np.sqrt(np.mean(((one - x) / w) ** 2, -1)), 1.0)
