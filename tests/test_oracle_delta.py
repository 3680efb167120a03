"""Pins of the delta rule's oracle: one token written out, the limits without decay or correction, differences of the
forward function, the flipped sequence, one call against two, and planted mistakes that the bounds have to see."""
import numpy as np
import pytest

import oracle


def make(batch=2, L=9, hk=1, heads=2, dk=4, dv=3, seed=0, state=True):
    r = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    inp = dict(q=unit(r.standard_normal((batch, L, hk, dk))), k=unit(r.standard_normal((batch, L, hk, dk))),
               v=r.standard_normal((batch, L, heads, dv)), dt=0.5 * r.standard_normal((batch, L, heads)),
               A=-r.uniform(0.2, 2.0, heads), b=r.standard_normal((batch, L, heads)),
               dt_bias=r.uniform(-3.0, 0.0, heads), h_in=r.standard_normal((batch, heads, dk, dv)) if state else None)
    return inp, r.standard_normal((batch, L, heads, dv)), r.standard_normal((batch, heads, dk, dv))


def test_one_token():
    inp, _, _ = make(batch=1, L=1, heads=1)
    out, h = oracle.delta_fwd(inp, scale=0.7)
    k, q, v, S = inp["k"][0, 0, 0], inp["q"][0, 0, 0], inp["v"][0, 0, 0], inp["h_in"][0, 0]
    a = np.exp(inp["A"][0] * np.log1p(np.exp(inp["dt"][0, 0, 0] + inp["dt_bias"][0])))
    want = a * S + np.outer(k, (v - a * S.T @ k)) / (1 + np.exp(-inp["b"][0, 0, 0]))
    np.testing.assert_allclose(h[0, 0], want, rtol=1e-13)
    np.testing.assert_allclose(out[0, 0, 0], 0.7 * want.T @ q, rtol=1e-12)


def test_full_correction_stores_the_value():
    """beta = 1 and |k| = 1: the state answers v_t to k_t, whatever it held."""
    inp, _, _ = make()
    inp["b"][:] = 40.0
    inp["q"] = inp["k"]
    out, _ = oracle.delta_fwd(inp, scale=1.0)
    np.testing.assert_allclose(out, inp["v"], atol=1e-12)


def test_masked_tokens_leave_the_state():
    inp, _, _ = make()
    whole = {n: x for n, x in inp.items()}
    for n in ("dt", "b"):
        whole[n] = inp[n].copy()
        whole[n][:, 4:7] = -np.inf
    cut = {n: np.delete(x, [4, 5, 6], 1) if n in ("q", "k", "v", "dt", "b") else x for n, x in inp.items()}
    np.testing.assert_allclose(oracle.delta_fwd(whole)[1], oracle.delta_fwd(cut)[1], rtol=1e-13)


def test_two_calls_and_flip():
    inp, _, _ = make()
    first = {n: x[:, :4] if n in ("q", "k", "v", "dt", "b") else x for n, x in inp.items()}
    o1, h = oracle.delta_fwd(first)
    o2, h2 = oracle.delta_fwd({n: x[:, 4:] if n in ("q", "k", "v", "dt", "b") else x for n, x in {**inp, "h_in": h}.items()})
    out, hw = oracle.delta_fwd(inp)
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), out, rtol=1e-12)
    np.testing.assert_allclose(h2, hw, rtol=1e-12)
    back = {n: x[:, ::-1] if n in ("q", "k", "v", "dt", "b") else x for n, x in inp.items()}
    np.testing.assert_array_equal(oracle.delta_fwd(back, rev=True)[0], out[:, ::-1])


@pytest.mark.parametrize("rev", [False, True])
def test_gradients_by_differences(rev):
    inp, dout, dh = make(heads=4, hk=2)
    loss = lambda x: (lambda o, h: (o * dout).sum() + (h * dh).sum())(*oracle.delta_fwd(x, rev=rev))  # noqa: E731
    g = oracle.delta_bwd(dout, inp, dh, rev=rev)
    r = np.random.default_rng(1)
    for n in ("q", "k", "v", "dt", "A", "b", "dt_bias", "h_in"):
        d = r.standard_normal(inp[n].shape)
        step = 1e-5
        num = (loss({**inp, n: inp[n] + step * d}) - loss({**inp, n: inp[n] - step * d})) / (2 * step)
        assert abs(num - (g[n] * d).sum()) <= 1e-7 * (1 + abs(num)), n


@pytest.mark.parametrize("mistake", ["decay", "beta", "order", "shared", "skip"])
def test_bounds_see_mistakes(mistake):
    """Each wrong variant of the forward function lies outside the bounds that the GPU results are held to."""
    inp, _, _ = make(L=70, heads=2, hk=2, dk=64, dv=64, batch=1)
    bad = {n: None if x is None else x.copy() for n, x in inp.items()}
    if mistake == "decay":
        bad["dt"][:, 64] = -30.0          # one token's decay left out
    elif mistake == "beta":
        bad["b"][:, 63] += 0.05
    elif mistake == "order":
        for n in ("q", "k", "v", "dt", "b"):
            bad[n][:, [10, 11]] = bad[n][:, [11, 10]]
    elif mistake == "shared":
        bad["k"] = bad["k"][:, :, ::-1]   # the wrong key head
    else:
        bad["b"][:, 69] = -np.inf
    out, h = oracle.delta_fwd(inp)
    got, hg = oracle.delta_fwd(bad)
    r = oracle.delta_bounds(inp)
    assert np.any(np.abs(got - out) > 2.0 ** -8 * np.abs(out) + r["out"][..., None]) or mistake == "skip"
    assert np.any(np.linalg.norm(hg - h, axis=(2, 3)) > r["h_out"]) or mistake == "order"
