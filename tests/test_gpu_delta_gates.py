"""Which tokens the delta rule's gates and their gradients reach, and what infinities in them mean."""
import numpy as np
import pytest

from tests.gpu_util import f32_dev, to_dev, to_host64, torch_mod
from tests.test_gpu_delta import close, make, upload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("L", [40, 64, 150])
def test_decay_gradients_reach_back_from_the_only_gradient(L, rev):
    """dout at one token: the gates of the tokens met up to it have gradients, the others exactly none, as the oracle."""
    import bidirectional_mamba_selective_amd as bm
    import oracle

    inp, dout, _ = make(1, L, 1, 2, 64, 64, seed=L)
    for at in (0, 1, L // 2, L - 1):
        do = np.zeros_like(dout)
        do[:, at] = dout[:, at]
        g = bm.bimamba_delta_bwd(to_dev(do, "bf16"), **upload(inp), flags=bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY)
        want = oracle.delta_bwd(do, inp, rev=rev)
        bound = oracle.delta_bounds(inp, do, rev=rev)
        met = np.arange(L)[::-1] if rev else np.arange(L)
        later = met[list(met).index(at) + 1:]
        for n in ("dt", "b"):
            got = to_host64(g[n])
            assert np.all(np.abs(got - want[n]) <= 2.0 ** -8 * 1.01 * np.abs(want[n]) + bound[n] + 1e-30), (n, at)
            assert np.all(got[:, later] == 0) and np.all(got[:, at] != 0), (n, at)


def infinite(L, where, seed=21):
    """Two versions of the same inputs: infinities in the gates, and large finite values that mean the same (a step of 2^60
    decays by more than e^-256, b = 200 gives beta = 1 to the last bit of 64-bit numbers)."""
    inp, dout, dh = make(2, L, 1, 2, 64, 128, seed=seed)
    fin = {n: None if x is None else x.copy() for n, x in inp.items()}
    for n, big in (("dt", 2.0 ** 60), ("b", 200.0)):
        if n in where:
            at = [t for t in (0, 4, 10, 63, 64, 65, 100) if t < L]
            inp[n][0, at], fin[n][0, at] = np.inf, big
            inp[n][1, at[::2], 1], fin[n][1, at[::2], 1] = np.inf, big
    return inp, fin, dout, dh


def a_terms(inp, ddt):
    x = inp["dt"].astype(np.float64) + inp["dt_bias"]
    return np.abs(ddt * np.logaddexp(x, 0.0) / (inp["A"] / (1 + np.exp(-x)))).sum((0, 1))


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("where", [("dt",), ("b",), ("dt", "b")])
@pytest.mark.parametrize("L", [1, 12, 64, 130])
def test_positive_infinities_are_limits(L, where, rev):
    import bidirectional_mamba_selective_amd as bm
    import oracle

    inp, fin, dout, dh = infinite(L, where)
    dev, flags = upload(inp), bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY
    h = torch_mod().empty(2, 2, 64, 128, device="cuda")
    out = bm.bimamba_delta_fwd(**dev, h_out=h, flags=flags)
    g = bm.bimamba_delta_bwd(to_dev(dout, "bf16"), **dev, dh_out=f32_dev(dh), flags=flags)
    wout, wh = oracle.delta_fwd(fin, rev=rev)
    want = oracle.delta_bwd(dout, fin, dh, rev=rev)
    r = oracle.delta_bounds(fin, dout, dh, rev=rev)
    close(to_host64(out), wout, r["out"], "out")
    close(to_host64(h), wh, r["h_out"], "h_out", bf16=False)
    for n, w in want.items():
        # A: 2^-16 (256 roundings) of its terms delta_t dg_t = delta_t ddt_t / (A sigmoid(x_t)), and 2^4 for what cancels
        # within a term; the oracle's bound holds the step of 2^60 times the errors of terms that are exactly 0
        bound = r[n] if n != "A" else 2.0 ** -12 * a_terms(fin, want["dt"])
        close(to_host64(g[n]), w, bound, "d" + n, bf16=n in ("q", "k", "v", "dt", "b"))
    for n in where:
        assert np.all(to_host64(g[n])[np.isinf(inp[n])] == 0), n


@pytest.mark.parametrize("L,first", [(12, 7), (150, 64)])
def test_where_other_non_finite_values_reach(L, first):
    """q: its own token's out; v: its column; k, dt and b: their heads; from the run (or, up to 16 tokens, the token) on."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    at = 7 if L == 12 else 80
    clean = upload(make(2, L, 2, 4, 64, 64, seed=23)[0])
    h0 = torch.empty(2, 4, 64, 64, device="cuda")
    o0 = bm.bimamba_delta_fwd(**clean, h_out=h0)
    for name in ("q", "k", "v", "dt", "b"):
        for value in (float("nan"),) + ((float("inf"),) if name in ("q", "k", "v") else ()):
            bad = {n: x.clone() for n, x in clean.items()}
            i = (1, at, 1) + ((5,) if name in ("q", "k", "v") else ())
            bad[name][i] = value
            h = torch.empty_like(h0)
            o = bm.bimamba_delta_fwd(**bad, h_out=h)
            heads = slice(2, 4) if name in ("q", "k") else slice(1, 2)  # key head 1 serves heads 2 and 3
            cols = slice(5, 6) if name == "v" else slice(None)
            toks = slice(at, at + 1) if name == "q" else slice(first, None)
            assert not bool(torch.isfinite(o[1, at, heads, cols]).any()), (name, value)
            if name != "q":
                assert bool((~torch.isfinite(h[1, heads][..., cols])).any()), (name, value)
                h[1, heads, :, cols] = h0[1, heads, :, cols]
            o[1, toks, heads, cols] = o0[1, toks, heads, cols]
            assert torch.equal(o, o0) and torch.equal(h, h0), (name, value)


def test_gradients_of_other_non_finite_values_stay_in_their_heads():
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    inp, dout, dh = make(2, 150, 2, 4, 64, 64, seed=29)
    clean, dout, dh = upload(inp), to_dev(dout, "bf16"), f32_dev(dh)
    want = bm.bimamba_delta_bwd(dout, **clean, dh_out=dh)
    for name in ("q", "k", "v", "dt", "b"):
        bad = {n: x.clone() for n, x in clean.items()}
        bad[name][(1, 80, 1) + ((5,) if name in ("q", "k", "v") else ())] = float("nan")
        got = bm.bimamba_delta_bwd(dout, **bad, dh_out=dh)
        heads = [2, 3] if name in ("q", "k") else [1]
        key = 1 if name in ("q", "k") else 0
        # (the gradients of q and v do not depend on q and v, but those of the others do)
        assert any(bool(torch.isnan(g).any()) for g in got.values()), name
        for n, w in want.items():
            g = got[n].clone()
            if n in ("A", "dt_bias"):
                g[heads] = w[heads]
            elif n == "h_in":
                g[1, heads] = w[1, heads]
            elif n in ("q", "k"):
                g[1, :, key] = w[1, :, key]
            else:
                g[1][:, heads] = w[1][:, heads]
            assert torch.equal(g, w), (name, n)
