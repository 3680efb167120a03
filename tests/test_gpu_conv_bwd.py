"""GPU parity of the short convolution's backward pass against the fp64 oracle, through the C ABI.

Bounds, derived from the arithmetic.  The filter's sum p carries 5 roundings of 2^-24 relative to m_p = |b| + sum |w u|;
silu'' is below 1/2, so they move silu'(p) by at most 2.5 x 2^-24 m_p, and its own evaluation (an exponential, a
reciprocal, four products) by less than 10 x 2^-24 of s (1 + |p| (1 - s)).  du adds eight products: an element is off by
at most 30 x 2^-24 of the magnitudes of its terms, those of dp taken as |dout| (s (1 + |p| (1 - s)) + m_p), plus half a
step of its type (2^-8 relative for bf16).  The sums over tokens add at most one rounding a token."""
import numpy as np
import pytest

from bidirectional_mamba_selective_amd import inputs
from tests.gpu_util import f32_dev, say, to_dev, to_host64, torch_mod

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def make(batch, L, C, io, seed=0, dirs="both", bias=True):
    r = np.random.default_rng(seed)
    act = lambda: inputs.round_to(r.standard_normal((batch, L, C)).astype(np.float32), io)  # noqa: E731
    inp = dict(u=act())
    for d in "fr":
        on = dirs in ("both", d)
        inp["dout_" + d] = act() if on else None
        inp["w_" + d] = (0.5 * r.standard_normal((C, 4))).astype(np.float32) if on else None
        inp["b_" + d] = (0.1 * r.standard_normal(C)).astype(np.float32) if on and bias else None
    return inp


NAMES = ("dout_f", "dout_r", "u", "w_f", "b_f", "w_r", "b_r")


def upload(inp, io):
    return {k: None if v is None else to_dev(v, io) if k[0] in "ud" else f32_dev(v) for k, v in inp.items()}


def magnitudes(inp, act):
    """Per result the magnitudes of its terms, by the oracle without its activation on the magnitudes of dp."""
    import oracle
    from oracle.grads import _taps, sigmoid

    u = np.abs(inp["u"].astype(np.float64))
    dm = {}
    for d, reverse in (("f", False), ("r", True)):
        if inp["w_" + d] is None:
            dm[d] = None
            continue
        w = inp["w_" + d].astype(np.float64)
        b = 0.0 if inp["b_" + d] is None else inp["b_" + d].astype(np.float64)
        p = sum(w[:, k] * t for k, t in enumerate(_taps(inp["u"].astype(np.float64), reverse))) + b
        mp = sum(np.abs(w[:, k]) * t for k, t in enumerate(_taps(u, reverse))) + np.abs(b)
        s = sigmoid(p)
        dm[d] = np.abs(inp["dout_" + d].astype(np.float64)) * ((s * (1 + np.abs(p) * (1 - s)) + mp) if act else 1.0)
    aw = {k: None if inp[k] is None else np.abs(inp[k]) for k in ("w_f", "b_f", "w_r", "b_r")}
    return oracle.conv_bwd(dm["f"], dm["r"], u, aw["w_f"], aw["b_f"], aw["w_r"], aw["b_r"], act=False)


def check(inp, io, act=True, **kw):
    import oracle
    import bidirectional_mamba_selective_amd as bm

    dev = upload(inp, io)
    got = bm.bimamba_conv1d_bidir_bwd(*[dev[k] for k in NAMES], flags=0 if act else bm.FLAG_NO_SILU, **kw)
    want = oracle.conv_bwd(*[inp[k] for k in NAMES], act=act)
    mag = magnitudes(inp, act)
    rows = inp["u"].shape[0] * inp["u"].shape[1]
    for k, g in got.items():
        if want[k] is None:
            assert g is None, k
            continue
        o = to_host64(g)
        half = 2.0 ** -8 * 1.01 if io == "bf16" and k == "u" else 0.0
        allow = half * np.abs(want[k]) + (30 + (0 if k == "u" else rows)) * U * mag[k] + 1e-30
        worst = float(np.max(np.abs(o - want[k]) / allow))
        say(f"d{k} {io}: worst element at {worst:.3f} of its bound")
        assert o.shape == want[k].shape and np.all(np.isfinite(o)) and worst <= 1.0, k
    return got


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,C", [(1, 1, 4), (2, 2, 8), (1, 3, 4), (1, 4, 132), (2, 7, 64), (1, 8, 128),
                                       (3, 9, 260), (2, 33, 1028), (1, 1000, 12), (2, 515, 256)])
def test_conv_bwd_shapes(batch, L, C, io):
    say(f"conv_bwd {batch}x{L}x{C} {io}")
    check(make(batch, L, C, io, seed=L), io)


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("dirs", ["both", "f", "r"])
def test_conv_bwd_variants(dirs, bias, act):
    say(f"conv_bwd {dirs} bias={bias} act={act}")
    check(make(2, 75, 68, "f32", seed=3, dirs=dirs, bias=bias), "f32", act)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_conv_bwd_long_tiles(io):
    """Enough channels that a wavefront walks a tile of several steps, the last one ragged."""
    say(f"conv_bwd long tiles {io}")
    check(make(8, 1037, 2048, io, seed=4), io)


def test_conv_bwd_one_token_gradients_reach_their_neighbours():
    """A gradient at one token of out_f or out_r moves exactly the four tokens its filter reads, across tile and
    workgroup borders and at both ends of the sequence."""
    import bidirectional_mamba_selective_amd as bm

    torch = torch_mod()
    L, C = 600, 4
    u = torch.randn(1, L, C, device="cuda")
    w = torch.ones(C, 4, device="cuda")
    for t in [0, 1, 3, 7, 8, 31, 32, 33, 300, L - 4, L - 1]:
        g = torch.zeros(1, L, C, device="cuda")
        g[0, t] = 1.0
        z = torch.zeros_like(g)
        f = bm.bimamba_conv1d_bidir_bwd(g, z, u, w, None, w, None, flags=bm.FLAG_NO_SILU)
        r = bm.bimamba_conv1d_bidir_bwd(z, g, u, w, None, w, None, flags=bm.FLAG_NO_SILU)
        for got, lo, hi in ((f["u"], t - 3, t), (r["u"], t, t + 3)):
            want = torch.zeros_like(g)
            want[0, max(lo, 0):min(hi, L - 1) + 1] = 1.0
            assert torch.equal(got, want), t
        pad = torch.nn.functional.pad(u[0], (0, 0, 3, 3))
        assert torch.equal(f["w_f"], pad[t:t + 4].T.contiguous()), t
        assert torch.equal(r["w_r"], pad[t + 3:t + 7].flip(0).T.contiguous()), t
        assert torch.count_nonzero(f["w_r"]) == 0 and torch.count_nonzero(r["w_f"]) == 0


def test_conv_bwd_determinism():
    torch = torch_mod()
    inp = make(2, 900, 512, "bf16", seed=5)
    one, two = check(inp, "bf16"), check(inp, "bf16")
    for k in one:
        assert torch.equal(one[k], two[k]), k
