"""GPU parity of the norm / gate / residual step and its backward pass against the fp64 oracle, through the C ABI.

Bounds, derived from the arithmetic.  Every result is a short expression of row values and of row sums.  A row sum adds
8 values a lane, 6 steps across the lanes and at most 16 wavefronts: below 32 roundings of 2^-24 relative to the sum of
the magnitudes; a reciprocal root halves the relative error of its argument and adds 2^-23.  With fewer than 20 products
around them an element is off by at most 100 x 2^-24 of the magnitudes of its terms (the centred value h - mean(h)
counting as |h| + mean|h|, since it may cancel), plus half a step of its type, 2^-8 relative for bf16.  The sums over
rows add at most one rounding a row: (100 + rows) 2^-24 of the magnitudes summed."""
import numpy as np
import pytest

from bidirectional_mamba_selective_amd import inputs
from tests.gpu_util import f32_dev, say, to_dev, to_host64, torch_mod

pytestmark = pytest.mark.gpu

EPS = 1e-5
U = 2.0 ** -24
ACTS = ("x", "h", "branch", "dout", "dres")


def make(batch, L, d, io, seed=0, rows=None, mean=0.3, scale=3.0, drop=()):
    r = np.random.default_rng(seed)
    rows = batch if rows is None else rows

    def act(m, s):
        return inputs.round_to((m + s * r.standard_normal((batch, L, d))).astype(np.float32), io)

    def vec(n, m, s):
        return (m + s * r.standard_normal((n, d))).astype(np.float32)

    inp = dict(x=act(mean, scale), branch=act(0.1, 1.5), dout=act(0, 1), dres=act(0, 1), gamma=vec(rows, 1, 0.3),
               beta=vec(rows, 0, 0.3), gate=vec(rows, 0.5, 0.4), post_weight=vec(1, 1, 0.3)[0])
    inp["h"] = act(mean, scale)
    for k in drop:
        inp[k] = None
    return inp


def upload(inp, io):
    return {k: None if v is None else to_dev(v, io) if k in ACTS else f32_dev(v) for k, v in inp.items()}


def close(got, want, mag, io, n, tag):
    half = 2.0 ** -8 * 1.01 if io == "bf16" else 0.0
    allow = half * np.abs(want) + n * U * mag + 1e-30
    worst = float(np.max(np.abs(got - want) / allow))
    say(f"{tag}: worst element at {worst:.3f} of its bound")
    assert got.shape == want.shape and np.all(np.isfinite(got)) and worst <= 1.0, tag


def mean_abs(v):
    return np.mean(np.abs(v), axis=-1, keepdims=True)


def mod(p):
    return 1.0 if p is None else np.abs(p.astype(np.float64))[:, None, :]


PARAMS = ("gamma", "beta", "branch", "post_weight", "gate")


def check_fwd(inp, io, rms=False, eps=EPS, **kw):
    import oracle
    import bidirectional_mamba_selective_amd as bm

    dev = upload(inp, io)
    h, out = bm.bimamba_adaln_fwd(dev["x"], *[dev[k] for k in PARAMS], eps=eps, flags=bm.FLAG_RMS_NORM if rms else 0,
                                  **kw)
    wh, wout = oracle.adaln_fwd(inp["x"], *[inp[k] for k in PARAMS], eps=eps, rms=rms)
    mag = np.abs(inp["x"].astype(np.float64))
    if inp["branch"] is not None:
        m = np.abs(inp["branch"].astype(np.float64))
        if inp["post_weight"] is not None:
            m = m / np.sqrt(np.mean(m * m, -1, keepdims=True) + eps) * np.abs(inp["post_weight"])
        mag = mag + m * mod(inp["gate"])
        close(to_host64(h), wh, mag, io, 100, f"h {io}")
    else:
        assert h is dev["x"]
    c = wh if rms else wh - wh.mean(-1, keepdims=True)
    rs = 1 / np.sqrt(np.mean(c * c, -1, keepdims=True) + eps)
    cm = mag if rms else mag + mean_abs(mag)
    # the root's relative error follows the centred values' own: their magnitudes over their size
    spread = np.sqrt(np.mean(cm * cm, -1, keepdims=True)) * rs
    omag = mod(inp["gamma"]) * rs * (cm + np.abs(c) * spread)
    omag = omag + (0.0 if inp["beta"] is None else mod(inp["beta"]))
    close(to_host64(out), wout, omag, io, 100, f"out {io}")


def check_bwd(inp, io, rms=False, eps=EPS, **kw):
    import oracle
    import bidirectional_mamba_selective_amd as bm

    dev = upload(inp, io)
    got = bm.bimamba_adaln_bwd(dev["dout"], dev["dres"], dev["h"], *[dev[k] for k in PARAMS], eps=eps,
                               flags=bm.FLAG_RMS_NORM if rms else 0, **kw)
    want = oracle.adaln_bwd(inp["dout"], inp["dres"], inp["h"], *[inp[k] for k in PARAMS], eps=eps, rms=rms)
    ab = lambda k: np.abs(inp[k].astype(np.float64))  # noqa: E731
    h = inp["h"].astype(np.float64)
    c = h if rms else h - h.mean(-1, keepdims=True)
    rs = 1 / np.sqrt(np.mean(c * c, -1, keepdims=True) + eps)
    cm = np.abs(h) if rms else np.abs(h) + mean_abs(h)
    spread = np.sqrt(np.mean(cm * cm, -1, keepdims=True)) * rs
    xm = rs * (cm + np.abs(c) * spread)
    e = ab("dout") * mod(inp["gamma"])
    dhm = rs * spread * (e + (0 if rms else mean_abs(e)) + xm * np.mean(e * xm, -1, keepdims=True))
    dhm = dhm + (0.0 if inp["dres"] is None else ab("dres"))
    nb, L, _ = h.shape

    def rows(v, like):
        s = v.sum(1)
        return s if like.shape[0] == nb else s.sum(0, keepdims=True)

    mags = {"x": dhm}
    if inp["gamma"] is not None:
        mags["gamma"] = rows(ab("dout") * xm, inp["gamma"])
    if inp["beta"] is not None:
        mags["beta"] = rows(ab("dout"), inp["beta"])
    if inp["branch"] is not None:
        m, g = ab("branch"), mod(inp["gate"])
        mp, w = m, 1.0
        if inp["post_weight"] is not None:
            q = 1 / np.sqrt(np.mean(m * m, -1, keepdims=True) + eps)
            w = np.abs(inp["post_weight"].astype(np.float64))
            mags["post_weight"] = (g * dhm * m * q).sum((0, 1))
            f = g * dhm * w
            mags["branch"] = q * (f + m * q * np.mean(f * m * q, -1, keepdims=True))
            mp = m * q * w
        else:
            mags["branch"] = g * dhm
        if inp["gate"] is not None:
            mags["gate"] = rows(dhm * mp, inp["gate"])
    for k, g in got.items():
        if k not in mags:
            assert g is None and want[k] is None, k
            continue
        act = k in ("x", "branch")
        close(to_host64(g), want[k], mags[k], io if act else "f32", 100 if act else 100 + nb * L, f"d{k} {io}")
    return got


SHAPES = [(1, 1, 8), (2, 3, 64), (1, 5, 512), (2, 7, 520), (3, 33, 1024), (1, 40, 1928), (2, 9, 2048), (1, 6, 4096),
          (2, 5, 8184), (1, 3, 8192)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,d", SHAPES)
def test_adaln_shapes(batch, L, d, io):
    say(f"adaln {batch}x{L}x{d} {io}")
    inp = make(batch, L, d, io, seed=d)
    check_fwd(inp, io)
    check_bwd(inp, io)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("drop", [(), ("branch", "post_weight", "gate"), ("post_weight",), ("gate",), ("gamma",),
                                  ("beta",), ("dres",), ("gamma", "beta", "gate", "post_weight", "dres")])
def test_adaln_options(drop, rms):
    say(f"adaln without {drop} rms={rms}")
    inp = make(2, 11, 264, "f32", seed=3, drop=drop)
    check_fwd(inp, "f32", rms)
    check_bwd(inp, "f32", rms)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_adaln_shared_rows(io):
    """One gamma, beta and gate for the batch: their gradients are sums over all sequences."""
    say(f"adaln shared {io}")
    inp = make(5, 300, 256, io, seed=4, rows=1)
    check_fwd(inp, io)
    check_bwd(inp, io)


def test_adaln_many_rows_per_workgroup():
    """More rows than the launch has workgroups, so that each walks several and the last ones are ragged."""
    say("adaln many rows")
    inp = make(2, 5003, 64, "bf16", seed=5)
    check_fwd(inp, "bf16")
    check_bwd(inp, "bf16")
    inp = make(1, 2500, 1032, "f32", seed=6)
    check_fwd(inp, "f32")
    check_bwd(inp, "f32")


def test_adaln_large_mean_and_outliers():
    """A mean a hundred times the spread, and single columns a thousand times the others: the variance is summed from
    centred values."""
    say("adaln large mean")
    inp = make(1, 9, 2048, "f32", seed=7, mean=300.0)
    check_fwd(inp, "f32")
    check_bwd(inp, "f32")
    inp = make(1, 9, 2048, "f32", seed=8)
    inp["x"][..., 0] += 3000.0
    inp["h"][..., 0] += 3000.0
    check_fwd(inp, "f32")
    check_bwd(inp, "f32")


def test_adaln_constant_rows():
    """Rows of equal values: zero variance leaves beta, and a zero branch leaves x."""
    import bidirectional_mamba_selective_amd as bm

    torch = torch_mod()
    x = torch.full((1, 3, 256), 2.0, device="cuda")
    beta = torch.randn(1, 256, device="cuda")
    h, out = bm.bimamba_adaln_fwd(x, None, beta, torch.zeros_like(x), torch.ones(256, device="cuda"))
    assert torch.equal(h, x) and torch.equal(out, beta.expand(1, 3, 256))
    g = bm.bimamba_adaln_bwd(torch.ones_like(x), None, x, None, beta, torch.zeros_like(x),
                             torch.ones(256, device="cuda"))
    assert all(torch.isfinite(v).all() for v in g.values() if v is not None)


def test_adaln_in_place_and_determinism():
    import bidirectional_mamba_selective_amd as bm

    torch = torch_mod()
    inp = make(3, 700, 1024, "bf16", seed=9)
    dev = upload(inp, "bf16")
    p = [dev[k] for k in PARAMS]
    h, out = bm.bimamba_adaln_fwd(dev["x"], *p)
    x2 = dev["x"].clone()
    h2, out2 = bm.bimamba_adaln_fwd(x2, *p, h=x2)
    assert h2 is x2 and torch.equal(h, h2) and torch.equal(out, out2)
    g = bm.bimamba_adaln_bwd(dev["dout"], dev["dres"], h, *p)
    r2 = dev["dres"].clone()
    g2 = bm.bimamba_adaln_bwd(dev["dout"], r2, h, *p, grads={"x": r2})
    assert g2["x"] is r2
    for k in g:
        assert torch.equal(g[k], g2[k]), k


def test_adaln_bad_values_stay_in_their_rows():
    """An infinity or NaN in a row leaves the other rows' results as they are."""
    import bidirectional_mamba_selective_amd as bm

    torch = torch_mod()
    inp = make(1, 64, 512, "f32", seed=10)
    dev = upload(inp, "f32")
    p = [dev[k] for k in PARAMS]
    h, out = bm.bimamba_adaln_fwd(dev["x"], *p)
    dev["x"][0, 5, 3] = float("inf")
    dev["x"][0, 40, 0] = float("nan")
    h2, out2 = bm.bimamba_adaln_fwd(dev["x"], *p)
    keep = [i for i in range(64) if i not in (5, 40)]
    assert torch.equal(out[:, keep], out2[:, keep]) and torch.equal(h[:, keep], h2[:, keep])
    assert not torch.isfinite(out2[0, 40]).any()


def test_adaln_bwd_agrees_with_differences_of_the_forward_pass():
    """Central differences of the fp32 forward pass, (4 d(h / 2) - d(h)) / 3 at h = 2^-6, along the gradient's sign times
    each element's size: truncation h^4 / 30 of a fifth derivative, rounding ~1e-6 / 2^-7 = 1.3e-4."""
    import bidirectional_mamba_selective_amd as bm

    torch = torch_mod()
    inp = make(2, 20, 264, "f32", seed=11)
    dev = upload(inp, "f32")
    args = {k: dev[k] for k in ("x",) + PARAMS}
    h, _ = bm.bimamba_adaln_fwd(*args.values())
    got = bm.bimamba_adaln_bwd(dev["dout"], dev["dres"], h, *[dev[k] for k in PARAMS])

    def loss(v):
        hh, out = bm.bimamba_adaln_fwd(*v.values())
        return ((out.double() * dev["dout"].double()).sum() + (hh.double() * dev["dres"].double()).sum()).item()

    for k in args:
        v = torch.sign(got[k]) * args[k].abs()
        want = (got[k].double() * v.double()).sum().item()

        def difference(step):
            hi, lo = (loss(dict(args, **{k: args[k] + s * step * v})) for s in (1, -1))
            return (hi - lo) / (2 * step)

        rate = (4 * difference(2.0 ** -7) - difference(2.0 ** -6)) / 3
        say(f"d{k}: difference {rate:.6g}, gradient {want:.6g}")
        assert abs(rate - want) <= 2e-3 * abs(want), k
