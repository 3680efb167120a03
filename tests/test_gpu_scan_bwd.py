"""GPU parity of the scan's backward pass against the fp64 gradient oracle, through the C ABI.

Bounds, derived from the arithmetic.  An element of a gradient is a sum of terms, each a product of inputs, step
sizes and a decay over at most L tokens.  Per step the decay carries the exponential's rounding (2^-23) and the
rounding of its argument, delta and the product (3 x 2^-24 relative of an argument whose own exponential it
weights, |arg| e^-|arg| < 0.4), and the recurrence one rounding of its own: below 5 x 2^-24 a step, for the scan
and again for its adjoint, so 10 L x 2^-24 over both in the worst case; the factors outside the recurrence (two
activations, their derivatives and about a dozen products, 2^-23 each) and the sums over channels and states (at
most 64 + 64 adds a partial sum) stay below 300 x 2^-24.  So |o - r| <= (10 L + 300) 2^-24 m, m the sum of the
terms' magnitudes, plus half a step of the output's type, 2^-8 |r| for bf16.  Normwise these roundings are
independent: of order sqrt(L) 2^-23 (1e-5 for L up to 1000) and 2^-8 / sqrt(3) = 2.3e-3 for a bf16 output.
"""
import numpy as np
import pytest

from bidirectional_mamba_selective_amd import inputs
from tests.gpu_util import say, to_dev, f32_dev, to_host64, torch_mod

pytestmark = pytest.mark.gpu

VECTORS = ("A", "D", "dt_bias")  # fp32 whatever the I/O type


def make(batch, L, d_inner, d_state, io, seed=0, trained=True, shift=0.0):
    rng = np.random.default_rng(seed)
    A, _, bias = inputs.make_params(d_inner, d_state, seed=seed, a_jitter=0.4 if trained else 0.0)
    act = inputs.make_activations(batch, L, d_inner, d_state, io, seed=seed + 1)
    inp = {k: act[k] for k in ("x", "dt", "z", "B", "C")}
    inp.update(A=A, D=rng.standard_normal(d_inner).astype(np.float32), dt_bias=(bias + np.float32(shift)))
    dout = inputs.round_to(rng.standard_normal((batch, L, d_inner)).astype(np.float32), io)
    return inp, dout


def upload(inp, dout, io):
    dev = {k: (f32_dev(v) if k in VECTORS else to_dev(v, io)) for k, v in inp.items()}
    return dev, to_dev(dout, io)


MODES = {"both": {}, "fwd": dict(rev=False), "rev": dict(fwd=False)}


def flags_of(dirs, gate):
    import bidirectional_mamba_selective_amd as bm

    return {"both": 0, "fwd": bm.FLAG_FWD_ONLY, "rev": bm.FLAG_REV_ONLY}[dirs] | (0 if gate else bm.FLAG_NO_GATE)


def run(dev, dout, dirs="both", gate=True, **kw):
    import bidirectional_mamba_selective_amd as bm

    return bm.bimamba_scan_bwd(dout, dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev.get("D"),
                               dev["z"] if gate else None, dev.get("dt_bias"), flags=flags_of(dirs, gate), **kw)


def check_grads(got, inp, dout, io, L, dirs="both", gate=True, tag=""):
    import oracle

    args = [inp[k] for k in ("x", "dt", "A", "B", "C")] + [inp.get("D"), inp["z"] if gate else None,
                                                            inp.get("dt_bias")]
    want = oracle.scan_bwd(dout, *args, gate=gate, **MODES[dirs])
    mag = oracle.scan_bwd_magnitudes(dout, *args, gate=gate, **MODES[dirs])
    for k, g in got.items():
        if g is None:
            assert k == "z" and not gate or inp.get(k) is None
            continue
        o, r = to_host64(g), want[k]
        assert o.shape == r.shape, k
        half = 2.0 ** -8 if io == "bf16" and k not in VECTORS else 0.0
        allow = half * np.abs(r) * 1.01 + (10 * L + 300) * 2.0 ** -24 * mag[k] + 1e-30
        worst = float(np.max(np.abs(o - r) / allow))
        norm = float(np.linalg.norm(o - r) / max(np.linalg.norm(r), 1e-300))
        say(f"{tag} d{k}: normwise {norm:.2e}, worst element at {worst:.3f} of its bound")
        assert np.all(np.isfinite(o)) and worst <= 1.0, (tag, k)
        # a gradient whose terms cancel (one token: dA = 0) has no norm to compare with
        if np.linalg.norm(r) > 1e-3 * np.linalg.norm(mag[k]):
            assert norm <= (2.5e-3 if half else 1e-5), (tag, k)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,d_inner,d_state", [
    (1, 1, 64, 1), (1, 2, 64, 16), (2, 15, 64, 3), (1, 16, 128, 16), (3, 17, 64, 5), (2, 33, 192, 16), (1, 257, 64, 7),
    (2, 100, 320, 12),
])
def test_scan_bwd_small(batch, L, d_inner, d_state, io):
    say(f"scan_bwd {batch}x{L}x{d_inner} N {d_state} {io}")
    inp, dout = make(batch, L, d_inner, d_state, io, seed=L)
    dev, g = upload(inp, dout, io)
    check_grads(run(dev, g), inp, dout, io, L, tag=f"{batch}x{L}x{d_inner}x{d_state} {io}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("dirs", ["both", "fwd", "rev"])
def test_scan_bwd_modes(dirs, gate, io):
    say(f"scan_bwd {dirs} gate={gate} {io}")
    inp, dout = make(2, 75, 128, 10, io, seed=5)
    dev, g = upload(inp, dout, io)
    check_grads(run(dev, g, dirs, gate), inp, dout, io, 75, dirs, gate, tag=f"{dirs} gate={gate} {io}")


@pytest.mark.parametrize("dirs,io", [("both", "f32"), ("fwd", "bf16"), ("rev", "f32")])
def test_scan_bwd_many_tiles_per_chunk(dirs, io):
    """Enough channels and batch that a chunk holds several tiles, the last one ragged."""
    from bidirectional_mamba_selective_amd import bimamba_scan_bwd_workspace_bytes

    batch, L, d_inner, d_state = 40, 139, 1024, 2
    assert bimamba_scan_bwd_workspace_bytes(batch, L, d_inner, d_state) > 0
    say(f"scan_bwd many tiles {dirs} {io}")
    inp, dout = make(batch, L, d_inner, d_state, io, seed=9)
    dev, g = upload(inp, dout, io)
    check_grads(run(dev, g, dirs), inp, dout, io, L, dirs, tag=f"tiles {dirs} {io}")


@pytest.mark.parametrize("shift", [-20.0, 20.0])
def test_scan_bwd_step_size_limits(shift):
    """Steps near zero (every decay 1) and large ones (every decay 0)."""
    say(f"scan_bwd shift {shift}")
    inp, dout = make(1, 40, 64, 16, "f32", seed=3, shift=shift)
    dev, g = upload(inp, dout, "f32")
    check_grads(run(dev, g), inp, dout, "f32", 40, tag=f"shift {shift}")


@pytest.mark.parametrize("drop", ["D", "dt_bias"])
def test_scan_bwd_optional_inputs(drop):
    say(f"scan_bwd without {drop}")
    inp, dout = make(2, 50, 64, 16, "f32", seed=6)
    inp[drop] = None
    dev, g = upload(inp, dout, "f32")
    got = run(dev, g)
    assert got[drop] is None
    check_grads(got, inp, dout, "f32", 50, tag=f"no {drop}")


def test_scan_bwd_zero_gradient_and_determinism():
    torch = torch_mod()
    inp, dout = make(2, 130, 256, 16, "bf16", seed=7)
    dev, g = upload(inp, dout, "bf16")
    zero = run(dev, torch.zeros_like(g))
    for k, v in zero.items():
        assert torch.count_nonzero(v) == 0, k
    one, two = run(dev, g), run(dev, g)
    for k in one:
        assert torch.equal(one[k], two[k]), k


def test_scan_bwd_agrees_with_differences_of_the_forward_pass():
    """d/ds loss(inputs + s v) at 0 against the gradients' product with v: central differences of the library's fp32
    forward pass.  v moves every element by its own size along its gradient's sign (so that A stays negative), and with
    h = 2^-6 the combination (4 d(h / 2) - d(h)) / 3 cancels the h^2 term of the truncation: what is left is h^4 / 30 of
    a fifth derivative (2e-9) and the forward pass's rounding, ~1e-6 / 2^-7 ~ 1.3e-4."""
    import bidirectional_mamba_selective_amd as bm

    torch = torch_mod()
    say("scan_bwd against differences")
    inp, dout = make(2, 90, 128, 16, "f32", seed=8)
    dev, g = upload(inp, dout, "f32")
    got = run(dev, g)

    def loss(v):
        out = bm.bimamba_scan_fwd(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["dt_bias"])
        return (out.double() * g.double()).sum().item()

    for k in got:
        v = torch.sign(got[k]) * dev[k].abs()
        want = (got[k].double() * v.double()).sum().item()

        def difference(step):
            hi, lo = (loss(dict(dev, **{k: dev[k] + s * step * v})) for s in (1, -1))
            return (hi - lo) / (2 * step)

        rate = (4 * difference(2.0 ** -7) - difference(2.0 ** -6)) / 3
        say(f"d{k}: difference {rate:.6g}, gradient {want:.6g}")
        assert abs(rate - want) <= 2e-3 * abs(want), k


def test_scan_bwd_layer_shape():
    """The 1.3B layer's width over a ragged length: the channel-wise gradients on a subset of the channels (exact:
    they do not depend on the others), dB and dC against the sum over all of them."""
    import oracle

    torch = torch_mod()
    L, nd, ns = 200, 4096, 16
    say("scan_bwd 4096 channels")
    inp, dout = make(1, L, nd, ns, "bf16", seed=12)
    dev, g = upload(inp, dout, "bf16")
    got = run(dev, g)
    torch.cuda.synchronize()
    want = {"B": 0.0, "C": 0.0}
    for c in np.array_split(np.arange(nd), 16):
        sub = {k: (v[..., c] if k in ("x", "dt", "z") else v[c] if k in VECTORS else v) for k, v in inp.items()}
        w = oracle.scan_bwd(dout[..., c], sub["x"], sub["dt"], sub["A"], sub["B"], sub["C"], sub["D"], sub["z"],
                            sub["dt_bias"])
        for k in ("x", "dt", "z", "A", "D", "dt_bias"):
            o = to_host64(got[k])
            o = o[..., c] if k in ("x", "dt", "z") else o[c]
            err = np.linalg.norm(o - w[k]) / np.linalg.norm(w[k])
            assert err <= (1e-5 if k in VECTORS else 2.5e-3), (k, err)
        for k in want:
            want[k] = want[k] + w[k]
    for k in want:
        err = np.linalg.norm(to_host64(got[k]) - want[k]) / np.linalg.norm(want[k])
        assert err <= 2.5e-3, (k, err)
