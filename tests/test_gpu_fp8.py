"""GPU parity of the 8-bit norm and of the product that reads it against fp64 references.

Bounds.  adaln_fwd_fp8: a scale is the largest magnitude of a block over 448, off by at most what the norm's value is (100
roundings of 2^-24 of its terms' magnitudes, as in the tests of bimamba_adaln_fwd) and three roundings; a value is off by that and by half a step
of e4m3: 2^-4 of it, or 2^-10 scales below the smallest normal number.  proj_fp8: fp32 results sum exact products, d_in roundings
of 2^-24 of the magnitudes at most; bf16 results half a step, 2^-8, and what the 8-bit matrix instruction drops, below
2^-12 of the magnitudes (2^-12.9 measured on single sums of 128 products of arbitrary e4m3 values)."""
import numpy as np
import pytest

from bidirectional_mamba_selective_amd import inputs
from tests.gpu_util import f32_dev, say, to_dev, to_host64, torch_mod

pytestmark = pytest.mark.gpu

EPS, U = 1e-5, 2.0 ** -24


def make_rows(batch, L, d, io, seed=0, shared=False, scale=3.0):
    r = np.random.default_rng(seed)
    rows = 1 if shared else batch
    act = lambda m, s: inputs.round_to((m + s * r.standard_normal((batch, L, d))).astype(np.float32), io)  # noqa: E731
    vec = lambda n, m, s: (m + s * r.standard_normal((n, d))).astype(np.float32)  # noqa: E731
    return dict(x=act(0.3, scale), branch=act(0.1, 1.5), gamma=vec(rows, 1, 0.3), beta=vec(rows, 0, 0.3),
                gate=vec(rows, 0.5, 0.4), post_weight=vec(1, 1, 0.3)[0])


def upload(inp, io):
    return {k: None if v is None else to_dev(v, io) if k in ("x", "branch") else f32_dev(v) for k, v in inp.items()}


def check_norm(inp, io, rms, **kw):
    import bidirectional_mamba_selective_amd as bm
    import oracle

    dev = upload(inp, io)
    flags = bm.FLAG_RMS_NORM if rms else 0
    h, out, scales = bm.bimamba_adaln_fwd_fp8(**dev, eps=EPS, flags=flags, **kw)
    wh, wout = oracle.adaln_fwd(**inp, eps=EPS, rms=rms)
    if inp["branch"] is not None:  # h as bimamba_adaln_fwd's, bit for bit
        assert torch_mod().equal(h, bm.bimamba_adaln_fwd(**upload(inp, io), eps=EPS, flags=flags)[0])
    mag = np.abs(inp["x"].astype(np.float64)) + np.abs(wh)
    c = wh if rms else wh - wh.mean(-1, keepdims=True)
    rs = 1 / np.sqrt(np.mean(c * c, -1, keepdims=True) + EPS)
    mod = lambda n: 1.0 if inp[n] is None else np.abs(inp[n].astype(np.float64))[:, None]  # noqa: E731
    cm = mag if rms else mag + mag.mean(-1, keepdims=True)
    spread = np.sqrt(np.mean(cm * cm, -1, keepdims=True)) * rs
    off = 100 * U * (mod("gamma") * rs * (cm + np.abs(c) * spread) + (0 if inp["beta"] is None else mod("beta")))
    off = np.broadcast_to(off, wout.shape)
    blocks = lambda v: v.reshape(*v.shape[:2], -1, 128)  # noqa: E731
    wscale = np.maximum(np.abs(blocks(wout)).max(-1), 2.0 ** -100) / 448
    s, q = to_host64(scales), to_host64(out)
    assert np.all(np.abs(s - wscale) <= blocks(off).max(-1) / 448 + 4 * U * wscale)
    step = np.repeat(s, 128, -1)
    allow = 2.0 ** -4 * np.abs(wout) * (1 + 1e-5) + 2.0 ** -10 * step * (1 + 1e-5) + 2 * off
    worst = float(np.max(np.abs(q * step - wout) / allow))
    say(f"{io} {'rms' if rms else 'layer'} {wout.shape}: worst value at {worst:.3f} of its bound")
    assert worst <= 1.0 and np.all(np.abs(q) <= 448)
    # a block's largest magnitude is 448 scales: none of the range is given away
    assert np.all(blocks(np.abs(q)).max(-1) == np.where(np.abs(blocks(wout)).max(-1) > 2.0 ** -99, 448, blocks(np.abs(q)).max(-1)))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 256, 384, 512, 1920, 2048, 4096, 8192])
def test_norm_widths(d, io):
    inp = make_rows(2, 5, d, io, seed=d)
    check_norm(inp, io, rms=d % 512 == 0)


@pytest.mark.parametrize("drop", [("branch", "gate", "post_weight"), ("gate",), ("post_weight", "beta"), ("gamma", "beta")])
@pytest.mark.parametrize("rms", [False, True])
def test_norm_options(drop, rms):
    inp = make_rows(3, 67, 640, "bf16", seed=len(drop), shared=rms)
    check_norm({**inp, **{n: None for n in drop}}, "bf16", rms)


def test_norm_of_rows_of_zeros_and_tiny_rows():
    inp = make_rows(1, 6, 256, "f32", seed=2)
    for n in ("beta", "branch", "gate", "post_weight"):
        inp[n] = None
    inp["x"][0, 1] = 0
    inp["x"][0, 2, :128] = 0
    inp["x"][0, 3] *= 1e-20
    check_norm(inp, "f32", True)


def test_norm_in_place_nan_and_determinism():
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    inp = make_rows(2, 9, 384, "bf16", seed=4)
    dev = upload(inp, "bf16")
    want = bm.bimamba_adaln_fwd_fp8(**dev)
    x = dev["x"].clone()
    got = bm.bimamba_adaln_fwd_fp8(**{**dev, "x": x}, h=x)
    assert got[0] is x and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    dev["x"][1, 4, 7] = float("nan")
    _, out, scales = bm.bimamba_adaln_fwd_fp8(**dev)
    bad = torch.isnan(out.float()).all(-1)
    assert bad.sum() == 1 and bool(bad[1, 4]) and not bool(torch.isnan(out.float()[~bad]).any())
    keep = ~bad
    assert torch.equal(scales[keep], want[2][keep])


def e4m3_values(shape, r, scale=1.0):
    torch = torch_mod()
    return (torch.from_numpy(r.standard_normal(shape).astype(np.float32)) * scale).clamp(-448, 448).to(torch.float8_e4m3fn)


def make_proj(m, n, k, seed=0, values="normal"):
    torch = torch_mod()
    r = np.random.default_rng(seed)
    if values == "any":  # every e4m3 pattern that is a number
        bits = lambda shape: torch.from_numpy((r.integers(0, 127, shape) + 128 * r.integers(0, 2, shape)).astype(np.uint8)).view(torch.float8_e4m3fn)  # noqa: E731,E501
        x, w = bits((1, m, k)), bits((n, k))
    else:
        x, w = e4m3_values((1, m, k), r, 120.0), e4m3_values((n, k), r, 120.0)
    xs = torch.from_numpy(np.exp(r.uniform(-6, 2, (1, m, k // 128))).astype(np.float32))
    ws = torch.from_numpy(np.exp(r.uniform(-6, 2, ((n + 127) // 128, k // 128))).astype(np.float32))
    return x, xs, w, ws


def check_proj(m, n, k, dtype, seed=0, values="normal", **kw):
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    t = make_proj(m, n, k, seed, values)
    got = bm.bimamba_proj_fp8(*[v.cuda() for v in t], out_dtype=dtype, **kw)
    x, xs, w, ws = (v.double().numpy() for v in t)
    x = x[0] * np.repeat(xs[0], 128, 1)
    w = w * np.repeat(np.repeat(ws, 128, 0)[:n], 128, 1)
    want, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    bf16 = dtype == torch.bfloat16
    allow = (2.0 ** -8 * 1.01 * np.abs(want) + 2.0 ** -12 * mag) if bf16 else 2.0 ** -24 * np.abs(want) + (k + 8) * U * mag
    worst = float(np.max(np.abs(to_host64(got)[0] - want) / (allow + 1e-30)))
    say(f"{m} x {n} x {k} {dtype} {values}: worst element at {worst:.3f} of its bound")
    assert got.shape == (1, m, n) and got.dtype == dtype and worst <= 1.0


SHAPES = [(1, 8, 128), (1, 1920, 3840), (3, 136, 256), (15, 24, 384), (16, 8056, 1920), (17, 200, 640), (32, 264, 128),
          (33, 1000, 1152), (63, 128, 256), (64, 72, 512), (65, 8, 128), (100, 264, 384), (129, 136, 1920), (257, 520, 256),
          (1000, 1096, 640)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_proj_shapes(m, n, k):
    torch = torch_mod()
    check_proj(m, n, k, torch.bfloat16, seed=m)
    check_proj(m, n, k, torch.float32, seed=m + 1)


@pytest.mark.parametrize("m,n,k", [(2000, 2056, 384), (4000, 2056, 128), (2049, 4104, 384), (8200, 4096, 256)])
def test_proj_large_tiles(m, n, k):
    """The tiles of 128 and 256 rows, with ragged edges and an odd and an even number of blocks."""
    torch = torch_mod()
    check_proj(m, n, k, torch.bfloat16)
    check_proj(m, n, k, torch.float32)


@pytest.mark.parametrize("m", [5, 200])
def test_proj_any_values(m):
    torch = torch_mod()
    for dtype in (torch.bfloat16, torch.float32):
        check_proj(m, 256, 512, dtype, values="any")


def test_proj_rows_apart_nan_and_used_buffers():
    """A row's NaN stays in its row and a weight's in its output, whatever out held; nothing is written past its rows."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    for m in (6, 70, 300):
        t = [v.cuda() for v in make_proj(m, 136, 384)]
        want = bm.bimamba_proj_fp8(*t)
        t[0].view(torch.uint8)[0, 3, 200] = 0x7F
        t[2].view(torch.uint8)[130, 5] = 0xFF
        buf = torch.full((1, m + 80, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
        buf[:, m:] = 3
        got = bm.bimamba_proj_fp8(*t, out=buf[:, :m])
        assert bool(torch.isnan(got[0, 3]).all()) and bool(torch.isnan(got[0, :, 130]).all()) and bool((buf[:, m:] == 3).all())
        got[0, 3], got[0, :, 130] = want[0, 3], want[0, :, 130]
        assert torch.equal(got, want)


def test_block_in_8_bits():
    """A block as it is served: norm, projection, short convolution, delta rule, norm, projection, against the chained
    references, and once more through a graph."""
    import bidirectional_mamba_selective_amd as bm
    import oracle
    torch = torch_mod()

    gen = torch.Generator("cuda").manual_seed(3)
    rnd = lambda *s, k=1.0: torch.randn(*s, generator=gen, device="cuda") * k  # noqa: E731
    nb, L, d, hk, nh, hd = 2, 100, 256, 2, 4, 64
    width = 2 * hk * hd + nh * hd
    x = rnd(nb, L, d, k=2.0).bfloat16()

    def quantise(w):
        n, k = w.shape
        pad = torch.zeros(-(-n // 128) * 128, k, device="cuda")
        pad[:n] = w
        s = pad.view(-1, 128, k // 128, 128).abs().amax((1, 3)) / 448
        return (pad / s.repeat_interleave(128, 0).repeat_interleave(128, 1))[:n].to(torch.float8_e4m3fn), s

    w1, s1 = quantise(rnd(width + 2 * nh, d, k=d ** -0.5))
    w2, s2 = quantise(rnd(d, nh * hd, k=(nh * hd) ** -0.5))
    gamma, cw, A = 1 + 0.2 * rnd(1, d), rnd(width, 4, k=0.5), -1 - 15 * torch.rand(nh, generator=gen, device="cuda")
    flags = bm.FLAG_RMS_NORM

    def run():
        _, u, us = bm.bimamba_adaln_fwd_fp8(x, gamma, flags=flags)
        p = bm.bimamba_proj_fp8(u, us, w1, s1)
        c, _ = bm.bimamba_conv1d_bidir(p[..., :width].contiguous(), cw)
        q, k, v = c.split([hk * hd, hk * hd, nh * hd], -1)
        unit = lambda t: torch.nn.functional.normalize(t.float().view(nb, L, hk, hd), dim=-1).bfloat16()  # noqa: E731
        q, k, v = unit(q), unit(k), v.reshape(nb, L, nh, hd).contiguous()
        dt, b = (p[..., width + i * nh:width + (i + 1) * nh].contiguous() for i in (0, 1))
        o = bm.bimamba_delta_fwd(q, k, v, dt, A, b)
        _, y, ys = bm.bimamba_adaln_fwd_fp8(o.view(nb, L, nh * hd), flags=flags)
        return dict(u=u, us=us, p=p, c=c, q=q, k=k, v=v, dt=dt, b=b, o=o, y=y, ys=ys, out=bm.bimamba_proj_fp8(y, ys, w2, s2))

    r = run()
    f = {n: to_host64(t) for n, t in r.items()}
    spread = lambda s, n: np.repeat(np.repeat(to_host64(s), 128, 0)[:n], 128, 1)  # noqa: E731
    rel = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)  # noqa: E731
    # each step on what the one before it gave: its own rounding, and 2^-5 for 8-bit values (half a step at most, 2^-4)
    _, wu = oracle.adaln_fwd(to_host64(x), to_host64(gamma), rms=True)
    assert rel(f["u"] * np.repeat(f["us"], 128, -1), wu) < 2.0 ** -5
    p = (f["u"] * np.repeat(f["us"], 128, -1)) @ (to_host64(w1) * spread(s1, w1.shape[0])).T
    assert rel(f["p"], p) < 2.0 ** -8
    c = oracle.conv_causal(f["p"][..., :width], to_host64(cw), None)
    assert rel(f["c"], c) < 2.0 ** -8
    o, _ = oracle.delta_fwd({n: f[n] for n in ("q", "k", "v", "dt", "b")} | {"A": to_host64(A)})
    assert rel(f["o"], o) < 2.0 ** -8
    _, wy = oracle.adaln_fwd(f["o"].reshape(nb, L, -1), rms=True)
    assert rel(f["y"] * np.repeat(f["ys"], 128, -1), wy) < 2.0 ** -5
    out = (f["y"] * np.repeat(f["ys"], 128, -1)) @ (to_host64(w2) * spread(s2, d)).T
    assert rel(f["out"], out) < 2.0 ** -8

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = run()
    for _ in range(3):
        again["out"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again["out"], r["out"])
        rnd(1 << 20)


def test_refusals():
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    x, xs, w, ws = (v.cuda() for v in make_proj(4, 136, 256))
    for bad in (dict(x=x.float()), dict(x_scales=xs[..., :1]), dict(w_scales=ws[:1]), dict(w=w.t()), dict(x=x[0]),
                dict(out=torch.empty(1, 4, 128, device="cuda")), dict(out_dtype=torch.float16)):
        with pytest.raises((ValueError, TypeError)):
            bm.bimamba_proj_fp8(**{**dict(x=x, x_scales=xs, w=w, w_scales=ws), **bad})
    with pytest.raises(bm.BimambaError):  # outputs in sevens
        bm.bimamba_proj_fp8(x, xs, w[:7], ws[:1])
    inp = upload(make_rows(1, 3, 192, "bf16"), "bf16")
    with pytest.raises(bm.BimambaError):  # a block and a half of columns
        bm.bimamba_adaln_fwd_fp8(**inp)
    inp = upload(make_rows(1, 3, 256, "bf16"), "bf16")
    for bad in (dict(out=torch.empty(1, 3, 256, device="cuda")), dict(scales=torch.empty(1, 3, 3, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            bm.bimamba_adaln_fwd_fp8(**inp, **bad)
