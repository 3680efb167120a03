"""GPU parity of the gated delta rule, forward and backward, against the fp64 oracle, through the C ABI.

Bounds: oracle.delta_bounds (derived there from the arithmetic), per (token, head) as 2-norms, plus half a step of bf16,
2^-8 of the value, on each element of a result that is rounded to it."""
import functools

import numpy as np
import pytest

from bidirectional_mamba_selective_amd import inputs
from tests.gpu_util import f32_dev, say, to_dev, to_host64, torch_mod

pytestmark = pytest.mark.gpu

SEQ = ("q", "k", "v", "dt", "b")
HALF = 2.0 ** -8 * 1.01


def make(batch, L, hk, heads, dk, dv, seed=0, state=True, bias=True, **kw):
    """Inputs as numpy arrays, rounded to bf16 where the call takes bf16."""
    r = np.random.default_rng(seed)

    def unit(*shape):
        x = r.standard_normal(shape)
        # 0.99: of unit length at most after the rounding too, as the bounds assume
        return 0.99 * x / np.linalg.norm(x, axis=-1, keepdims=True)

    step = np.exp(r.uniform(np.log(1e-3), np.log(1e-1), heads))
    inp = dict(q=unit(batch, L, hk, dk), k=unit(batch, L, hk, dk), v=r.standard_normal((batch, L, heads, dv)),
               dt=0.5 * r.standard_normal((batch, L, heads)), A=-r.uniform(1.0, 16.0, heads),
               b=r.standard_normal((batch, L, heads)), dt_bias=np.log(np.expm1(step)) if bias else None,
               h_in=0.3 * r.standard_normal((batch, heads, dk, dv)) if state else None)
    inp.update(kw)
    for n in SEQ:
        inp[n] = inputs.round_to(inp[n].astype(np.float32), "bf16")
    for n in ("A", "dt_bias", "h_in"):
        inp[n] = None if inp[n] is None else inp[n].astype(np.float32)
    dout = inputs.round_to(r.standard_normal((batch, L, heads, dv)).astype(np.float32), "bf16")
    dh = (0.1 * r.standard_normal((batch, heads, dk, dv))).astype(np.float32) if state else None
    return inp, dout, dh


def upload(inp):
    return {n: None if x is None else to_dev(x, "bf16") if n in SEQ else f32_dev(x) for n, x in inp.items()}


def close(got, want, bound, tag, bf16=True):
    """Every element within the bound of its (token, head) or (batch, head) and, for bf16, half a step."""
    extra = bound.reshape(bound.shape + (1,) * (want.ndim - bound.ndim))
    allow = (HALF if bf16 else 2.0 ** -22) * np.abs(want) + extra + 1e-30
    worst = float(np.max(np.abs(got - want) / allow)) if want.size else 0.0
    say(f"{tag}: worst element at {worst:.3f} of its bound")
    assert got.shape == want.shape and np.all(np.isfinite(got)) and worst <= 1.0, tag


def run_fwd(bm, dev, rev, **kw):
    torch = torch_mod()
    nb, nh, dk, dv = dev["v"].shape[0], dev["v"].shape[2], dev["q"].shape[3], dev["v"].shape[3]
    h_out = torch.full((nb, nh, dk, dv), float("nan"), device="cuda")
    out = bm.bimamba_delta_fwd(**dev, h_out=h_out, flags=bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY, **kw)
    return out, h_out


def check_fwd(inp, rev=False, tag="", **kw):
    import bidirectional_mamba_selective_amd as bm
    import oracle

    out, h = run_fwd(bm, upload(inp), rev, **kw)
    wout, wh = oracle.delta_fwd(inp, rev=rev)
    r = oracle.delta_bounds(inp, rev=rev)
    close(to_host64(out), wout, r["out"], f"out {tag}")
    close(to_host64(h), wh, r["h_out"], f"h_out {tag}", bf16=False)


def check_bwd(inp, dout, dh, rev=False, tag=""):
    import bidirectional_mamba_selective_amd as bm
    import oracle

    got = bm.bimamba_delta_bwd(to_dev(dout, "bf16"), **upload(inp), dh_out=f32_dev(dh),
                               flags=bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY)
    want = oracle.delta_bwd(dout, inp, dh, rev=rev)
    r = oracle.delta_bounds(inp, dout, dh, rev=rev)
    for n, w in want.items():
        if inp.get(n) is None:
            assert got[n] is None
        else:
            close(to_host64(got[n]), w, r[n], f"d{n} {tag}", bf16=n in SEQ)


LENGTHS = [1, 2, 7, 15, 16, 17, 63, 64, 65, 127, 128, 150, 200]


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("L", LENGTHS)
def test_fwd_lengths(L, rev):
    check_fwd(make(2, L, 1, 2, 128, 128, seed=L)[0], rev, f"L {L}")


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("L", [5, 16, 70, 193])
def test_fwd_head_sizes(dk, dv, L):
    check_fwd(make(1, L, 3, 3, dk, dv, seed=L, bias=False, state=False)[0], L % 2 == 1, f"{dk} x {dv}")


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("L", LENGTHS)
def test_bwd_lengths(L, rev):
    check_bwd(*make(2, L, 1, 2, 128, 128, seed=L), rev, f"L {L}")


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("hk,heads", [(1, 1), (2, 6), (5, 5)])
def test_bwd_heads(dk, dv, hk, heads):
    check_bwd(*make(2, 130, hk, heads, dk, dv, seed=heads, bias=heads != 1, state=heads != 5), heads == 6, f"{hk}/{heads}")


def extreme(name):
    inp, dout, dh = make(1, 140, 2, 2, 64, 64, seed=3)
    if name == "masked":          # padded places and a whole padded sequence's worth of them
        for n in ("dt", "b"):
            inp[n][:, [0, 5, 63, 64, 90, 139]] = -np.inf
            inp[n][:, 100:130, 1] = -np.inf
    elif name == "all_masked":
        inp["dt"][:] = inp["b"][:] = -np.inf
    elif name == "strong_decay":  # every state gone by the next token
        inp["dt"][:] = 60.0
    elif name == "reset":         # single tokens that clear the state, one beyond e^-256
        inp["dt"][:, [20, 64, 65]] = 100.0
    elif name == "no_decay":
        inp["A"][:] = 0.0
    elif name == "same_key":      # the triangular system at its worst: every key the same, beta near 1
        inp["k"][:] = inp["k"][:, :1]
        inp["b"][:] = 12.0
    elif name == "zero_key":
        inp["k"][:, ::3] = 0.0
    elif name == "small_beta":
        inp["b"][:] = -40.0
    elif name == "large_values":
        inp["v"] = inputs.round_to((inp["v"] * 1e4).astype(np.float32), "bf16")
    return inp, dout, dh


EXTREMES = ["masked", "all_masked", "strong_decay", "reset", "no_decay", "same_key", "zero_key", "small_beta",
            "large_values"]


@pytest.mark.parametrize("name", EXTREMES)
def test_fwd_extremes(name):
    inp = extreme(name)[0]
    check_fwd(inp, False, name)
    check_fwd({n: x[:, :12] if n in SEQ else x for n, x in inp.items()}, True, name + ", step")


@pytest.mark.parametrize("name", EXTREMES)
def test_bwd_extremes(name):
    check_bwd(*extreme(name), name in ("reset", "masked"), name)


def test_segments():
    """More chunks than are prepared at a time: the state is carried from one set to the next."""
    import bidirectional_mamba_selective_amd as bm
    import oracle

    inp, _, _ = make(1, 1800, 96, 96, 64, 64, seed=5)
    # two sets of 15 chunks, where 21 are still one
    assert (bm.bimamba_delta_fwd_workspace_bytes(1, 1800, 96, 96, 64, 64)
            < bm.bimamba_delta_fwd_workspace_bytes(1, 1300, 96, 96, 64, 64))
    for rev in (False, True):
        out, h = run_fwd(bm, upload(inp), rev)
        part = {n: x[:, :, ::48] if n in SEQ else x[::48] if x.ndim == 1 else x[:, ::48] for n, x in inp.items()}
        wout, wh = oracle.delta_fwd(part, rev=rev)
        r = oracle.delta_bounds(part, rev=rev)
        close(to_host64(out[:, :, ::48]), wout, r["out"], "out")
        close(to_host64(h[:, ::48]), wh, r["h_out"], "h_out", bf16=False)


@pytest.mark.parametrize("cuts", [(40, 41, 57), (64, 128, 200), (3, 100, 101)])
@pytest.mark.parametrize("rev", [False, True])
def test_blocks_in_place(cuts, rev):
    """A sequence in four calls, the cache updated in place, against the oracle's one."""
    import bidirectional_mamba_selective_amd as bm
    import oracle

    inp, _, _ = make(2, 230, 2, 4, 128, 64, seed=7)
    dev = upload(inp)
    h = dev.pop("h_in").clone()
    edges = [0, *cuts, 230]
    parts = [(a, b) for a, b in zip(edges, edges[1:])]
    outs = {}
    for a, b in reversed(parts) if rev else parts:
        piece = {n: x[:, a:b].contiguous() if n in SEQ else x for n, x in dev.items()}
        outs[a] = bm.bimamba_delta_fwd(**piece, h_in=h, h_out=h, flags=bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY)
    wout, wh = oracle.delta_fwd(inp, rev=rev)
    r = oracle.delta_bounds(inp, rev=rev)
    got = np.concatenate([to_host64(outs[a]) for a, _ in parts], 1)
    close(got, wout, r["out"], "out")
    close(to_host64(h), wh, r["h_out"], "h", bf16=False)


def test_gradient_against_differences_of_the_forward_call():
    """Along one direction per input, on the GPU's own fp32 end state (out is bf16: too coarse to difference)."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    inp, dout, dh = make(1, 90, 1, 2, 64, 64, seed=11)
    dev = upload(inp)
    dh = f32_dev(dh)
    g = bm.bimamba_delta_bwd(torch.zeros_like(dev["v"]), **dev, dh_out=dh)
    for n in ("A", "dt_bias", "h_in"):
        d = torch.randn(dev[n].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(2)) * dev[n].abs()
        vals = []
        for s in (2.0 ** -6, -(2.0 ** -6)):
            h = run_fwd(bm, {**dev, n: dev[n] + s * d}, False)[1]
            vals.append((h.double() * dh.double()).sum().item())
        num, want = (vals[0] - vals[1]) * 2.0 ** 5, (g[n].double() * d.double()).sum().item()
        # the third derivative's share: steps of 2^-6 relative leave 2^-12 of the terms
        size = (g[n].double() * d.double()).abs().sum().item()
        assert abs(num - want) <= 2.0 ** -9 * size + 1e-5, (n, num, want)


def test_same_bits_used_workspace_and_guarded_buffers():
    """Two calls give the same bits; what the workspace held and what lies around the results does not matter."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    inp, dout, dh = make(2, 200, 1, 3, 128, 128, seed=13)
    dev, dout, dh = upload(inp), to_dev(dout, "bf16"), f32_dev(dh)
    shape = (2, 200, 1, 3, 128, 128)
    first = run_fwd(bm, dev, True)
    gfirst = bm.bimamba_delta_bwd(dout, **dev, dh_out=dh, flags=bm.FLAG_REV_ONLY)
    ws = torch.full((bm.bimamba_delta_fwd_workspace_bytes(*shape) // 4,), float("nan"), device="cuda")
    bws = torch.full((bm.bimamba_delta_bwd_workspace_bytes(*shape) // 4,), float("nan"), device="cuda")
    pads, views = {}, {}
    for n, t in {**{n: dev[n] for n in SEQ}, "A": dev["A"], "dt_bias": dev["dt_bias"], "h_in": dev["h_in"]}.items():
        pads[n] = torch.full((t.numel() + 128,), 7.0, dtype=t.dtype, device="cuda")
        views[n] = pads[n][64:64 + t.numel()].view(t.shape)
    again = run_fwd(bm, dev, True, workspace=ws)
    g = bm.bimamba_delta_bwd(dout, **dev, dh_out=dh, flags=bm.FLAG_REV_ONLY, workspace=bws, grads=views)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    for n in views:
        assert torch.equal(g[n], gfirst[n]), n
        assert bool((pads[n][:64] == 7).all()) and bool((pads[n][-64:] == 7).all()), n


def test_rows_behind_the_batch_stay():
    """out, the last of it inside a larger buffer: a partial last run writes nothing past its tokens."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    for L in (9, 70):
        dev = upload(make(1, L, 2, 2, 64, 64, seed=L)[0])
        buf = torch.full((1, L + 64, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        for rev in (False, True):
            run_fwd(bm, dev, rev, out=buf[:, :L])
            assert bool((buf[:, L:] == 5).all())


def test_graphs_streams_and_two_captures_with_one_workspace():
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    sets = [make(1, L, 1, 2, 128, 128, seed=L) for L in (100, 12)]
    devs = [(upload(i), to_dev(o, "bf16"), f32_dev(h)) for i, o, h in sets]
    ws = torch.empty(max(max(bm.bimamba_delta_bwd_workspace_bytes(1, L, 1, 2, 128, 128),
                             bm.bimamba_delta_fwd_workspace_bytes(1, L, 1, 2, 128, 128)) for L in (100, 12)),
                     dtype=torch.uint8, device="cuda")
    want = []
    for d, o, h in devs:
        want.append((run_fwd(bm, d, False), bm.bimamba_delta_bwd(o, **d, dh_out=h)))
    torch.cuda.synchronize()
    graphs = []
    for d, o, h in devs:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            run_fwd(bm, d, False, workspace=ws)
            bm.bimamba_delta_bwd(o, **d, dh_out=h, workspace=ws)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got = (run_fwd(bm, d, False, workspace=ws), bm.bimamba_delta_bwd(o, **d, dh_out=h, workspace=ws))
        graphs.append((gr, got))
    for turn in range(3):
        for (gr, got), w in zip(graphs, want):  # one after the other: they share the workspace
            for t in got[0]:
                t.zero_()
            gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got[0], w[0])), turn
            assert all(torch.equal(got[1][n], w[1][n]) for n in w[1]), turn
        ws.random_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = bm.bimamba_delta_fwd(**devs[0][0], stream=s)
    s.synchronize()
    assert torch.equal(out, want[0][0][0])


def test_non_finite_values_stay_in_their_head():
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    inp, dout, dh = make(2, 150, 2, 4, 64, 64, seed=17)
    clean = upload(inp)
    bad = {n: None if x is None else x.clone() for n, x in clean.items()}
    bad["v"][0, 80, 1, 5] = float("nan")
    bad["b"][1, 3, 2] = float("nan")
    (o, h), (co, ch) = run_fwd(bm, bad, False), run_fwd(bm, clean, False)
    for b, hd in ((0, 1), (1, 2)):
        assert bool(torch.isnan(h[b, hd]).any())
        o[b, :, hd], co[b, :, hd], h[b, hd], ch[b, hd] = 0, 0, 0, 0
    assert torch.equal(o, co) and torch.equal(h, ch)


def test_refusals():
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    inp, dout, dh = make(1, 20, 2, 4, 64, 64)
    d, dout = upload(inp), to_dev(dout, "bf16")
    fwd = functools.partial(bm.bimamba_delta_fwd)
    for bad in (dict(q=d["q"][:, :, :1]), dict(A=d["A"].double()), dict(v=d["v"].transpose(2, 3)),
                dict(h_in=d["h_in"][:, :2]), dict(out=d["v"].float()), dict(k=d["k"].cpu())):
        with pytest.raises((ValueError, TypeError)):
            fwd(**{**d, **bad})
    for bad in (dict(flags=0), dict(flags=bm.FLAG_FWD_ONLY | bm.FLAG_REV_ONLY), dict(scale=float("inf")),
                dict(out=d["v"]), dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(bm.BimambaError):
            fwd(**{**d, **bad})
    with pytest.raises(bm.BimambaError):  # fp32 activations
        fwd(**{n: None if x is None else x.float() for n, x in d.items()})
    with pytest.raises(ValueError):
        bm.bimamba_delta_bwd(dout, **{**d, "dt_bias": None}, grads={"dt_bias": d["dt_bias"].clone()})
    with pytest.raises(bm.BimambaError):
        bm.bimamba_delta_bwd(dout, **d, grads={"q": d["q"]})
