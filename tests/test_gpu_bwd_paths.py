"""The backward and norm entry points as a program uses them: together through one block of the denoiser, captured into
HIP graphs, on several streams at once, with a used workspace, into the caller's buffers, and on tensors past 4 GiB."""
import numpy as np
import pytest

from bidirectional_mamba_selective_amd import inputs
from tests.gpu_util import f32_dev, say, to_host64, torch_mod

pytestmark = pytest.mark.gpu


def scan_inputs(torch, gen, nb, L, nd, ns, io):
    def n(*shape, dtype=io, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    f32 = torch.float32
    return dict(dout=n(nb, L, nd), x=n(nb, L, nd), dt=n(nb, L, nd, scale=0.5),
                A=-torch.exp(n(nd, ns, dtype=f32, scale=0.5)), B=n(nb, L, ns), C=n(nb, L, ns), D=n(nd, dtype=f32),
                z=n(nb, L, nd), dt_bias=n(nd, dtype=f32) - 4)


def conv_inputs(torch, gen, nb, L, nc, io):
    def n(*shape, dtype=io):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    f32 = torch.float32
    return dict(dout_f=n(nb, L, nc), dout_r=n(nb, L, nc), u=n(nb, L, nc), w_f=n(nc, 4, dtype=f32),
                b_f=n(nc, dtype=f32), w_r=n(nc, 4, dtype=f32), b_r=n(nc, dtype=f32))


def adaln_inputs(torch, gen, nb, L, nd, io, fwd):
    def n(*shape, dtype=io):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    f32 = torch.float32
    p = dict(gamma=n(nb, nd, dtype=f32), beta=n(nb, nd, dtype=f32), branch=n(nb, L, nd), post_weight=n(nd, dtype=f32),
             gate=n(nb, nd, dtype=f32))
    return dict(x=n(nb, L, nd), **p) if fwd else dict(dout=n(nb, L, nd), dres=n(nb, L, nd), h=n(nb, L, nd), **p)


CASES = {
    "scan": lambda t, g, io: scan_inputs(t, g, 2, 333, 256, 16, io),
    "scan_long": lambda t, g, io: scan_inputs(t, g, 16, 300, 1024, 5, io),  # several tiles a chunk
    "conv": lambda t, g, io: conv_inputs(t, g, 2, 700, 260, io),
    "adaln_fwd": lambda t, g, io: adaln_inputs(t, g, 3, 100, 1032, io, True),
    "adaln_bwd": lambda t, g, io: adaln_inputs(t, g, 3, 400, 1032, io, False),
}


def call(name, v, **kw):
    import bidirectional_mamba_selective_amd as bm

    f = {"scan": bm.bimamba_scan_bwd, "scan_long": bm.bimamba_scan_bwd, "conv": bm.bimamba_conv1d_bidir_bwd,
         "adaln_fwd": bm.bimamba_adaln_fwd, "adaln_bwd": bm.bimamba_adaln_bwd}[name]
    r = f(**v, **kw)
    return dict(zip(("h", "out"), r)) if isinstance(r, tuple) else r


def workspace_bytes(name, v):
    import bidirectional_mamba_selective_amd as bm

    if name.startswith("scan"):
        return bm.bimamba_scan_bwd_workspace_bytes(*v["x"].shape, v["A"].shape[1])
    if name == "conv":
        return bm.bimamba_conv1d_bidir_bwd_workspace_bytes(*v["u"].shape)
    return bm.bimamba_adaln_bwd_workspace_bytes(*v["h"].shape)


def same(torch, a, b, tag):
    for k in a:
        assert (a[k] is None) == (b[k] is None) and (a[k] is None or torch.equal(a[k], b[k])), (tag, k)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["scan", "scan_long", "conv", "adaln_bwd"])
def test_workspace_contents_do_not_matter(name, io):
    """A workspace of NaNs, and one that another call has used, give the same bits."""
    torch = torch_mod()
    say(f"used workspace {name} {io}")
    v = CASES[name](torch, torch.Generator("cuda").manual_seed(1), {"f32": torch.float32, "bf16": torch.bfloat16}[io])
    want = call(name, v)
    n = workspace_bytes(name, v)
    ws = torch.full(((n + 3) // 4,), float("nan"), device="cuda")
    for i in range(2):
        same(torch, want, call(name, v, workspace=ws), f"{name} {i}")
    assert all(torch.isfinite(t).all() for t in want.values() if t is not None)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["scan", "conv", "adaln_fwd", "adaln_bwd"])
def test_results_stay_in_the_callers_buffers(name, io):
    """Every output written into the middle of a larger buffer: the values around it are left as they were."""
    torch = torch_mod()
    say(f"buffers {name} {io}")
    v = CASES[name](torch, torch.Generator("cuda").manual_seed(2), {"f32": torch.float32, "bf16": torch.bfloat16}[io])
    want = call(name, v)
    pads, outs = {}, {}
    for k, t in want.items():
        if t is None:
            continue
        pads[k] = torch.full((t.numel() + 4096,), 7.0, dtype=t.dtype, device="cuda")
        outs[k] = pads[k][2048:2048 + t.numel()].view(t.shape)
    got = call(name, v, **(outs if name == "adaln_fwd" else {"grads": outs}))
    for k in outs:
        assert got[k] is outs[k] and torch.equal(got[k], want[k]), k
        assert (pads[k][:2048] == 7).all() and (pads[k][2048 + want[k].numel():] == 7).all(), k


@pytest.mark.parametrize("name", sorted(CASES))
def test_captured_and_replayed(name):
    """One capture, three replays on new inputs copied into the captured tensors with eager work between: each equals the
    eager call bit for bit."""
    torch = torch_mod()
    say(f"graph {name}")
    gen = torch.Generator("cuda").manual_seed(3)
    v = CASES[name](torch, gen, torch.bfloat16)
    call(name, v)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(name, v)
    for i in range(3):
        new = CASES[name](torch, gen, torch.bfloat16)
        for k in v:
            v[k].copy_(new[k])
        g.replay()
        torch.cuda.synchronize()
        same(torch, call(name, new), out, f"{name} replay {i}")
        torch.cuda.synchronize()


def test_two_graphs_with_their_own_workspaces():
    """Two captured calls whose workspaces come from their graphs' own pools, replayed in turn on two streams."""
    torch = torch_mod()
    say("two graphs")
    gen = torch.Generator("cuda").manual_seed(4)
    vs = [CASES["scan"](torch, gen, torch.bfloat16) for _ in range(2)]
    want = [call("scan", v) for v in vs]
    graphs, outs = [], []
    for v in vs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call("scan", v))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in vs]
    torch.cuda.synchronize()
    for i in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            same(torch, w, o, f"replay {i}")


def test_calls_on_several_streams_at_once():
    torch = torch_mod()
    say("streams")
    gen = torch.Generator("cuda").manual_seed(5)
    vs = {n: CASES[n](torch, gen, torch.bfloat16) for n in sorted(CASES)}
    want = {n: call(n, v) for n, v in vs.items()}
    torch.cuda.synchronize()
    streams = {n: torch.cuda.Stream() for n in vs}
    for i in range(3):
        got = {n: call(n, v, stream=streams[n]) for n, v in vs.items()}
        # the default stream allocates and fills blocks of the same sizes meanwhile
        junk = [torch.full_like(t, 3.0) for w in want.values() for t in w.values() if t is not None]
        torch.cuda.synchronize()
        del junk
        for n in vs:
            same(torch, want[n], got[n], f"{n} round {i}")


def test_a_bad_sequence_leaves_the_others_alone():
    """An infinity in one sequence's inputs does not reach another sequence's gradients."""
    torch = torch_mod()
    for name, key in (("scan", "x"), ("conv", "u"), ("adaln_bwd", "h")):
        v = CASES[name](torch, torch.Generator("cuda").manual_seed(6), torch.float32)
        want = call(name, v)
        v[key] = v[key].clone()
        v[key][0, 50, 3] = float("inf")
        got = call(name, v)
        for k, t in want.items():
            if t.dim() == 3:
                assert torch.equal(t[1:], got[k][1:]), (name, k)


def test_one_block_forward_and_backward():
    """A whole block in fp32: norm, short convolution, both untied scans, and the gated residual sum with its post-norm
    and the next norm; then its gradients in reverse order, against the same chain of fp64 oracles.  Each of the six
    calls carries at most ~1e-5 normwise (its own tests), gains of the chain below 3: held to 1e-4."""
    import bidirectional_mamba_selective_amd as bm
    import oracle

    torch = torch_mod()
    say("one block")
    nb, L, d, ns = 2, 90, 128, 8
    r = np.random.default_rng(7)
    n = lambda *s: r.standard_normal(s).astype(np.float32)  # noqa: E731
    x, dout, dres = n(nb, L, d), n(nb, L, d), n(nb, L, d)
    n1 = dict(gamma=1 + 0.2 * n(nb, d), beta=0.2 * n(nb, d))
    cv = dict(w_f=0.5 * n(d, 4), b_f=0.1 * n(d), w_r=0.5 * n(d, 4), b_r=0.1 * n(d))
    A, _, bias = inputs.make_params(d, ns, a_jitter=0.3)
    sets = [dict(dt=0.5 * n(nb, L, d), A=A, B=n(nb, L, ns), C=n(nb, L, ns), D=n(d), z=n(nb, L, d), dt_bias=bias)
            for _ in range(2)]
    n2 = dict(gamma=1 + 0.2 * n(nb, d), beta=0.2 * n(nb, d), post_weight=1 + 0.2 * n(d), gate=0.5 + 0.3 * n(nb, d))

    # oracle
    _, u = oracle.adaln_fwd(x, **n1)
    cf, cr = oracle.conv_bidir(u, cv["w_f"], cv["b_f"], cv["w_r"], cv["b_r"])
    of, orr = oracle.scan_fwd_untied(dict(x=cf, **sets[0]), dict(x=cr, **sets[1]))
    h, out = oracle.adaln_fwd(x, branch=of + orr, **n2)
    g2 = oracle.adaln_bwd(dout, dres, h, branch=of + orr, **n2)
    gf = oracle.scan_bwd(g2["branch"], cf, **sets[0], rev=False)
    gr = oracle.scan_bwd(g2["branch"], cr, **sets[1], fwd=False)
    gc = oracle.conv_bwd(gf["x"], gr["x"], u, **cv)
    g1 = oracle.adaln_bwd(gc["u"], g2["x"], x, **n1)

    # library
    dev = lambda v: {k: f32_dev(a) for k, a in v.items()}  # noqa: E731
    X, N1, CV, S, N2 = f32_dev(x), dev(n1), dev(cv), [dev(s) for s in sets], dev(n2)
    _, U = bm.bimamba_adaln_fwd(X, **N1)
    CF, CR = bm.bimamba_conv1d_bidir(U, **CV)
    OF, OR = bm.bimamba_scan_fwd_untied(dict(x=CF, **S[0]), dict(x=CR, **S[1]))
    M = OF + OR
    H, OUT = bm.bimamba_adaln_fwd(X, branch=M, **N2)
    G2 = bm.bimamba_adaln_bwd(f32_dev(dout), f32_dev(dres), H, branch=M, **N2)
    GF = bm.bimamba_scan_bwd(G2["branch"], CF, **S[0], flags=bm.FLAG_FWD_ONLY)
    GR = bm.bimamba_scan_bwd(G2["branch"], CR, **S[1], flags=bm.FLAG_REV_ONLY)
    GC = bm.bimamba_conv1d_bidir_bwd(GF["x"], GR["x"], U, **CV)
    G1 = bm.bimamba_adaln_bwd(GC["u"], G2["x"], X, **N1)
    torch.cuda.synchronize()
    for tag, got, want in (("out", {"h": H, "out": OUT}, {"h": h, "out": out}), ("norm 2", G2, g2), ("forward", GF, gf),
                           ("reverse", GR, gr), ("conv", GC, gc), ("norm 1", G1, g1)):
        for k, t in got.items():
            if t is None:
                continue
            err = np.linalg.norm(to_host64(t) - want[k]) / np.linalg.norm(want[k])
            say(f"{tag} {k}: {err:.2e}")
            assert err <= 1e-4, (tag, k)


def test_untied_gradients_are_two_one_direction_calls():
    """With one set for both directions the two one-direction gradients add up to the tied call's (fp32 roundings of
    either: 1e-5 normwise)."""
    import bidirectional_mamba_selective_amd as bm

    torch = torch_mod()
    v = scan_inputs(torch, torch.Generator("cuda").manual_seed(8), 2, 120, 128, 16, torch.float32)
    both = bm.bimamba_scan_bwd(**v)
    f, r = (bm.bimamba_scan_bwd(**v, flags=k) for k in (bm.FLAG_FWD_ONLY, bm.FLAG_REV_ONLY))
    for k, t in both.items():
        assert ((f[k].double() + r[k].double()) - t.double()).norm() <= 1e-5 * t.double().norm(), k


def test_bindings_refuse_what_does_not_fit():
    import bidirectional_mamba_selective_amd as bm

    torch = torch_mod()
    gen = torch.Generator("cuda").manual_seed(9)
    s, c, a = (CASES[k](torch, gen, torch.bfloat16) for k in ("scan", "conv", "adaln_bwd"))
    f = CASES["adaln_fwd"](torch, gen, torch.bfloat16)
    bad = [
        (bm.bimamba_scan_bwd, dict(s, dout=None)),
        (bm.bimamba_scan_bwd, dict(s, dout=s["dout"][:, 1:])),
        (bm.bimamba_scan_bwd, dict(s, dout=s["dout"].float())),
        (bm.bimamba_scan_bwd, dict(s, x=s["x"].transpose(0, 1))),
        (bm.bimamba_scan_bwd, dict(s, z=None)),
        (bm.bimamba_scan_bwd, dict(s, flags=bm.FLAG_NO_GATE, grads={"z": s["z"].clone()})),
        (bm.bimamba_scan_bwd, dict(s, grads={"x": s["x"]})),  # over an input
        (bm.bimamba_scan_bwd, dict(s, grads={"y": s["x"].clone()})),
        (bm.bimamba_scan_bwd, dict(s, workspace=torch.empty(16, device="cuda"))),
        (bm.bimamba_scan_bwd, dict(s, workspace=torch.empty(1 << 20))),
        (bm.bimamba_conv1d_bidir_bwd, dict(c, dout_f=None)),
        (bm.bimamba_conv1d_bidir_bwd, dict(c, w_r=None)),
        (bm.bimamba_conv1d_bidir_bwd, dict(c, dout_r=c["dout_r"][:1])),
        (bm.bimamba_conv1d_bidir_bwd, dict(c, w_f=c["w_f"][:, :3].contiguous())),
        (bm.bimamba_adaln_bwd, dict(a, gate=a["gate"][:2])),
        (bm.bimamba_adaln_bwd, dict(a, dout=None)),
        (bm.bimamba_adaln_bwd, dict(a, branch=None)),
        (bm.bimamba_adaln_bwd, dict(a, eps=0.0)),
        (bm.bimamba_adaln_fwd, dict(f, gamma=f["gamma"].bfloat16())),
        (bm.bimamba_adaln_fwd, dict(f, gamma=f["gamma"][:1])),  # one row beside one per sequence
        (bm.bimamba_adaln_fwd, dict(f, out=f["x"])),
        (bm.bimamba_adaln_fwd, dict(f, branch=None)),
    ]
    for i, (fn, kw) in enumerate(bad):
        with pytest.raises((ValueError, TypeError, bm.BimambaError)):
            fn(**kw)
            raise AssertionError(f"call {i} was accepted")


def test_scan_bwd_past_4_gib():
    """x and the like of 4.3 GiB: two channels of the last sequence against the oracle (channels do not depend on each
    other; dB, dC and the parameters' gradients sum over all and are not compared)."""
    import oracle

    torch = torch_mod()
    nb, L, nd, ns = 9, 4096, 61440, 1
    say(f"scan_bwd {nb}x{L}x{nd}")
    gen = torch.Generator("cuda").manual_seed(10)
    v = scan_inputs(torch, gen, nb, L, nd, ns, torch.bfloat16)
    got = call("scan", v)
    torch.cuda.synchronize()
    ch = [0, nd - 1]
    h = {k: to_host64(t[-1:] if t.dim() == 3 and k in ("B", "C") else t[-1:, :, ch] if t.dim() == 3 else t[ch])
         for k, t in v.items()}
    want = oracle.scan_bwd(**h)
    for k in ("x", "dt", "z"):
        o = to_host64(got[k][-1:, :, ch])
        err = np.linalg.norm(o - want[k]) / np.linalg.norm(want[k])
        say(f"d{k}: {err:.2e}")
        assert err <= 2.5e-3, k


def test_adaln_past_4_gib():
    """Rows of the last sequence of tensors of 4.3 GiB, against the oracle on those rows."""
    import oracle
    import bidirectional_mamba_selective_amd as bm

    torch = torch_mod()
    nb, L, d = 3, 98304, 8192
    say(f"adaln {nb}x{L}x{d}")
    gen = torch.Generator("cuda").manual_seed(11)
    v = adaln_inputs(torch, gen, nb, L, d, torch.bfloat16, False)
    got = bm.bimamba_adaln_bwd(**v)
    torch.cuda.synchronize()
    rows = [0, L // 2, L - 1]
    h = {k: to_host64(t[-1:, rows] if t.dim() == 3 else t[-1:] if t.dim() == 2 else t) for k, t in v.items()}
    want = oracle.adaln_bwd(**h)
    for k in ("x", "branch"):
        err = np.linalg.norm(to_host64(got[k][-1:, rows]) - want[k]) / np.linalg.norm(want[k])
        say(f"d{k}: {err:.2e}")
        assert err <= 2.5e-3, k
    total = v["dout"][-1].double().sum(0)
    assert ((got["beta"][-1].double() - total).norm() / total.norm()).item() <= 1e-5


def test_conv_bwd_most_channels():
    """The largest accepted channel count, whose rows set the tile length: 24 channels against the oracle."""
    import oracle

    torch = torch_mod()
    C, L = 1 << 22, 70
    say(f"conv_bwd 1x{L}x{C}")
    gen = torch.Generator("cuda").manual_seed(12)
    v = conv_inputs(torch, gen, 1, L, C, torch.float32)
    got = call("conv", v)
    torch.cuda.synchronize()
    ch = list(range(8)) + list(range(C // 2, C // 2 + 8)) + list(range(C - 8, C))
    h = {k: to_host64(t[..., ch] if k[0] in "ud" else t[ch]) for k, t in v.items()}
    want = oracle.conv_bwd(**h)
    for k, t in got.items():
        o = to_host64(t[..., ch] if k == "u" else t[ch])
        err = np.linalg.norm(o - want[k]) / np.linalg.norm(want[k])
        say(f"d{k}: {err:.2e}")
        assert err <= 1e-5, k
