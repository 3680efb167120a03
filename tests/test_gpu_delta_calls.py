"""Calls of the delta rule, the 8-bit norm and the projection that their documentation allows beside the plain ones: the cache's
gradient in place, gradients asked for of inputs that were not given, calls on two streams at once, one tensor in two places."""
import ctypes

import pytest

from tests.gpu_util import f32_dev, to_dev, torch_mod
from tests.test_gpu_delta import make, run_fwd, upload
from tests.test_gpu_fp8 import make_proj

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,heads,dk,dv", [(1, 2, 64, 64), (100, 2, 128, 128), (130, 40, 64, 128)])
def test_gradient_of_the_cache_in_place(L, heads, dk, dv):
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    inp, dout, dh = make(1, L, heads, heads, dk, dv, seed=L)
    dev, dout, dh = upload(inp), to_dev(dout, "bf16"), f32_dev(dh)
    want = bm.bimamba_delta_bwd(dout, **dev, dh_out=dh)
    both = dh.clone()
    got = bm.bimamba_delta_bwd(dout, **dev, dh_out=both, grads={"h_in": both})
    assert got["h_in"] is both and all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("rev", [False, True])
def test_gradients_of_inputs_that_are_not_given(rev):
    """ddt_bias and dh_in without dt_bias and h_in, as where these are zeros; then neither of the two outputs."""
    import bidirectional_mamba_selective_amd as bm
    from bidirectional_mamba_selective_amd import _lib
    torch = torch_mod()

    nb, L, hk, nh, dk, dv = 2, 90, 2, 4, 64, 128
    inp, dout, _ = make(nb, L, hk, nh, dk, dv, seed=41, state=False, bias=False)
    dev, dout = upload(inp), to_dev(dout, "bf16")
    flags = bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY
    zeros = dict(dt_bias=torch.zeros(nh, device="cuda"), h_in=torch.zeros(nb, nh, dk, dv, device="cuda"))
    want = bm.bimamba_delta_bwd(dout, **{**dev, **zeros}, flags=flags)
    ws = torch.empty(bm.bimamba_delta_bwd_workspace_bytes(nb, L, hk, nh, dk, dv), dtype=torch.uint8, device="cuda")
    for asked in (True, False):
        got = {n: torch.full_like(x, float("nan")) for n, x in want.items()}
        p = lambda t: ctypes.c_void_p(None if t is None else t.data_ptr())  # noqa: E731
        st = _lib.load().bimamba_delta_bwd(
            p(dout), *[p(dev[n]) for n in ("q", "k", "v", "dt", "A", "b")], None, None, None,
            *[p(got[n]) for n in ("q", "k", "v", "dt", "A", "b")], p(got["dt_bias"]) if asked else None,
            p(got["h_in"]) if asked else None, nb, L, hk, nh, dk, dv, dk ** -0.5, bm.BIMAMBA_BF16, flags, p(ws),
            ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert st == 0
        for n in want:
            if asked or n not in ("dt_bias", "h_in"):
                assert torch.equal(got[n], want[n]), n
            else:
                assert bool(torch.isnan(got[n]).all()), n


def test_two_streams_at_once():
    """Calls on two streams, workspaces and results of the binding's own, several times over: the same bits as one by one."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    sets = [make(1, L, 2, 4, 128, 64, seed=L) for L in (500, 700)]
    sets = [(upload(i), to_dev(o, "bf16"), f32_dev(h)) for i, o, h in sets]
    proj = [[v.cuda() for v in make_proj(m, 520, 640, seed=m)] for m in (40, 300)]
    x = [torch.randn(1, 60, 640, device="cuda") for _ in range(2)]

    def work(i, s):
        d, o, h = sets[i]
        return [bm.bimamba_delta_fwd(**d, stream=s), *bm.bimamba_delta_bwd(o, **d, dh_out=h, stream=s).values(),
                bm.bimamba_proj_fp8(*proj[i], stream=s), *bm.bimamba_adaln_fwd_fp8(x[i], stream=s)[1:]]

    want = [work(i, None) for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i in (0, 1):
            got[i].append(work(i, streams[i]))
    torch.cuda.synchronize()
    bits = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t  # noqa: E731
    for i in (0, 1):
        for run in got[i]:
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(run, want[i]))


@pytest.mark.parametrize("L", [9, 100])
def test_one_tensor_as_query_and_key_and_gate(L):
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    inp, dout, _ = make(1, L, 2, 2, 64, 64, seed=L)
    dev, dout = upload(inp), to_dev(dout, "bf16")
    apart = {**dev, "q": dev["k"].clone(), "b": dev["dt"].clone()}
    shared = {**dev, "q": dev["k"], "b": dev["dt"]}
    assert all(torch.equal(a, b) for a, b in zip(run_fwd(bm, shared, False), run_fwd(bm, apart, False)))
    g, w = bm.bimamba_delta_bwd(dout, **shared), bm.bimamba_delta_bwd(dout, **apart)
    assert all(torch.equal(g[n], w[n]) for n in w if w[n] is not None)


def test_two_tiles_in_a_replayed_graph():
    """Many heads, several segments, forward and backward, captured once and replayed between other work."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    inp, dout, dh = make(1, 900, 80, 80, 64, 64, seed=43)
    dev, dout, dh = upload(inp), to_dev(dout, "bf16"), f32_dev(dh)
    run = lambda: [*run_fwd(bm, dev, False), *bm.bimamba_delta_bwd(dout, **dev, dh_out=dh).values()]  # noqa: E731
    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for turn in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), turn
        run()  # eager work in between
