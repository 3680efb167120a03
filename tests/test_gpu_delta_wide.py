"""The delta rule with many heads: calls that go token by token up to 24 tokens, and walks of two tiles of 16 columns a
workgroup, which a call has from 256 tiles on.

A sample of the heads, the first and the last among them, is compared with the oracle; where a workgroup has two tiles, every
head with a call of few heads, whose workgroups have one: the same arithmetic, so the same bits."""
import numpy as np
import pytest

from tests.gpu_util import f32_dev, to_dev, to_host64, torch_mod
from tests.test_gpu_delta import SEQ, close, make, run_fwd, upload

pytestmark = pytest.mark.gpu


def heads_of(inp, sel):
    return {n: None if x is None else x[:, :, sel] if n in SEQ else x[sel] if x.ndim == 1 else x[:, sel]
            for n, x in inp.items()}


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("batch,heads,dk,dv", [(4, 64, 128, 128), (2, 256, 128, 64), (16, 64, 64, 64)])
@pytest.mark.parametrize("L", [17, 24, 25])
def test_tokens_one_by_one_in_wide_calls(batch, heads, dk, dv, L, rev):
    import bidirectional_mamba_selective_amd as bm
    import oracle

    assert (bm.bimamba_delta_fwd_workspace_bytes(batch, L, heads, heads, dk, dv) == 0) == (L <= 24)
    inp, _, _ = make(batch, L, heads, heads, dk, dv, seed=L)
    out, h = run_fwd(bm, upload(inp), rev)
    sel = [0, 1, heads // 2 + 1, heads - 1]
    part = heads_of(inp, sel)
    wout, wh = oracle.delta_fwd(part, rev=rev)
    r = oracle.delta_bounds(part, rev=rev)
    close(to_host64(out)[:, :, sel], wout, r["out"], "out")
    close(to_host64(h)[:, sel], wh, r["h_out"], "h_out", bf16=False)


WIDE = [(1, 40, 128, 128), (2, 20, 64, 128), (1, 72, 128, 64), (1, 80, 64, 64), (3, 25, 64, 64)]


def halves(x, n, part, nh):
    """Heads [0, nh / 2) or the others of a tensor that has them."""
    sel = slice(0, nh // 2) if part == 0 else slice(nh // 2, nh)
    return None if x is None else (x[sel] if x.ndim == 1 else x[:, :, sel] if n in SEQ else x[:, sel]).contiguous()


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("L", [64, 130, 187])
@pytest.mark.parametrize("batch,heads,dk,dv", WIDE)
def test_two_tiles_forward(batch, heads, dk, dv, L, rev):
    import bidirectional_mamba_selective_amd as bm
    import oracle
    torch = torch_mod()

    assert batch * heads * dv // 16 > 256 >= batch * (heads - heads // 2) * dv // 16
    inp, _, _ = make(batch, L, heads, heads, dk, dv, seed=L)
    dev = upload(inp)
    out, h = run_fwd(bm, dev, rev)
    few = [run_fwd(bm, {n: halves(x, n, p, heads) for n, x in dev.items()}, rev) for p in (0, 1)]
    assert torch.equal(out, torch.cat([o for o, _ in few], 2)) and torch.equal(h, torch.cat([s for _, s in few], 1))
    sel = [0, heads // 3, heads - 1]
    part = heads_of(inp, sel)
    wout, wh = oracle.delta_fwd(part, rev=rev)
    r = oracle.delta_bounds(part, rev=rev)
    close(to_host64(out)[:, :, sel], wout, r["out"], "out")
    close(to_host64(h)[:, sel], wh, r["h_out"], "h_out", bf16=False)


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("L", [64, 130])
@pytest.mark.parametrize("batch,heads,dk,dv", WIDE)
def test_two_tiles_backward(batch, heads, dk, dv, L, rev):
    import bidirectional_mamba_selective_amd as bm
    import oracle
    torch = torch_mod()

    assert batch * heads * dv // 16 > 256 >= batch * (heads - heads // 2) * dv // 16
    inp, dout, dh = make(batch, L, heads, heads, dk, dv, seed=L)
    dev, do, dhd = upload(inp), to_dev(dout, "bf16"), f32_dev(dh)
    flags = bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY
    got = bm.bimamba_delta_bwd(do, **dev, dh_out=dhd, flags=flags)
    few = [bm.bimamba_delta_bwd(halves(do, "v", p, heads), **{n: halves(x, n, p, heads) for n, x in dev.items()},
                                dh_out=halves(dhd, "h_in", p, heads), flags=flags) for p in (0, 1)]
    for n, g in got.items():
        assert torch.equal(g, torch.cat([f[n] for f in few], 2 if n in SEQ else 0 if g.ndim == 1 else 1)), n
    sel = [0, heads // 3, heads - 1]
    part = heads_of(inp, sel)
    want = oracle.delta_bwd(dout[:, :, sel], part, dh[:, sel], rev=rev)
    r = oracle.delta_bounds(part, dout[:, :, sel], dh[:, sel], rev=rev)
    for n, w in want.items():
        g = to_host64(got[n])
        close(g[:, :, sel] if n in SEQ else g[sel] if g.ndim == 1 else g[:, sel], w, r[n], "d" + n, bf16=n in SEQ)


def test_two_tiles_with_shared_keys_and_segments():
    """Two value heads to a key head, a long sequence in segments, the gradients' sums over shared heads: the first heads
    alone give the same bits."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    L, hk, heads = 4000, 20, 40
    inp, dout, dh = make(1, L, hk, heads, 128, 128, seed=31)
    assert (bm.bimamba_delta_fwd_workspace_bytes(1, L, hk, heads, 128, 128)
            < L // 64 * (bm.bimamba_delta_fwd_workspace_bytes(1, 64, hk, heads, 128, 128)))  # several segments
    dev, do, dhd = upload(inp), to_dev(dout, "bf16"), f32_dev(dh)
    first = {n: None if x is None else x[:, :, :10].contiguous() if n in ("q", "k") else x[:, :, :20].contiguous()
             if n in SEQ else x[:20] if x.ndim == 1 else x[:, :20].contiguous() for n, x in dev.items()}
    for rev in (False, True):
        flags = bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY
        (out, h), (o1, h1) = run_fwd(bm, dev, rev), run_fwd(bm, first, rev)
        assert torch.equal(out[:, :, :20], o1) and torch.equal(h[:, :20], h1)
        g = bm.bimamba_delta_bwd(do, **dev, dh_out=dhd, flags=flags)
        g1 = bm.bimamba_delta_bwd(do[:, :, :20].contiguous(), **first, dh_out=dhd[:, :20].contiguous(), flags=flags)
        for n, x in g1.items():
            k = x.shape[2] if n in SEQ else 20
            assert torch.equal(x, g[n][:, :, :k] if n in SEQ else g[n][:k] if x.ndim == 1 else g[n][:, :k]), n
