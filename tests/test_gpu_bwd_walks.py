"""The loops that short inputs do not enter, against the fp64 oracle: many tiles per chunk in the scan's backward pass, and
several rows per workgroup in the norm / gate / residual step at every number of wavefronts per row.

The scan's chunks grow only once the chip is full, so its inputs here are wide, and the incoming gradient is zero but for
a few sequences or channels: every gradient of the others is exactly zero, and what is left is small enough for the
oracle.  A parameter's gradient and dB, dC then sum the chosen part alone, the zeros adding nothing.  Bounds: those of
test_gpu_scan_bwd.py and test_gpu_adaln.py."""
import numpy as np
import pytest

from tests import test_gpu_adaln as ad
from tests import test_gpu_scan_bwd as sb
from tests.gpu_util import say, to_host64, torch_mod
from tests.test_bwd_plans import adaln_workgroups, scan_chunks

pytestmark = pytest.mark.gpu

PER_TOKEN = ("x", "dt", "z")


@pytest.mark.parametrize("dirs,gate,io", [("both", True, "f32"), ("both", True, "bf16"), ("fwd", True, "f32"),
                                          ("rev", False, "bf16"), ("rev", True, "f32")])
@pytest.mark.parametrize("batch,L", [(137, 277), (410, 331)])
def test_scan_bwd_many_tiles_few_sequences(batch, L, dirs, gate, io):
    """Nine tiles per chunk in two chunks, and 21 in one; the last tile ragged; 16 states, 320 channels."""
    torch = torch_mod()
    d, n = 320, 16
    chunks = scan_chunks(batch, L, d, n)
    assert -(-L // 16) // chunks >= 8
    say(f"scan_bwd {batch}x{L}x{d} {dirs} gate={gate} {io}: {chunks} chunks")
    picked = [0, batch // 2, batch - 1]
    inp, dout = sb.make(len(picked), L, d, n, io, seed=21)
    small, g = sb.upload(inp, dout, io)
    gen = torch.Generator("cuda").manual_seed(21)
    dev = {}
    for k, v in small.items():
        if k in sb.VECTORS:
            dev[k] = v
            continue
        dev[k] = torch.randn((batch,) + v.shape[1:], generator=gen, device="cuda").to(v.dtype)
        dev[k][picked] = v
    full = torch.zeros((batch,) + g.shape[1:], dtype=g.dtype, device="cuda")
    full[picked] = g
    got = sb.run(dev, full, dirs, gate)
    rest = torch.ones(batch, dtype=torch.bool, device="cuda")
    rest[picked] = False
    for k, t in got.items():
        if t is not None and k not in sb.VECTORS:
            assert torch.count_nonzero(t[rest]) == 0, k
            got[k] = t[picked]
    sb.check_grads(got, inp, dout, io, L, dirs, gate, tag=f"{batch} sequences {dirs} {io}")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_bwd_many_tiles_few_channels(io):
    """One sequence of the paper's width, nine tiles per chunk in 31 chunks, the last one short and ragged."""
    torch = torch_mod()
    L, d, n = 4389, 3840, 16
    chunks = scan_chunks(1, L, d, n)
    assert chunks == 31 and -(-L // 16) == 275
    say(f"scan_bwd 1x{L}x{d} {io}")
    picked = [0, 1, 63, 64, 1900, 3775, 3776, 3839]
    inp, dout = sb.make(1, L, len(picked), n, io, seed=22)
    small, g = sb.upload(inp, dout, io)
    gen = torch.Generator("cuda").manual_seed(22)
    dev = {}
    for k, v in small.items():
        if k in ("B", "C"):
            dev[k] = v
        elif k in PER_TOKEN:
            dev[k] = torch.randn((1, L, d), generator=gen, device="cuda").to(v.dtype)
            dev[k][..., picked] = v
        else:
            dev[k] = -torch.rand((d,) + v.shape[1:], generator=gen, device="cuda")
            dev[k][picked] = v
    full = torch.zeros((1, L, d), dtype=g.dtype, device="cuda")
    full[..., picked] = g
    got = sb.run(dev, full)
    rest = torch.ones(d, dtype=torch.bool, device="cuda")
    rest[picked] = False
    for k, t in got.items():
        if k in PER_TOKEN:
            assert torch.count_nonzero(t[..., rest]) == 0, k
            got[k] = t[..., picked]
        elif k in sb.VECTORS:
            assert torch.count_nonzero(t[rest]) == 0, k
            got[k] = t[picked]
    sb.check_grads(got, inp, dout, io, L, tag=f"8 channels of {d} {io}")


# widths of 2, 4, 8 and 16 wavefronts a row; the last one of 8 and the first of 16 not filled
WIDTHS = [1000, 1928, 4096, 2056, 8192, 4104]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("d", WIDTHS)
def test_adaln_bwd_several_rows_per_workgroup(d, post, rms, io):
    """Three or four rows a workgroup, the last one with fewer.  With and without the mean and the post-norm a row takes
    one to three sums, so the alternating buffers start rows on either one."""
    L = {1000: 4999, 1928: 2699}.get(d, 799)
    groups, _ = adaln_workgroups(1, L, d)
    assert -(-L // groups) >= 3 and L % -(-L // groups)
    say(f"adaln_bwd 1x{L}x{d} rms={rms} post={post} {io}")
    ad.check_bwd(ad.make(1, L, d, io, seed=d, drop=() if post else ("post_weight",)), io, rms)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", WIDTHS)
def test_adaln_bwd_several_rows_shared_modulation(d, io):
    """One gamma, beta and gate for three sequences, several rows a workgroup."""
    L = {1000: 1700, 1928: 901}.get(d, 271)
    groups, _ = adaln_workgroups(3, L, d)
    assert -(-L // (groups // 3)) >= 3
    say(f"adaln_bwd 3x{L}x{d} shared {io}")
    ad.check_bwd(ad.make(3, L, d, io, seed=d + 1, rows=1), io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("d", [1000, 1928, 4096, 8192])
def test_adaln_fwd_several_rows_per_workgroup(d, post, rms, io):
    """2048 workgroups of four rows (the last one of three): the rows of the first, a middle and the last two workgroups,
    as a batch of their own for the oracle."""
    import oracle
    import bidirectional_mamba_selective_amd as bm

    torch = torch_mod()
    L = 4 * 2047 + 3
    say(f"adaln_fwd 1x{L}x{d} rms={rms} post={post} {io}")
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[io]
    gen = torch.Generator("cuda").manual_seed(d)

    def rnd(*shape, m=0.0, s=1.0, dtype=torch.float32):
        return (m + s * torch.randn(shape, generator=gen, device="cuda")).to(dtype)

    x, m = rnd(1, L, d, m=0.3, s=3.0, dtype=dt), rnd(1, L, d, m=0.1, s=1.5, dtype=dt)
    gamma, beta, gate = rnd(1, d, m=1.0, s=0.3), rnd(1, d, s=0.3), rnd(1, d, m=0.5, s=0.4)
    w = rnd(d, m=1.0, s=0.3) if post else None
    h, out = bm.bimamba_adaln_fwd(x, gamma, beta, m, w, gate, eps=ad.EPS, flags=bm.FLAG_RMS_NORM if rms else 0)
    rows = list(range(4)) + list(range(4000, 4008)) + list(range(L - 7, L))
    hx, hm, got_h, got_out = (to_host64(t[:, rows]) for t in (x, m, h, out))
    hg, hb, hgate = (to_host64(t) for t in (gamma, beta, gate))
    hw = None if w is None else to_host64(w)
    wh, wout = oracle.adaln_fwd(hx, hg, hb, hm, hw, hgate, eps=ad.EPS, rms=rms)
    # the magnitudes of each element's terms, as test_gpu_adaln.py's check_fwd forms them
    branch = np.abs(hm)
    if post:
        branch = branch / np.sqrt(np.mean(hm * hm, -1, keepdims=True) + ad.EPS) * np.abs(hw)
    mag = np.abs(hx) + branch * ad.mod(hgate)
    ad.close(got_h, wh, mag, io, 100, f"h {io}")
    c = wh if rms else wh - wh.mean(-1, keepdims=True)
    rs = 1 / np.sqrt(np.mean(c * c, -1, keepdims=True) + ad.EPS)
    cm = mag if rms else mag + ad.mean_abs(mag)
    spread = np.sqrt(np.mean(cm * cm, -1, keepdims=True)) * rs
    ad.close(got_out, wout, ad.mod(hg) * rs * (cm + np.abs(c) * spread) + ad.mod(hb), io, 100, f"out {io}")
