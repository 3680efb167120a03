"""How accurate the fp32 results of the delta rule and the products of the 8-bit projection are, normwise against 64 bits.

Tighter than the bounds per element, which hold for the worst inputs: errors of many roundings are taken as independent, so
their squares add.
- delta rule: a state, its gradient and a sum over tokens pass, per 64-token run, through four chained products of at most
  128 terms, their operands and partial sums held to 2^-24: 4 x 128 roundings, sqrt(512) 2^-24 = 2^-19.5 of a run's terms;
  2^-18 allows as much again from the runs before (which decay) and for terms that cancel within a run.  Operands of two
  bf16 parts would leave 2^-17 each.
- projection to fp32, n blocks of 128 inputs: four chained sums of 32 products and two roundings of the scales per block, of
  block sums whose squares add up to the result's; n additions to partial sums, n / 2 of the result's square on average:
  2^-24 sqrt(n / 2 + 6), doubled.
- projection to bf16: the 8-bit matrix instruction's own sums, which are not fp32 ones, keep 2^-15 of the result normwise for
  operands of one scale, whatever the number of blocks (each block's error has the block sum's size, and squares add).  Seen
  on results smaller than 2^-9 of the rms, whose own rounding is at most 2^-17 of it."""
import numpy as np
import pytest

from tests.gpu_util import f32_dev, rel_err, say, to_dev, to_host64, torch_mod
from tests.test_gpu_delta import make, run_fwd, upload
from tests.test_gpu_fp8 import e4m3_values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("decay", [1.0, 0.01])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
def test_delta_fp32_results(dk, dv, decay, rev):
    import bidirectional_mamba_selective_amd as bm
    import oracle

    inp, dout, dh = make(1, 700, 1, 2, dk, dv, seed=37)
    inp["A"] = (inp["A"] * decay).astype(np.float32)
    dev = upload(inp)
    _, h = run_fwd(bm, dev, rev)
    g = bm.bimamba_delta_bwd(to_dev(dout, "bf16"), **dev, dh_out=f32_dev(dh),
                             flags=bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY)
    want = oracle.delta_bwd(dout, inp, dh, rev=rev)
    off = {n: rel_err(to_host64(g[n]), want[n]) for n in ("A", "dt_bias", "h_in")}
    off["h_out"] = rel_err(to_host64(h), oracle.delta_fwd(inp, rev=rev)[1])
    say(f"{dk} x {dv}, A x {decay}: " + ", ".join(f"{n} {v:.2e}" for n, v in off.items()))
    assert all(v <= 2.0 ** -18 for v in off.values()), off


def product(m, n, k, dtype):
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    r = np.random.default_rng(k + m)
    x, w = e4m3_values((1, m, k), r, 120.0), e4m3_values((n, k), r, 120.0)
    xs = torch.from_numpy(r.uniform(0.5, 2, (1, m, k // 128)).astype(np.float32))
    ws = torch.from_numpy(r.uniform(0.5, 2, (-(-n // 128), k // 128)).astype(np.float32))
    got = to_host64(bm.bimamba_proj_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), out_dtype=dtype))[0]
    x = x[0].double().numpy() * np.repeat(xs[0].double().numpy(), 128, 1)
    w = w.double().numpy() * np.repeat(np.repeat(ws.double().numpy(), 128, 0)[:n], 128, 1)
    return got, x @ w.T


SIZES = [(20, 1024, 4096), (200, 1024, 128), (200, 1024, 1920), (1024, 3200, 1024), (600, 520, 16384)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_projection_to_fp32(m, n, k):
    got, want = product(m, n, k, torch_mod().float32)
    off, allow = rel_err(got, want), 2.0 ** -23 * (k / 256 + 6) ** 0.5
    say(f"{m} x {n} x {k}: {off:.2e} (bound {allow:.2e})")
    assert off <= allow


@pytest.mark.parametrize("m,n,k", SIZES + [(4096, 2304, 512)])
def test_projection_to_bf16(m, n, k):
    got, want = product(m, n, k, torch_mod().bfloat16)
    rms = np.sqrt(np.mean(want ** 2))
    small = np.abs(want) < 2.0 ** -9 * rms
    off = float(np.sqrt(np.mean((got - want)[small] ** 2)) / rms)
    say(f"{m} x {n} x {k}: {off:.2e} of the rms over {int(small.sum())} small results")
    assert small.sum() >= 20 and off <= 2.0 ** -15 + 2.0 ** -17
