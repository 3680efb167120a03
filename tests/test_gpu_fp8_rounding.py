"""The 8-bit norm's values bit for bit: y over its block's scale, one fp32 division, rounded to nearest even e4m3.

With gamma = 0 the norm's value is beta itself, so a test chooses y.  Here every value lies within one step of fp32 of a
border between two e4m3 values (times its block's scale), where a second rounding on the way shows."""
import numpy as np
import pytest

from tests.gpu_util import torch_mod

E4M3_BORDERS = np.array(sorted({(m + 0.5) / 8 * 2.0 ** e for m in range(8, 16) for e in range(-6, 8)} |
                               {(m + 0.5) * 2.0 ** -9 for m in range(8)} | {447.0, 448.0}), np.float32)
E4M3_BORDERS = E4M3_BORDERS[E4M3_BORDERS <= 448]


def border_values(blocks, seed=0):
    """fp32 [blocks, 128]: one value is the block's largest, the others at a border, the fp32 value below or above it."""
    r = np.random.default_rng(seed)
    largest = np.exp(r.uniform(-66, 80, (blocks, 1))).astype(np.float32)
    s = largest / np.float32(448)
    y = r.choice(E4M3_BORDERS, (blocks, 128)) * s
    y = np.where(r.integers(0, 3, y.shape) == 0, np.nextafter(y, np.float32(0)), y)
    y = np.where(r.integers(0, 3, y.shape) == 0, np.nextafter(y, np.float32(np.inf)), y)
    y = np.minimum(y, largest) * r.choice(np.float32([-1, 1]), y.shape)
    y[np.arange(blocks), r.integers(0, 128, blocks)] = largest[:, 0]
    return y.astype(np.float32)


def divided(y):
    torch = torch_mod()
    t = torch.from_numpy(y)
    s = t.abs().amax(-1, keepdim=True) / 448
    return (t / s).to(torch.float8_e4m3fn), s.squeeze(-1)


def test_values_tell_a_division_from_a_reciprocal():
    torch = torch_mod()
    y = border_values(4096)
    q, s = divided(y)
    other = (torch.from_numpy(y) * (1 / s)[:, None]).to(torch.float8_e4m3fn)
    assert int((q.view(torch.uint8) != other.view(torch.uint8)).sum()) > 1000


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 640, 2048, 8192])
def test_values_at_borders(d):
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    batch = 40
    y = border_values(batch * d // 128, seed=d)
    q, s = divided(y)
    for io in (torch.float32, torch.bfloat16):
        x = torch.randn(batch, 3, d, device="cuda").to(io)
        _, out, scales = bm.bimamba_adaln_fwd_fp8(x, torch.zeros(batch, d, device="cuda"),
                                                  torch.from_numpy(y).view(batch, d).cuda())
        want = q.view(batch, 1, d).expand(-1, 3, -1).contiguous().view(torch.uint8)
        assert torch.equal(scales.cpu(), s.view(batch, 1, -1).expand(-1, 3, -1))
        assert torch.equal(out.cpu().view(torch.uint8), want)


@pytest.mark.gpu
def test_infinities_and_the_least_blocks():
    """A block with an infinity has the scale infinity: NaN there and 0 in its other places, as the division gives; blocks
    whose largest magnitude is 2^-100, one step around it, subnormal or zero."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    least = np.float32(2.0 ** -100)
    y = np.repeat(np.linspace(-1, 1, 128, dtype=np.float32)[None], 8, 0)
    y[0, 7] = np.inf
    y[1, [3, 4]] = -np.inf, np.inf
    y[2:6] *= np.float32([least, np.nextafter(least, np.float32(1)), np.nextafter(least, np.float32(0)), 2.0 ** -140])[:, None]
    y[6] = 0
    t = torch.from_numpy(y)
    s = t.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100) / 448
    want = (t / s).to(torch.float8_e4m3fn)
    x = torch.randn(8, 1, 128, device="cuda")
    _, out, scales = bm.bimamba_adaln_fwd_fp8(x, torch.zeros(8, 128, device="cuda"), t.cuda())
    assert torch.equal(scales.cpu().view(8, 1), s)
    nan = torch.isnan(want.float())
    got = out.cpu().view(8, 128)
    assert torch.equal(torch.isnan(got.float()), nan) and int(nan.sum()) == 3
    assert torch.equal(got.float()[~nan], want.float()[~nan])
