"""The delta rule, the 8-bit norm and the 8-bit projection on tensors of more than 2^31 values or 4 GiB.  Heads, batch elements,
rows and outputs do not depend on one another, so the parts with the lowest and the highest addresses are compared, bit for
bit, with a call on those parts alone, which other tests compare with the oracle."""
import pytest

from tests.gpu_util import say, torch_mod

pytestmark = pytest.mark.gpu

SEQ = ("q", "k", "v", "dt", "b")


def normal(*shape, dtype=None, scale=1.0, seed=0):
    torch = torch_mod()
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.empty(shape, device="cuda", dtype=dtype or torch.bfloat16).normal_(generator=g)).mul_(scale)


def delta_inputs(batch, L, heads, dk, dv, state, seed=1):
    torch = torch_mod()
    unit = lambda t: t.div_(t.float().square().sum(-1, keepdim=True).sqrt_())  # noqa: E731
    d = dict(q=unit(normal(batch, L, heads, dk, seed=seed)), k=unit(normal(batch, L, heads, dk, seed=seed + 1)),
             v=normal(batch, L, heads, dv, seed=seed + 2), dt=normal(batch, L, heads, scale=0.5, seed=seed + 3),
             b=normal(batch, L, heads, seed=seed + 4), A=-1 - normal(heads, dtype=torch.float32, seed=seed + 5).abs(),
             dt_bias=normal(heads, dtype=torch.float32, seed=seed + 6) - 3)
    if state:
        d["h_in"] = normal(batch, heads, dk, dv, dtype=torch.float32, scale=0.3, seed=seed + 7)
    return d


def head(d, i):
    return {n: (x[:, :, i:i + 1] if n in SEQ else x[i:i + 1] if x.ndim == 1 else x[:, i:i + 1]).contiguous()
            for n, x in d.items()}


def last(d, n):
    return {k: x if x.ndim == 1 else x[-n:].contiguous() for k, x in d.items()}


@pytest.fixture(autouse=True)
def release():
    yield
    torch_mod().cuda.empty_cache()


@pytest.mark.parametrize("rev", [False, True])
def test_delta_long_sequence(rev):
    """524358 tokens of 32 heads of 128 x 128: q, k, v and out hold 2^31 values and more each, the backward workspace 66 GB."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    L, heads = (1 << 19) + 70, 32
    d = delta_inputs(1, L, heads, 128, 128, True)
    assert d["v"].numel() > 1 << 31
    flags = bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY
    h = torch.empty_like(d["h_in"])
    say("forward")
    out = bm.bimamba_delta_fwd(**d, h_out=h, flags=flags)
    for i in (0, heads - 1):
        h1 = torch.empty_like(h[:, :1])
        o1 = bm.bimamba_delta_fwd(**head(d, i), h_out=h1, flags=flags)
        assert bool(torch.isfinite(o1).all()) and bool((o1 != 0).any())
        assert torch.equal(out[:, :, i:i + 1], o1) and torch.equal(h[:, i:i + 1], h1)
    say("backward")
    dout = out.copy_(normal(*out.shape, seed=9))
    g = bm.bimamba_delta_bwd(dout, **d, dh_out=h, flags=flags)
    for i in (0, heads - 1):
        g1 = bm.bimamba_delta_bwd(dout[:, :, i:i + 1].contiguous(), **head(d, i), dh_out=h[:, i:i + 1].contiguous(),
                                  flags=flags)
        for n, x in head(g, i).items():
            assert bool(torch.isfinite(g1[n]).all()) and torch.equal(x, g1[n]), n


@pytest.mark.parametrize("L", [2, 30])
def test_delta_many_states(L):
    """2050 sequences of 32 heads of 128 x 128, token by token and by chunks: 4.3 GB of states."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    d = delta_inputs(2050, L, 32, 128, 128, True)
    assert d["h_in"].numel() * 4 > 1 << 32
    h = torch.empty_like(d["h_in"])
    out = bm.bimamba_delta_fwd(**d, h_out=h)
    few = last(d, 16)  # 512 states: token by token, or two tiles a workgroup, as the whole call
    h1 = torch.empty_like(few["h_in"])
    o1 = bm.bimamba_delta_fwd(**few, h_out=h1)
    assert bool(torch.isfinite(o1).all()) and torch.equal(out[-16:], o1) and torch.equal(h[-16:], h1)


def test_norm_of_many_rows():
    """294912 rows of 8192 bf16 values: 4.8 GB in and 2^31 values of 8 bits out."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    nb, L, nd = 9, 32768, 8192
    x, m = normal(nb, L, nd, seed=1), normal(nb, L, nd, seed=2)
    p = [normal(nb, nd, dtype=torch.float32, seed=3 + i) for i in range(3)]
    h, out, scales = bm.bimamba_adaln_fwd_fp8(x, p[0], p[1], m, None, p[2])
    assert out.numel() > 1 << 31
    bits = lambda t: t.view(torch.uint8)  # noqa: E731
    for b, t in ((0, 0), (nb - 1, L - 40)):
        part = [v[b:b + 1, t:t + 40].contiguous() for v in (x, m)]
        h1, o1, s1 = bm.bimamba_adaln_fwd_fp8(part[0], p[0][b:b + 1], p[1][b:b + 1], part[1], None, p[2][b:b + 1])
        assert torch.equal(h[b:b + 1, t:t + 40], h1) and torch.equal(scales[b:b + 1, t:t + 40], s1)
        assert torch.equal(bits(out[b:b + 1, t:t + 40]), bits(o1))


def e4m3(*shape, seed):
    torch = torch_mod()
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):  # a piece at a time: the normal numbers are 4 times as many bytes
        n = min(1 << 28, flat.numel() - at)
        flat[at:at + n] = normal(n, dtype=torch.float32, scale=60.0, seed=seed + at % 1009).to(torch.float8_e4m3fn)
    return out


@pytest.mark.parametrize("m,n,k,dtype", [((1 << 20) + 100, 2056, 4096, "bfloat16"), ((1 << 20) + 100, 2056, 128, "float32"),
                                         (64, (1 << 20) + 136, 4096, "bfloat16"), (20, (1 << 22), 1152, "float32")])
def test_projection(m, n, k, dtype):
    """Rows, weights or results past 2^31 values (4 GiB)."""
    import bidirectional_mamba_selective_amd as bm
    torch = torch_mod()

    dt = getattr(torch, dtype)
    assert max(m * k, n * k, m * n * dt.itemsize) > 1 << 32
    x, w = e4m3(1, m, k, seed=1), e4m3(n, k, seed=2)
    xs = normal(1, m, k // 128, dtype=torch.float32, seed=3).abs()
    ws = normal(-(-n // 128), k // 128, dtype=torch.float32, seed=4).abs()
    say(f"{m} x {n} x {k}")
    out = bm.bimamba_proj_fp8(x, xs, w, ws, out_dtype=dt)
    # 300 rows and 2048 outputs at a time: tiles, whose sums run in one order whatever the tile (few rows: in another)
    same = m > 64
    for r0 in {0, max(m - 300, 0)}:
        for c0 in (0, (n - 1024) // 128 * 128):
            rows, cols = slice(r0, r0 + 300), slice(c0, min(c0 + 2048, n))
            o1 = bm.bimamba_proj_fp8(x[:, rows].contiguous(), xs[:, rows].contiguous(), w[cols], ws[c0 // 128:c0 // 128 + 16]
                                     [:-(-w[cols].shape[0] // 128)].contiguous(), out_dtype=dt)
            got = out[:, rows, cols]
            assert bool(torch.isfinite(o1).all()) and bool((o1 != 0).any())
            if same:
                assert torch.equal(got, o1), (r0, c0)
            else:  # sums in two orders: k / 128 + 8 roundings of each, and of a bf16 result one step
                f = lambda t: t[0, rows].float() * xs[0, rows].repeat_interleave(128, 1)  # noqa: E731
                s = ws[c0 // 128:c0 // 128 + 16].repeat_interleave(128, 0)[:w[cols].shape[0]].repeat_interleave(128, 1)
                mag = f(x).abs() @ (w[cols].float() * s).abs().t()
                step = 2.0 ** -7 if dtype == "bfloat16" else 0.0
                unit = 2.0 ** -12 if dtype == "bfloat16" else 2.0 ** -24 * (k // 128 + 8)
                assert bool(((got[0] - o1[0]).float().abs() <= 2 * unit * mag + step * o1[0].float().abs()).all())
