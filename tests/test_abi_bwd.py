"""Refusals of the backward and norm entry points, on the host before any HIP call (no GPU).

The pointer values are never dereferenced: every call here fails validation."""
import ctypes
import os

import pytest

from bidirectional_mamba_selective_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libbimamba.so not built")

INV, UNS, WS = _lib.BIMAMBA_ERR_INVALID_ARGUMENT, _lib.BIMAMBA_ERR_UNSUPPORTED, _lib.BIMAMBA_ERR_WORKSPACE_TOO_SMALL
BF16, F32 = _lib.BIMAMBA_BF16, _lib.BIMAMBA_F32
BASE, SPAN = 1 << 30, 1 << 26


def fake(i, off=0):
    return ctypes.c_void_p(BASE + i * SPAN + off)


def call(entry, names, sizes, kw):
    """entry(pointers in the order of names, then sizes): fake pointers far apart, replaced by kw."""
    a = {n: fake(i) for i, n in enumerate(names)}
    a.update(sizes)
    a.update(kw)
    return getattr(_lib.load(), entry)(*[a[k] for k in list(names) + list(sizes)])


SCAN = ("dout", "x", "dt", "A", "B", "C", "D", "z", "dt_bias", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")
SCAN_SIZES = dict(batch=2, L=64, d=64, n=16, io=BF16, flags=0, ws=fake(40), wsb=0, stream=None)
SI = {n: i for i, n in enumerate(SCAN)}


@pytest.mark.parametrize("kw,want", [
    *[({n: None}, INV) for n in ("dout", "x", "dt", "A", "B", "C", "dx", "ddt", "dA", "dB", "dC", "z", "dz")],
    ({"flags": _lib.FLAG_FWD_ONLY | _lib.FLAG_REV_ONLY}, INV),
    ({"flags": 32}, INV),
    ({"flags": _lib.FLAG_NO_GATE, "wsb": 1 << 40}, INV),  # dz without a gate
    ({"batch": 0}, INV),
    ({"L": 0}, INV),
    ({"n": 17}, UNS),
    ({"d": 96}, UNS),
    ({"io": 2}, UNS),
    ({"batch": 1 << 15, "L": 1 << 13}, UNS),  # 2^32 threads for B and C
    ({}, WS),
    ({"D": None, "dt_bias": None, "dD": None, "ddt_bias": None}, WS),  # optional: gets to the workspace
    ({"z": None, "dz": None, "flags": _lib.FLAG_NO_GATE}, WS),
    ({"ws": None, "wsb": 1 << 40}, INV),
    ({"ws": fake(40, 16), "wsb": 1 << 40}, INV),
    ({"x": fake(SI["x"], 8), "wsb": 1 << 40}, INV),
    ({"dB": fake(SI["dB"], 1), "wsb": 1 << 40}, INV),
    ({"dA": fake(SI["dA"], 4), "wsb": 1 << 40}, INV),
    ({"dx": fake(SI["x"], 64), "wsb": 1 << 40}, INV),       # an output over an input
    ({"dB": fake(SI["dC"], 32), "wsb": 1 << 40}, INV),      # two outputs over each other
    ({"ddt_bias": fake(SI["D"]), "wsb": 1 << 40}, INV),
    ({"ws": fake(SI["dout"]), "wsb": 1 << 40}, INV),        # workspace over an input
    ({"dz": fake(40, 4096), "wsb": 1 << 40}, INV),          # an output inside the workspace
])
def test_scan_bwd_rejects(kw, want):
    assert call("bimamba_scan_bwd", SCAN, SCAN_SIZES, kw) == want


def test_scan_bwd_workspace_bytes():
    f = _lib.bimamba_scan_bwd_workspace_bytes
    sizes = [f(1, L, 4096, 16) for L in (1, 16, 17, 1000, 2048, 65536)]
    assert sizes == sorted(sizes) and all(s > 0 and s % 256 == 0 for s in sizes)
    assert f(1, 64, 96, 16) == 0 and f(1, 64, 64, 17) == 0 and f(0, 64, 64, 16) == 0
    assert f(1 << 15, 1 << 13, 64, 16) == 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    import bidirectional_mamba_selective_amd as bm

    x = torch.zeros(1, 4, 64)
    with pytest.raises((ValueError, RuntimeError)):
        bm.bimamba_scan_bwd(x, x, x, torch.zeros(64, 2), torch.zeros(1, 4, 2), torch.zeros(1, 4, 2), z=x)
