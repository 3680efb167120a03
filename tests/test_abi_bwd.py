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


CONV = ("dout_f", "dout_r", "u", "w_f", "b_f", "w_r", "b_r", "du", "dw_f", "db_f", "dw_r", "db_r")
CONV_SIZES = dict(batch=2, L=64, C=64, K=4, io=BF16, flags=0, ws=fake(40), wsb=0, stream=None)
CI = {n: i for i, n in enumerate(CONV)}
NO_F = {n: None for n in ("dout_f", "dw_f", "db_f")}


@pytest.mark.parametrize("kw,want", [
    *[({n: None}, INV) for n in ("u", "w_f", "w_r", "du", "dw_f", "dw_r")],
    ({"dout_f": None, "dout_r": None}, INV),
    ({"dout_f": None}, INV),  # its gradients are asked for
    ({"dout_f": None, "dw_f": None}, INV),
    ({**NO_F, "w_f": None, "b_f": None}, WS),
    (NO_F, WS),  # the parameters of the missing direction are ignored
    ({"b_f": None, "b_r": None, "db_f": None}, WS),
    ({"flags": 1}, INV),
    ({"flags": _lib.FLAG_NO_SILU}, WS),
    ({"K": 3}, UNS),
    ({"K": 0}, INV),
    ({"C": 66}, UNS),
    ({"C": 1 << 23}, UNS),
    ({"batch": 1 << 17}, UNS),
    ({"L": 0}, INV),
    ({"io": 3}, UNS),
    ({"ws": None, "wsb": 1 << 40}, INV),
    ({"ws": fake(40, 8), "wsb": 1 << 40}, INV),
    ({"u": fake(CI["u"], 4), "wsb": 1 << 40}, INV),
    ({"dw_f": fake(CI["dw_f"], 2), "wsb": 1 << 40}, INV),
    ({"du": fake(CI["u"]), "wsb": 1 << 40}, INV),
    ({"dw_f": fake(CI["dw_r"]), "wsb": 1 << 40}, INV),
    ({"db_r": fake(CI["w_f"]), "wsb": 1 << 40}, INV),
    ({"ws": fake(CI["dout_r"]), "wsb": 1 << 40}, INV),
])
def test_conv_bwd_rejects(kw, want):
    assert call("bimamba_conv1d_bidir_bwd", CONV, CONV_SIZES, kw) == want


FWD = ("x", "branch", "post_weight", "gate", "gamma", "beta", "h", "out")
FWD_SIZES = dict(batch=2, L=64, d=64, rows=2, eps=ctypes.c_float(1e-5), io=BF16, flags=0, stream=None)
FI = {n: i for i, n in enumerate(FWD)}


@pytest.mark.parametrize("kw,want", [
    *[({n: None}, INV) for n in ("x", "branch", "h", "out")],
    ({"branch": None, "h": None}, INV),  # post_weight and gate without a branch
    ({"flags": 1}, INV),
    ({"rows": 3}, INV),
    ({"rows": 0}, INV),
    *[({"eps": ctypes.c_float(e)}, INV) for e in (0.0, -1e-5, float("inf"), float("nan"))],
    ({"d": 60}, UNS),
    ({"d": 8200}, UNS),
    ({"d": 0}, INV),
    ({"L": -1}, INV),
    ({"io": 5}, UNS),
    ({"batch": 65536, "rows": 1}, UNS),
    ({"x": fake(FI["x"], 8)}, INV),
    ({"gamma": fake(FI["gamma"], 4)}, INV),
    ({"out": fake(FI["x"])}, INV),
    ({"out": fake(FI["h"], 64)}, INV),
    ({"h": fake(FI["x"], 16)}, INV),  # in place only as a whole
    ({"h": fake(FI["branch"])}, INV),
])
def test_adaln_fwd_rejects(kw, want):
    assert call("bimamba_adaln_fwd", FWD, FWD_SIZES, kw) == want


BWD = ("dout", "dres", "h", "branch", "post_weight", "gate", "gamma", "dx", "dbranch", "dpost_weight", "dgate", "dgamma",
       "dbeta")
BWD_SIZES = dict(batch=2, L=64, d=64, rows=2, eps=ctypes.c_float(1e-5), io=F32, flags=0, ws=fake(40), wsb=0,
                 stream=None)
BI = {n: i for i, n in enumerate(BWD)}


@pytest.mark.parametrize("kw,want", [
    *[({n: None}, INV) for n in ("dout", "h", "branch", "dx", "dbranch", "post_weight")],
    ({"branch": None, "dbranch": None, "post_weight": None, "gate": None, "dpost_weight": None}, INV),  # dgate
    ({"branch": None, "dbranch": None, "post_weight": None, "gate": None, "dpost_weight": None, "dgate": None}, WS),
    ({n: None for n in ("dres", "gate", "gamma", "dpost_weight", "dgamma", "dbeta", "dgate")}, WS),
    ({"flags": 64}, INV),
    ({"rows": 7}, INV),
    ({"d": 12}, UNS),
    ({"ws": None, "wsb": 1 << 40}, INV),
    ({"ws": fake(40, 128), "wsb": 1 << 40}, INV),
    ({"dres": fake(BI["dres"], 8), "wsb": 1 << 40}, INV),
    ({"dx": fake(BI["dout"]), "wsb": 1 << 40}, INV),
    ({"dx": fake(BI["dres"], 16), "wsb": 1 << 40}, INV),
    ({"dbranch": fake(BI["branch"]), "wsb": 1 << 40}, INV),
    ({"dgamma": fake(BI["dbeta"]), "wsb": 1 << 40}, INV),
    ({"ws": fake(BI["h"]), "wsb": 1 << 40}, INV),
])
def test_adaln_bwd_rejects(kw, want):
    assert call("bimamba_adaln_bwd", BWD, BWD_SIZES, kw) == want


@pytest.mark.parametrize("eps", [1e-39, 1e-45])
def test_adaln_rejects_a_subnormal_eps(eps):
    """A reciprocal square root that takes subnormal numbers for zero would make NaN of a row of zeros."""
    e = {"eps": ctypes.c_float(eps)}
    assert call("bimamba_adaln_fwd", FWD, FWD_SIZES, e) == INV
    assert call("bimamba_adaln_bwd", BWD, BWD_SIZES, e) == INV


def test_workspace_bytes_of_the_stream_operators():
    f = _lib.bimamba_conv1d_bidir_bwd_workspace_bytes
    g = _lib.bimamba_adaln_bwd_workspace_bytes
    for bytes_of, bad in ((f, 66), (g, 60)):
        assert bytes_of(2, 100, 64) > 0 and bytes_of(2, 100, 64) % 256 == 0
        assert bytes_of(2, 100, bad) == 0 and bytes_of(0, 100, 64) == 0 and bytes_of(2, 0, 64) == 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    import bidirectional_mamba_selective_amd as bm

    x = torch.zeros(1, 4, 64)
    with pytest.raises((ValueError, RuntimeError)):
        bm.bimamba_scan_bwd(x, x, x, torch.zeros(64, 2), torch.zeros(1, 4, 2), torch.zeros(1, 4, 2), z=x)
    u = torch.zeros(1, 4, 8)
    with pytest.raises((ValueError, RuntimeError)):
        bm.bimamba_conv1d_bidir_bwd(u, None, u, torch.zeros(8, 4))
    with pytest.raises((ValueError, RuntimeError)):
        bm.bimamba_adaln_fwd(u)
    with pytest.raises((ValueError, RuntimeError)):
        bm.bimamba_adaln_bwd(u, None, u)
