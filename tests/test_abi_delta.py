"""Refusals of the delta rule, the 8-bit norm and the 8-bit projection on the host, before any HIP call (no GPU), and the
workspaces they ask for.

The pointer values are never dereferenced: every call here fails validation."""
import os

import pytest

from bidirectional_mamba_selective_amd import _lib
from tests.test_abi_bwd import call, fake

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libbimamba.so not built")

INV, UNS, WS = _lib.BIMAMBA_ERR_INVALID_ARGUMENT, _lib.BIMAMBA_ERR_UNSUPPORTED, _lib.BIMAMBA_ERR_WORKSPACE_TOO_SMALL
BF16, F32 = _lib.BIMAMBA_BF16, _lib.BIMAMBA_F32
INF = float("inf")
BIG = {"wsb": 1 << 40}

FWD = ("q", "k", "v", "dt", "A", "b", "dt_bias", "h_in", "h_out", "out")
SIZES = dict(batch=2, L=100, hk=2, heads=4, dk=64, dv=128, scale=0.1, io=BF16, flags=_lib.FLAG_FWD_ONLY, ws=fake(40),
             wsb=0, stream=None)
I = {n: i for i, n in enumerate(FWD)}

SHAPES = [
    *[({n: 0}, INV) for n in ("batch", "L", "hk", "heads", "dk", "dv")],
    ({"heads": -4}, INV),
    ({"hk": 3}, INV),
    ({"dk": 32}, UNS),
    ({"dk": 256}, UNS),
    ({"dv": 96}, UNS),
    ({"io": F32}, UNS),
    ({"io": 7}, UNS),
    ({"batch": 65536}, UNS),
    ({"heads": 65536}, UNS),
    ({"batch": 1 << 12, "heads": 1 << 12}, UNS),
    ({"L": 1 << 31}, UNS),
    ({"flags": 0}, INV),
    ({"flags": _lib.FLAG_FWD_ONLY | _lib.FLAG_REV_ONLY}, INV),
    ({"flags": _lib.FLAG_FWD_ONLY | _lib.FLAG_NO_GATE}, INV),
    ({"scale": INF}, INV),
    ({"scale": float("nan")}, INV),
    ({}, WS),
    ({"dt_bias": None, "h_in": None}, WS),  # optional: gets to the workspace
    ({"flags": _lib.FLAG_REV_ONLY}, WS),
    ({"ws": None, **BIG}, INV),
    ({"ws": fake(40, 64), **BIG}, INV),
]


@pytest.mark.parametrize("kw,want", SHAPES + [
    *[({n: None}, INV) for n in ("q", "k", "v", "dt", "A", "b", "out")],
    ({"h_out": None}, WS),
    ({"q": fake(I["q"], 8), **BIG}, INV),
    ({"h_in": fake(I["h_in"], 4), **BIG}, INV),
    ({"dt": fake(I["dt"], 1), **BIG}, INV),
    ({"A": fake(I["A"], 2), **BIG}, INV),
    ({"out": fake(I["v"]), **BIG}, INV),
    ({"h_out": fake(I["h_in"], 64), **BIG}, INV),   # over part of the state it starts from
    ({"h_out": fake(I["out"], 128), **BIG}, INV),
    ({"ws": fake(I["k"]), **BIG}, INV),
    ({"out": fake(40, 4096), **BIG}, INV),
    ({"L": 9, "out": fake(I["q"])}, INV),           # the call without a workspace checks the rest
    ({"L": 9, "h_out": fake(I["b"])}, INV),
])
def test_delta_fwd_rejects(kw, want):
    assert call("bimamba_delta_fwd", FWD, SIZES, kw) == want


BWD = ("dout", "q", "k", "v", "dt", "A", "b", "dt_bias", "h_in", "dh_out", "dq", "dk_", "dv_", "ddt", "dA", "db",
       "ddt_bias", "dh_in")
B = {n: i for i, n in enumerate(BWD)}


@pytest.mark.parametrize("kw,want", SHAPES + [
    *[({n: None}, INV) for n in ("dout", "q", "k", "v", "dt", "A", "b", "dq", "dk_", "dv_", "ddt", "dA", "db")],
    ({"ddt_bias": None, "dh_in": None, "dh_out": None}, WS),
    ({"L": 1}, WS),                                 # every length needs it
    ({"dq": fake(B["dq"], 8), **BIG}, INV),
    ({"dA": fake(B["dA"], 2), **BIG}, INV),
    ({"db": fake(B["db"], 1), **BIG}, INV),
    ({"dh_out": fake(B["dh_out"], 4), **BIG}, INV),
    ({"dq": fake(B["q"]), **BIG}, INV),
    ({"dq": fake(B["dk_"], 16), **BIG}, INV),
    ({"dh_in": fake(B["h_in"]), **BIG}, INV),
    ({"dh_in": fake(B["dh_out"], 64), **BIG}, INV),
    ({"ws": fake(B["dout"]), **BIG}, INV),
    ({"dv_": fake(40, 8192), **BIG}, INV),
])
def test_delta_bwd_rejects(kw, want):
    assert call("bimamba_delta_bwd", BWD, SIZES, kw) == want


def test_delta_workspaces():
    lib = _lib.load()
    f, b = lib.bimamba_delta_fwd_workspace_bytes, lib.bimamba_delta_bwd_workspace_bytes
    for L in (1, 16):
        assert f(3, L, 2, 4, 128, 64) == 0 and b(3, L, 2, 4, 128, 64) > 0
    for bad in ((0, 9, 1, 1, 64, 64), (1, 100, 2, 3, 64, 64), (1, 100, 1, 1, 96, 64), (1 << 16, 100, 1, 1, 64, 64)):
        assert f(*bad) == 0 and b(*bad) == 0
    # forward: bounded however long the sequence, up to eight chunks of every head; backward: by chunk
    assert f(1, 1 << 20, 32, 32, 128, 128) < 128 << 20
    assert f(1, 1 << 20, 32, 32, 128, 128) % 256 == 0 and b(1, 1 << 14, 32, 32, 128, 128) % 256 == 0
    per_chunk = b(1, 64 * 400, 2, 4, 64, 64) - b(1, 64 * 200, 2, 4, 64, 64)
    assert abs(b(1, 64 * 600, 2, 4, 64, 64) - b(1, 64 * 400, 2, 4, 64, 64) - per_chunk) <= 512


ADA = ("x", "branch", "post_weight", "gate", "gamma", "beta", "h", "out", "scales")
ADA_SIZES = dict(batch=2, L=10, d=256, rows=2, eps=1e-5, io=BF16, flags=0, stream=None)
A = {n: i for i, n in enumerate(ADA)}


@pytest.mark.parametrize("kw,want", [
    *[({n: 0}, INV) for n in ("batch", "L", "d")],
    ({"d": 192}, UNS),
    ({"d": 8320}, UNS),
    ({"io": 3}, UNS),
    ({"rows": 3}, INV),
    ({"eps": 0.0}, INV),
    ({"flags": 2}, INV),
    *[({n: None}, INV) for n in ("x", "out", "scales", "h")],
    ({"branch": None}, INV),
    ({"x": fake(A["x"], 8)}, INV),
    ({"scales": fake(A["scales"], 2)}, INV),
    ({"out": fake(A["x"], 256)}, INV),
    ({"scales": fake(A["out"], 64)}, INV),
    ({"scales": fake(A["gamma"])}, INV),
    ({"h": fake(A["x"], 16)}, INV),
])
def test_adaln_fp8_rejects(kw, want):
    assert call("bimamba_adaln_fwd_fp8", ADA, ADA_SIZES, kw) == want


PROJ = ("x", "xs", "w", "ws_", "out")
PROJ_SIZES = dict(rows=100, n=264, k=256, out_dtype=BF16, stream=None)
P = {n: i for i, n in enumerate(PROJ)}


@pytest.mark.parametrize("kw,want", [
    *[({n: 0}, INV) for n in ("rows", "n", "k")],
    ({"rows": -1}, INV),
    ({"n": 260}, UNS),
    ({"k": 192}, UNS),
    ({"n": (1 << 22) + 8}, UNS),
    ({"k": (1 << 22) + 128}, UNS),
    ({"rows": (1 << 31) + 1}, UNS),
    ({"rows": 1 << 24, "n": 1 << 14}, UNS),
    ({"out_dtype": 2}, UNS),
    *[({n: None}, INV) for n in PROJ],
    ({"x": fake(P["x"], 8)}, INV),
    ({"w": fake(P["w"], 8)}, INV),
    ({"out": fake(P["out"], 8)}, INV),
    ({"xs": fake(P["xs"], 2)}, INV),
    ({"out": fake(P["w"])}, INV),
    ({"out": fake(P["xs"])}, INV),
])
def test_proj_rejects(kw, want):
    assert call("bimamba_proj_fp8", PROJ, PROJ_SIZES, kw) == want
