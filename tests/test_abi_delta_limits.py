"""The longest sequences that the delta rule's calls take, on the host (no GPU): a grid dimension holds fewer than 2^32 threads,
the chunks' workgroups have 256 of them in the forward call and 512 in the backward one."""
import os

import pytest

from bidirectional_mamba_selective_amd import _lib
from tests.test_abi_bwd import call
from tests.test_abi_delta import BWD, FWD, SIZES, UNS, WS

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libbimamba.so not built")

ONE = {"batch": 1, "hk": 1, "heads": 1, "dv": 64}


@pytest.mark.parametrize("L,fwd,bwd", [(5 * 10 ** 8, WS, WS), (2 ** 29, WS, UNS), (10 ** 9, WS, UNS), (10 ** 9 + 1, UNS, UNS)])
def test_longest_sequences(L, fwd, bwd):
    lib = _lib.load()
    assert call("bimamba_delta_fwd", FWD, SIZES, {**ONE, "L": L}) == fwd
    assert call("bimamba_delta_bwd", BWD, SIZES, {**ONE, "L": L}) == bwd
    assert (lib.bimamba_delta_fwd_workspace_bytes(1, L, 1, 1, 64, 64) > 0) == (fwd == WS)
    assert (lib.bimamba_delta_bwd_workspace_bytes(1, L, 1, 1, 64, 64) > 0) == (bwd == WS)
    if bwd == WS:
        assert (L + 63) // 64 * 512 < 2 ** 32
    if fwd == WS:
        assert (L + 63) // 64 * 256 < 2 ** 32
