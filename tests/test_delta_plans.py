"""Which way the delta rule's forward call goes, read off its workspace sizes (no GPU)."""
import os

import pytest

from bidirectional_mamba_selective_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libbimamba.so not built")


@pytest.mark.parametrize("batch,heads,dk,dv,tokens", [
    (1, 1, 64, 64, 16), (1, 32, 128, 128, 16), (4, 32, 128, 128, 16), (3, 85, 128, 128, 16), (4, 64, 128, 128, 24),
    (16, 32, 128, 128, 24), (511, 1, 64, 128, 16), (512, 1, 128, 64, 24), (31, 33, 64, 64, 16), (32, 32, 64, 64, 24)])
def test_token_by_token_without_a_workspace(batch, heads, dk, dv, tokens):
    """Up to 16 tokens, 24 where the states hold 2^22 values."""
    need = lambda L: _lib.bimamba_delta_fwd_workspace_bytes(batch, L, heads, heads, dk, dv)  # noqa: E731
    assert tokens == (24 if batch * heads * dk * dv >= 1 << 22 else 16)
    assert all(need(L) == 0 for L in range(1, tokens + 1))
    assert all(need(L) > 0 for L in (tokens + 1, 25, 64, 65))
