"""How the backward entry points cut their work into wavefronts and workgroups, read off their workspace sizes (no GPU).

A launch of more pieces than the chip holds at once leaves a second round in which a few of them run alone."""
import os

import pytest

from bidirectional_mamba_selective_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libbimamba.so not built")

TILE = 16
SCAN_WAVES = 2048  # two wavefronts of the main backward kernel per SIMD, 4 x 256 SIMDs


def scan_chunks(batch, L, d, n):
    """Chunks per sequence: of the workspace's parts, six arrays of d_state rows and two more rows of d channels are kept
    per chunk (every part is a multiple of 256 bytes, so nothing is padded)."""
    row = 4 * d
    tiles = batch * (-(-L // TILE))
    fixed = tiles * row * (2 * n + 1) + n * row + tiles * n * 2 * TILE * 4 * (1 + d // 64)
    per_chunk = batch * row * (6 * n + 2)
    left = _lib.bimamba_scan_bwd_workspace_bytes(batch, L, d, n) - fixed
    assert left > 0 and left % per_chunk == 0, (batch, L, d, n)
    return left // per_chunk


@pytest.mark.parametrize("L", [100, 1024, 2730, 8192, 65536])
def test_scan_bwd_chunks_stay_in_one_round(L):
    """All wavefronts resident at once wherever two chunks per row of channels are, and no fewer chunks than that allows;
    two half-length rounds up to 2048 rows; whole sequences beyond."""
    tiles = -(-L // TILE)
    for d in list(range(64, 8192, 64)) + [61440]:
        for batch in (1, 2, 3, 5, 6, 7, 8, 20, 40):
            rows = batch * d // 64
            got = scan_chunks(batch, L, d, 8)
            if 2 * rows <= SCAN_WAVES:
                assert rows * got <= SCAN_WAVES, (batch, L, d)
                want = SCAN_WAVES // rows
            else:
                want = 2 if rows < SCAN_WAVES else 1
            per_chunk = -(-tiles // want)
            assert got == -(-tiles // per_chunk), (batch, L, d)
