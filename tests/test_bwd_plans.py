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


def adaln_workgroups(batch, L, d):
    """Workgroups of the backward pass: each keeps four column sums per row group (the workspace is padded to 256 bytes)."""
    waves = 1
    while waves * 512 < d:
        waves *= 2
    bytes_of = 4 * 4 * d * (4 if waves == 1 else 1)
    return _lib.bimamba_adaln_bwd_workspace_bytes(batch, L, d) // bytes_of, waves


@pytest.mark.parametrize("d", [64, 512, 1024, 1928, 2048, 4096, 8192])
def test_adaln_bwd_workgroups_stay_in_one_round(d):
    """No more workgroups than 256 CUs hold (12 wavefronts each, whole workgroups), except where there are more
    sequences than that: then one a sequence."""
    for L in (1, 7, 100, 1001, 2048, 8192):
        for batch in list(range(1, 13)) + [40, 100, 129, 200, 257, 400, 512, 1000, 2000]:
            got, waves = adaln_workgroups(batch, L, d)
            per_wg = 4 if waves == 1 else waves
            resident = 256 * max(1, 12 // per_wg)
            assert got % batch == 0
            assert got <= resident or got == batch, (batch, L, d, got)
            # no fewer than the rows and that limit allow
            rows = -(-L // max(1, resident // batch))
            rows += -rows % (4 if waves == 1 else 1)
            assert got == batch * -(-L // rows), (batch, L, d, got)


def scan_fits(batch, L, d, n):
    """The limits that include/bimamba.h states for bimamba_scan_bwd beside those of the forward call."""
    tokens = -(-L // TILE) * TILE
    return 2 * batch * n * tokens + 4 * (n + 2) * d + 1024 < 2 ** 32 and batch * n * d + 256 < 2 ** 32


@pytest.mark.parametrize("batch,L,d,n,fits", [
    (2, 1073741360, 64, 1, True),
    (2, 1073741361, 64, 1, False),   # rounded up to 1073741376: 2 * 1 * that is still below 2^31
    (1, 131857920, 1 << 20, 16, True),
    (1, 131900000, 1 << 20, 16, False),  # the channels' term alone decides
    (8, 16, 33554368, 16, True),
    (9, 16, 33554368, 16, False),
])
def test_scan_bwd_limits_are_the_documented_ones(batch, L, d, n, fits):
    assert scan_fits(batch, L, d, n) == fits
    assert (_lib.bimamba_scan_bwd_workspace_bytes(batch, L, d, n) > 0) == fits


def test_the_header_states_the_limits():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bimamba.h")
    with open(path) as f:
        text = " ".join(line.strip(" *\n") for line in f)
    assert "2 * batch * d_state * (seqlen rounded up to 16) + 4 * (d_state + 2) * d_inner + 1024" in text
    assert "batch * d_state * d_inner + 256" in text
