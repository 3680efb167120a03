"""How the delta rule's calls are cut, read off their workspace sizes and the plan's header (no GPU)."""
import os
import shutil
import subprocess

import pytest

from bidirectional_mamba_selective_amd import _lib
from tests.conftest import ROOT

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


def test_two_tiles_a_workgroup_from_256_tiles(tmp_path):
    """walk_tiles, compiled on its own: what the tests of two-tile walks take for granted of their sizes."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "tiles.cpp", tmp_path / "tiles"
    src.write_text('#include <cstdio>\n#include "delta_plan.h"\n'
                   "int main() { for (int h = 1; h < 200; ++h) for (int v = 64; v <= 128; v += 64)\n"
                   '  std::printf("%d %d %d\\n", h, v, bimamba::delta::walk_tiles(h, v)); }\n')
    csrc = os.path.join(ROOT, "bidirectional_mamba_selective_amd", "csrc")
    subprocess.run([gxx, "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True, timeout=120)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=60).stdout.splitlines():
        heads, dv, tiles = map(int, line.split())
        assert tiles == (2 if heads * dv // 16 > 256 else 1), line
