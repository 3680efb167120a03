"""One HIP runtime in a process, whichever of the library and torch is asked for first (no GPU): with two of them, a stream of
torch's is none of the library's and every launch fails."""
import os
import subprocess
import sys

import pytest

from bidirectional_mamba_selective_amd import _lib
from tests.conftest import ROOT

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libbimamba.so not built")

LIBRARY = "import bidirectional_mamba_selective_amd as bm; bm.bimamba_scan_fwd_workspace_bytes(1, 64, 64, 16)"
TORCH = "import torch"
RUNTIMES = "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))"


@pytest.mark.parametrize("order", [(LIBRARY, TORCH), (TORCH, LIBRARY)])
def test_one_hip_runtime(order):
    pytest.importorskip("torch")
    got = subprocess.run([sys.executable, "-c", "\n".join((*order, RUNTIMES))], cwd=ROOT, capture_output=True, text=True,
                         timeout=300, check=True).stdout
    assert int(got) == 1
