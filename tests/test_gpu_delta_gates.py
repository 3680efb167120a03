"""Which tokens the delta rule's gates and their gradients reach, and what infinities in them mean."""
import numpy as np
import pytest

from tests.gpu_util import to_dev, to_host64
from tests.test_gpu_delta import make, upload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("L", [40, 64, 150])
def test_decay_gradients_reach_back_from_the_only_gradient(L, rev):
    """dout at one token: the gates of the tokens met up to it have gradients, the others exactly none, as the oracle."""
    import bidirectional_mamba_selective_amd as bm
    import oracle

    inp, dout, _ = make(1, L, 1, 2, 64, 64, seed=L)
    for at in (0, 1, L // 2, L - 1):
        do = np.zeros_like(dout)
        do[:, at] = dout[:, at]
        g = bm.bimamba_delta_bwd(to_dev(do, "bf16"), **upload(inp), flags=bm.FLAG_REV_ONLY if rev else bm.FLAG_FWD_ONLY)
        want = oracle.delta_bwd(do, inp, rev=rev)
        bound = oracle.delta_bounds(inp, do, rev=rev)
        met = np.arange(L)[::-1] if rev else np.arange(L)
        later = met[list(met).index(at) + 1:]
        for n in ("dt", "b"):
            got = to_host64(g[n])
            assert np.all(np.abs(got - want[n]) <= 2.0 ** -8 * 1.01 * np.abs(want[n]) + bound[n] + 1e-30), (n, at)
            assert np.all(got[:, later] == 0) and np.all(got[:, at] != 0), (n, at)
