"""The delta rule with many heads: calls that go token by token up to 24 tokens.

A sample of the heads, the first and the last among them, is compared with the oracle."""
import numpy as np
import pytest

from tests.gpu_util import to_host64, torch_mod
from tests.test_gpu_delta import SEQ, close, make, run_fwd, upload

pytestmark = pytest.mark.gpu


def heads_of(inp, sel):
    return {n: None if x is None else x[:, :, sel] if n in SEQ else x[sel] if x.ndim == 1 else x[:, sel]
            for n, x in inp.items()}


@pytest.mark.parametrize("rev", [False, True])
@pytest.mark.parametrize("batch,heads,dk,dv", [(4, 64, 128, 128), (2, 256, 128, 64), (16, 64, 64, 64)])
@pytest.mark.parametrize("L", [17, 24, 25])
def test_tokens_one_by_one_in_wide_calls(batch, heads, dk, dv, L, rev):
    import bidirectional_mamba_selective_amd as bm
    import oracle

    assert (bm.bimamba_delta_fwd_workspace_bytes(batch, L, heads, heads, dk, dv) == 0) == (L <= 24)
    inp, _, _ = make(batch, L, heads, heads, dk, dv, seed=L)
    out, h = run_fwd(bm, upload(inp), rev)
    sel = [0, 1, heads // 2 + 1, heads - 1]
    part = heads_of(inp, sel)
    wout, wh = oracle.delta_fwd(part, rev=rev)
    r = oracle.delta_bounds(part, rev=rev)
    close(to_host64(out)[:, :, sel], wout, r["out"], "out")
    close(to_host64(h)[:, sel], wh, r["h_out"], "h_out", bf16=False)
