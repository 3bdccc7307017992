"""The kernels of the fused linears and of the BF16 products that only large or ragged
sizes reach, each shown to be the one that runs, against float64. Tolerances as in
test_gpu_fused.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.conftest import gpu_available
from tests.gpu_util import DEV, dev, show, sync

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def w():
    import moe_token_amax_amd as w
    return w


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_aligned_prompt_reserves_only_its_output(w, kind):
    """A product without a workspace of the caller's takes no memory that it does not touch."""
    M, N, K = 8192, 4096, 1024
    show(f"{kind} {M} x {N} x {K}")
    if kind == "int8":
        x = torch.ones((M, K), dtype=torch.int8, device=DEV)
        wp = w.prepack_weight(torch.ones((N, K), dtype=torch.int8, device=DEV))
        xs, ws = dev(np.ones(M, np.float32)), dev(np.ones(N, np.float32))
        call = lambda: w.linear_fused(x, xs, wp, ws, N)                                   # noqa: E731
        plan = w.linear_fused_plan(x, N)
    else:
        x = torch.ones((M, K), dtype=torch.bfloat16, device=DEV)
        wp = w.bf16_prepack_weight(torch.ones((N, K), dtype=torch.bfloat16, device=DEV))
        call = lambda: w.bf16_linear(x, wp, N)                                            # noqa: E731
        plan = w.bf16_linear_plan(x, N)
    assert (plan.tile_rows, plan.workspace_bytes) == (256, 0)
    sync()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    y = call()
    sync()
    assert torch.cuda.max_memory_allocated() - before == 2 * M * N
    assert (y == K).all()
