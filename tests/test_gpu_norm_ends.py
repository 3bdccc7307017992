"""The norm's ends: the output over its own input, infinities with a weight and a residual,
rows of zeros without an eps."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from tests.conftest import gpu_available
from tests.gpu_util import DEV, bf16_dev, bf16_host, host, show, sync
from tests.test_gpu_norm import _acts, _call, _quant, _weight

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

SIZES = [(2, 32), (4, 544), (3, 2048), (2, 8192), (2, 16416), (600, 96), (520, 2112), (515, 7168), (513, 9024)]


@pytest.fixture(scope="module")
def w():
    import moe_token_amax_amd as w
    return w


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8", "mx"])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_norm_over_its_input(w, M, K, res, fmt):
    """y is x: a row is read whole before any of it is written, or by the thread that writes it."""
    show(f"{M} x {K} residual {res} {fmt}")
    rng = np.random.default_rng(M + K)
    x, g, r = _acts(rng, M, K, 1.0), _weight(rng, K), _acts(rng, M, K) if res else None
    h, n = O.fused.norm(x, g, 1e-6, r)
    xd, rd = bf16_dev(x), bf16_dev(r) if res else None
    if fmt == "bf16":
        w.rms_norm(xd, bf16_dev(g), residual=rd, y=xd)
    else:
        q, s = _call(w, fmt)(xd, bf16_dev(g), residual=rd, y=xd)
        qo, so = _quant(fmt, n)
    sync()
    assert np.array_equal(bf16_host(xd), O.f32_to_bf16(n))
    assert not res or np.array_equal(bf16_host(rd), h)
    if fmt != "bf16":
        assert np.array_equal(host(q), qo) and np.array_equal(host(s), so)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8", "mx"])
@pytest.mark.parametrize("M,K", SIZES)
def test_norm_over_its_sum(w, M, K, fmt):
    """y is h, here the residual: the norm stands there, not the sum."""
    rng = np.random.default_rng(M + K)
    x, g, r = _acts(rng, M, K, 1.0), _weight(rng, K), _acts(rng, M, K)
    _, n = O.fused.norm(x, g, 1e-6, r)
    rd = bf16_dev(r)
    if fmt == "bf16":
        w.rms_norm(bf16_dev(x), bf16_dev(g), residual=rd, y=rd)
    else:
        q, s = _call(w, fmt)(bf16_dev(x), bf16_dev(g), residual=rd, y=rd)
        qo, so = _quant(fmt, n)
    sync()
    assert np.array_equal(bf16_host(rd), O.f32_to_bf16(n))
    if fmt != "bf16":
        assert np.array_equal(host(q), qo) and np.array_equal(host(s), so)


@pytest.mark.parametrize("M,K", SIZES)
def test_infinities_leave_zeros_and_nan(w, M, K):
    """The factor of a row with an infinity is 0: NaN at the infinity, 0 elsewhere, with the
    value's and the weight's sign. x + residual past BF16 is such a row, inf - inf a NaN's."""
    show(f"{M} x {K}")
    x, r = np.full((M, K), 0x3F80, np.uint16), np.zeros((M, K), np.uint16)
    x[:, 1] = 0xBF80                                      # -1
    x[0, 5], r[0, 5] = 0x7F7F, 0x7F7F                     # the largest value twice
    x[1, 7], r[1, 7] = 0x7F80, 0xFF80                     # inf - inf
    rd = bf16_dev(r)
    y = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    got = {}
    for fmt in ("int8", "fp8", "mx"):
        h = torch.empty_like(y)
        got[fmt] = [host(t) for t in _call(w, fmt)(bf16_dev(x), None, residual=rd, h=h, y=y)]
        sync()
        hv, yv = h.float().cpu().numpy(), y.float().cpu().numpy()
        assert np.isinf(hv[0, 5]) and np.isnan(hv[1, 7]) and np.isnan(yv[1]).all()
        assert np.flatnonzero(np.isnan(yv[0])).tolist() == [5] and (np.delete(yv[0], 5) == 0).all()
        assert np.signbit(yv[0, 1]) and not np.signbit(yv[0, 0])
    q, s = got["int8"]
    assert np.isnan(s[:2]).all() and (q[:2] == 0).all()
    q, s = got["fp8"]
    assert np.isnan(s[0, 0]) and (s[1:, 0] == 0).all() and np.isnan(s[:, 1]).all()
    assert ((q[:2] & 0x7F) == 0).all()
    q, s = got["mx"]
    assert s[0, 0] == 255 and (s[0, 1:] == 0).all() and (s[1] == 255).all()
    assert (q[0, :32] == 0x7F).all() and ((q[0, 32:] & 0x7F) == 0).all() and (q[1] == 0x7F).all()


@pytest.mark.parametrize("M,K", [(2, 32), (3, 2048), (2, 16416), (600, 96)])
def test_rows_of_zeros(w, M, K):
    """0 with an eps; NaN without one, as 0 times the infinite factor."""
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    for fmt in ("int8", "fp8", "mx"):
        y = torch.empty_like(x)
        q, s = _call(w, fmt)(x, None, 1e-6, y=y)
        sync()
        assert (y == 0).all() and (q == 0).all() and (s == 0).all()
        q, s = _call(w, fmt)(x, None, 0.0, y=y)
        sync()
        assert torch.isnan(y).all() and (s == 255 if fmt == "mx" else torch.isnan(s)).all()
        assert (q == (0x7F if fmt == "mx" else 0)).all()
