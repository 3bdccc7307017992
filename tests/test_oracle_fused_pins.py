"""Pins of the oracle's RMS norm and activations (CPU): hand values and torch in float64."""

from __future__ import annotations

import numpy as np
import torch

import oracle as O

F = O.fused


def _bits(v):
    return O.f32_to_bf16(np.asarray(v, np.float32))


def test_norm_by_hand():
    # sum of squares 4 * 4 over 4 values, eps 0: r = 1/2
    h, n = F.norm(_bits([[2.0, -2.0, 2.0, 2.0]]), _bits([1.0, 2.0, 0.5, 0.0]), 0.0)
    assert n.tolist() == [[1.0, -2.0, 0.5, 0.0]]
    # the residual is added and rounded to BF16 first: 256 + 1 is halfway to 258, even is 256
    h, n = F.norm(_bits([[256.0, 0.0]]), None, 0.0, _bits([[1.0, 0.0]]))
    assert O.bf16_to_f32(h).tolist() == [[256.0, 0.0]]
    assert n[0, 0] == np.float32(256.0) * np.float32(1 / np.sqrt(32768.0))
    # zeros: eps alone
    assert F.norm(_bits([[0.0, 0.0]]), None, 1e-6)[1].tolist() == [[0.0, 0.0]]


def test_norm_against_torch():
    rng = np.random.default_rng(1)
    x, r, w = (_bits(rng.standard_normal(s) * 3) for s in ((7, 1000), (7, 1000), 1000))
    h, n = F.norm(x, w, 1e-5, r)
    t = torch.from_numpy(O.bf16_to_f32(x)) + torch.from_numpy(O.bf16_to_f32(r))
    t = t.to(torch.bfloat16)
    assert np.array_equal(t.float().numpy(), O.bf16_to_f32(h))
    t = t.double()
    want = t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-5) * torch.from_numpy(O.bf16_to_f32(w)).double()
    assert np.allclose(n, want.numpy(), rtol=2.0 ** -22, atol=0)


def test_activations_against_torch():
    v = torch.linspace(-40, 40, 8001, dtype=torch.float64)
    a = {k: F.act64(v.numpy(), k) for k in ("relu", "silu", "gelu", "gelu_tanh")}
    fn = torch.nn.functional
    assert np.array_equal(a["relu"], fn.relu(v).numpy())
    assert np.allclose(a["silu"], fn.silu(v).numpy(), rtol=1e-13, atol=0)
    assert np.allclose(a["gelu"], fn.gelu(v).numpy(), rtol=1e-9, atol=1e-15)
    assert np.allclose(a["gelu_tanh"], fn.gelu(v, approximate="tanh").numpy(), rtol=1e-9, atol=1e-14)
    assert F.act64([2.0], "silu")[0] == 2.0 / (1.0 + np.exp(-2.0))
    # gate and up are the halves, in that order
    assert np.allclose(F.swiglu64(np.array([[2.0, 0.0, 3.0, 5.0]])), [[6.0 / (1 + np.exp(-2.0)), 0.0]])


def test_product64_brute_force():
    rng = np.random.default_rng(2)
    x, w = _bits(rng.standard_normal((3, 5))), _bits(rng.standard_normal((4, 5)))
    y, a = F.product64(x, w)
    xf, wf = O.bf16_to_f32(x), O.bf16_to_f32(w)
    for m in range(3):
        for n in range(4):
            t = [float(xf[m, k]) * float(wf[n, k]) for k in range(5)]
            assert abs(y[m, n] - sum(t)) < 1e-14 and abs(a[m, n] - sum(map(abs, t))) < 1e-14
