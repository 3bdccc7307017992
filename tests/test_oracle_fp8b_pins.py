"""Pins of the block-scaled FP8 and router oracle (CPU only)."""

from __future__ import annotations

import numpy as np
import torch

import oracle as O

F = O.fp8b


def _bits(x):
    return O.f32_to_bf16(np.asarray(x, np.float32))


def test_quant_hand_block():
    x = np.zeros((1, 130), np.float32)
    x[0, :5] = [448.0, -224.0, 1.0, 17.0, 19.0]   # scale 1: 17 and 19 are ties between 16, 18, 20
    x[0, 128] = 0.875
    q, s = F.quant(_bits(x))
    assert q.shape == (1, 256) and s.shape == (2, 1)
    assert s[0, 0] == 1.0 and s[1, 0] == np.float32(0.875) / np.float32(448.0)
    assert list(O.mx.e4m3_decode(q[0, :5])) == [448.0, -224.0, 1.0, 16.0, 20.0]
    assert q[0, 128] == 0x7E and not q[0, 129:].any()


def test_quant_zero_block_and_power_of_two_scale():
    x = np.zeros((2, 256), np.float32)
    x[0, 0] = 448.0 * 1.25
    x[1, 200] = 448.0
    q, s = F.quant(_bits(x), scale_alg=1)
    assert s[0, 0] == 2.0 and s[1, 0] == 0.0 and s[1, 1] == 1.0 and s[0, 1] == 0.0
    # 560 / 2 = 280; E4M3 steps by 32 from 256: 288 is nearest
    assert O.mx.e4m3_decode(q[0, 0]) == 288.0 and not q[1, :128].any()


def test_quant_codes_against_torch():
    rng = np.random.default_rng(1)
    b = _bits(rng.standard_normal((7, 384)) * np.exp(rng.uniform(-6, 6, (7, 384))))
    q, s = F.quant(b)
    v = torch.from_numpy(O.bf16_to_f32(b)).view(7, 3, 128)
    t = (v / torch.from_numpy(s.T.copy())[..., None]).clamp(-448, 448)
    assert np.array_equal(t.to(torch.float8_e4m3fn).view(torch.uint8).view(7, 384).numpy(), q)


def test_product_by_loops():
    rng = np.random.default_rng(2)
    M, N, K = 3, 130, 200
    q, sx = F.quant(_bits(rng.standard_normal((M, K))))
    w = O.mx.e4m3_encode(rng.standard_normal((N, K)) * 50)
    sw = rng.uniform(0.5, 2, (2, 2)).astype(np.float32)
    y = F.product64(q, sx, w, sw)
    for m, n in ((0, 0), (1, 127), (2, 128), (2, 129)):
        want = sum(float(O.mx.e4m3_decode(q[m, k])) * float(sx[k // 128, m]) * float(O.mx.e4m3_decode(w[n, k])) *
                   float(sw[n // 128, k // 128]) for k in range(K))
        assert abs(y[m, n] - want) <= 1e-12 * max(1.0, abs(want))


def test_cut_bound_hand_group():
    # one group holds 1 * 256 and 7 products of 1 * 1: E = 8, bound 7 * 2^-5 per unit scale
    q = np.full((1, 128), 0x00, np.uint8)
    q[0, :8] = 0x38
    w = np.zeros((1, 128), np.uint8)
    w[0, 0], w[0, 1:8] = 0x78, 0x38
    assert F.cut_bound(q, np.ones((1, 1)), w, np.ones((1, 1)))[0, 0] == 7.0 * 2.0 ** (8 - 13)


def test_gate_hand():
    l = np.array([[0.0, 2.0, 2.0, -np.inf, 1.0, np.nan]])
    ids, w = F.gate(l, 4, scoring="sigmoid")
    assert ids[0].tolist() == [1, 2, 4, 0]                    # equal keys: the lower index first
    assert abs(w.sum() - 1) < 1e-15
    ids, w = F.gate(l, 6, scoring="softmax", renormalize=False, scale=2.0)
    assert ids[0].tolist() == [1, 2, 4, 0, -1, -1] and w[0, 4] == 0 and abs(w.sum() - 2) < 1e-15
    # the bias moves the choice, not the weight
    ids, w = F.gate(l, 1, bias=[0, 0, 0, 9, 0.3, 9], scoring="sigmoid", renormalize=False)
    assert ids[0, 0] == 4 and abs(w[0, 0] - 1 / (1 + np.exp(-1.0))) < 1e-15
    # groups of 2: marks 0.5 + s(2), s(2) alone, s(1) alone
    ids, _ = F.gate(l, 2, scoring="sigmoid", n_group=3, topk_group=1)
    assert ids[0].tolist() == [1, 0]
    ids, w = F.gate(np.full((1, 4), -np.inf), 2, scoring="softmax", n_group=2, topk_group=1)
    assert ids[0].tolist() == [-1, -1] and not w.any()


def test_gate_against_torch():
    rng = np.random.default_rng(3)
    l = rng.standard_normal((50, 32))
    b = 0.1 * rng.standard_normal(32)
    ids, w = F.gate(l, 5, bias=b, scoring="sigmoid", n_group=4, topk_group=2)
    s = torch.sigmoid(torch.from_numpy(l))
    key = s + torch.from_numpy(b)
    mark = key.view(50, 4, 8).topk(2, 2)[0].sum(2)
    keep = torch.zeros(50, 4).scatter_(1, mark.topk(2, 1)[1], 1.0)
    key = key.view(50, 4, 8).masked_fill(keep[..., None] == 0, -9.0).view(50, 32)
    top = key.topk(5, 1)[1]
    assert np.array_equal(top.numpy(), ids)
    p = s.gather(1, top)
    assert np.allclose((p / p.sum(1, keepdim=True)).numpy(), w, rtol=1e-14)


def test_quant_infinity_and_nan():
    x = np.zeros((3, 128), np.uint16)
    x[0, :3] = [0x7F80, 0x3F80, 0xBF80]                       # inf, 1, -1
    x[1, :2] = [0x3F80, 0xFF80]
    x[2, :2] = [0x7FC0, 0x3F80]
    for alg in (0, 1):
        q, s = F.quant(x, 0, alg)
        assert np.isinf(s[0, :2]).all() and np.isnan(s[0, 2])
        assert q[0, 0] == 0x7F and q[1, 1] == 0x7F and not (q[0, 1:] & 0x7F).any() and not q[1, 0] and not q[2].any()
