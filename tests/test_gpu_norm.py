"""RMS norm with 8-bit outputs through the C ABI against the oracle: the sum with the
residual, the norm in BF16, codes and scales, all bit for bit.

The sum of squares runs in doubles on both sides. Two orders of K additions of terms of
one sign differ by K 2^-53 of the sum at most, so the float r could differ only where
the exact value lies within that of a rounding boundary (K 2^-29 of all values: 1e-5 at
K = 8192, for the worst case of every rounding the same way); the inputs here do not.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from tests.conftest import gpu_available
from tests.gpu_util import DEV, bf16_dev, bf16_host, dev, host, show, sync

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def w():
    import moe_token_amax_amd as w
    return w


def _acts(rng, M, K, spread=0.0):
    x = rng.standard_normal((M, K)) * np.exp(spread * rng.standard_normal((M, 1)))
    x[rng.random((M, K)) < 0.01] *= 20.0
    return O.f32_to_bf16(x.astype(np.float32))


def _weight(rng, K):
    return O.f32_to_bf16((1.0 + 0.2 * rng.standard_normal(K)).astype(np.float32))


def _quant(fmt, n, alg=0):
    if fmt == "int8":
        return O.dynamic_quant_f32(n)
    if fmt == "fp8":
        return O.fp8b.quant_f32(n, alg)
    return O.mx.mx_quant(n, alg)


def _call(w, fmt):
    return {"int8": w.rms_norm_quant, "fp8": w.fp8b_rms_norm_quant, "mx": w.mx_rms_norm_quant}[fmt]


SIZES = [(1, 1), (1, 7168), (2, 8), (3, 37), (5, 511), (4, 512), (4, 513), (7, 1024), (1, 2048), (3, 2049), (2, 8192),
         (2, 8193), (3, 16384), (2, 16385), (2, 33000), (1, 133144), (600, 100), (513, 513), (700, 1030), (520, 2100),
         (514, 4096), (600, 4097), (515, 7168), (513, 8192), (513, 9000), (9000, 64), (4200, 520)]


@pytest.mark.parametrize("fmt", ["int8", "fp8", "mx"])
@pytest.mark.parametrize("M,K", SIZES)
def test_norm_bit_exact(w, M, K, fmt):
    if fmt == "mx":
        K = -(-K // 32) * 32
        if K > 133144:
            K -= 32
    show(f"norm {fmt} {M} x {K}")
    rng = np.random.default_rng(M * 1000 + K)
    x, res, g = _acts(rng, M, K, 1.0), _acts(rng, M, K), _weight(rng, K)
    if M > 2:
        x[1] = 0
        res[1] = 0                       # a row of zeros
        x[2, : K // 2] = 0x8000          # -0
        res[2, : K // 2] = 0x8000
    for with_res in (False, True):
        for alg in ((0,) if fmt == "int8" else (0, 1)):
            kw = {} if fmt == "int8" else {"scale_alg": alg}
            r = bf16_dev(res) if with_res else None
            y = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
            q, s = _call(w, fmt)(bf16_dev(x), bf16_dev(g), 1e-6, residual=r, y=y, **kw)
            sync()
            h, n = O.fused.norm(x, g, 1e-6, res if with_res else None)
            qo, so = _quant(fmt, n, alg)
            if with_res:
                assert np.array_equal(bf16_host(r), h)          # the residual took the sum
            assert np.array_equal(bf16_host(y), O.f32_to_bf16(n))
            assert np.array_equal(host(s), so)
            assert np.array_equal(host(q), qo)


@pytest.mark.parametrize("M,K", [(1, 5), (3, 7168), (600, 1000), (700, 4100), (2, 17000)])
def test_norm_in_bf16_alone(w, M, K):
    rng = np.random.default_rng(K)
    x, res, g = _acts(rng, M, K), _acts(rng, M, K), _weight(rng, K)
    y = w.rms_norm(bf16_dev(x), bf16_dev(g), 1e-5)
    y1 = w.rms_norm(bf16_dev(x), None, 1e-5)
    xd = bf16_dev(x)
    h = torch.empty_like(xd)
    rd = bf16_dev(res)
    y2 = w.rms_norm(xd, bf16_dev(g), 1e-5, residual=rd, h=h)
    y3 = w.rms_norm(xd, bf16_dev(g), 1e-5, residual=rd, h=xd, y=rd)      # the sum into x, the norm into the residual
    sync()
    assert np.array_equal(bf16_host(y), O.f32_to_bf16(O.fused.norm(x, g, 1e-5)[1]))
    assert np.array_equal(bf16_host(y1), O.f32_to_bf16(O.fused.norm(x, None, 1e-5)[1]))
    ho, n = O.fused.norm(x, g, 1e-5, res)
    assert np.array_equal(bf16_host(h), ho) and np.array_equal(bf16_host(y2), O.f32_to_bf16(n))
    assert np.array_equal(bf16_host(xd), ho) and np.array_equal(bf16_host(y3), O.f32_to_bf16(n))


@pytest.mark.parametrize("M,K,lo", [(5, 700, 3), (600, 392, 8), (600, 1001, 5), (3, 16500, 1)])
def test_norm_strided_rows_and_untouched_surroundings(w, M, K, lo):
    rng = np.random.default_rng(K)
    x, res, g = _acts(rng, M, K + 16), _acts(rng, M, K + 16), _weight(rng, K)
    rd = bf16_dev(res)
    room = torch.full((M + 2, K + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    codes = torch.full((M + 2, K + 11), 99, dtype=torch.int8, device=DEV)
    q, s = w.rms_norm_quant(bf16_dev(x)[:, lo:lo + K], bf16_dev(g), residual=rd[:, lo:lo + K], y=room[1:M + 1, 8:8 + K],
                            q=codes[1:M + 1, lo:lo + K])
    sync()
    h, n = O.fused.norm(x[:, lo:lo + K], g, 1e-6, res[:, lo:lo + K])
    qo, so = O.dynamic_quant_f32(n)
    assert np.array_equal(host(q), qo) and np.array_equal(host(s), so)
    got = bf16_host(rd)
    assert np.array_equal(got[:, lo:lo + K], h)
    assert np.array_equal(np.delete(got, np.s_[lo:lo + K], 1), np.delete(res, np.s_[lo:lo + K], 1))
    assert np.array_equal(bf16_host(room[1:M + 1, 8:8 + K]), O.f32_to_bf16(n))
    room[1:M + 1, 8:8 + K] = 7.0
    codes[1:M + 1, lo:lo + K] = 99
    assert (room == 7).all() and (codes == 99).all()


@pytest.mark.parametrize("M,K", [(3, 256), (600, 256), (3, 16640)])
@pytest.mark.parametrize("fmt", ["int8", "fp8", "mx"])
def test_norm_non_finite_values_show(w, fmt, M, K):
    x = np.full((M, K), 0x3F80, np.uint16)
    x[0, 5], x[1, 200] = 0x7F80, 0x7FC0                 # an infinity, a NaN
    y = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    q, s = _call(w, fmt)(bf16_dev(x), None, y=y)
    sync()
    q, s, y = host(q), host(s), y.float().cpu().numpy()
    assert np.isnan(y[0, 5]) and np.isnan(y[1]).all() and (y[2:] == 1).all()
    assert (y[0, np.arange(K) != 5] == 0).all()         # 1 / inf
    if fmt == "int8":
        assert np.isnan(s[:2]).all() and (q[:2] == 0).all() and (q[2:] == 127).all()
    elif fmt == "fp8":
        assert np.isnan(s[0, 0]) and (s[1:, 0] == 0).all() and np.isnan(s[:, 1]).all() and (q[:2] == 0).all()
    else:
        assert s[0, 0] == 255 and (s[0, 1:] == 0).all() and (s[1] == 255).all()
        assert (q[0, :32] == 0x7F).all() and (q[0, 32:] == 0).all() and (q[1] == 0x7F).all()


def test_norm_extremes(w):
    """The largest and the smallest BF16 values: squares that floats do not hold."""
    rng = np.random.default_rng(3)
    base = rng.standard_normal((4, 512))
    sizes = np.array([[1e37], [1e-37], [2.0 ** -133], [1e-20]])
    for eps in (0.0, 1e-6):
        # without eps 1 / 2^-133 is past a float
        x = O.f32_to_bf16((base * sizes)[[0, 1, 3] if eps == 0.0 else [0, 1, 2, 3]].astype(np.float32))
        for fmt in ("int8", "fp8", "mx"):
            q, s = _call(w, fmt)(bf16_dev(x), None, eps)
            sync()
            _, n = O.fused.norm(x, None, eps)
            qo, so = _quant(fmt, n)
            assert np.array_equal(host(s), so) and np.array_equal(host(q), qo)


def test_norm_feeds_every_linear(w):
    """The codes go into the linears as their own quantizers' would."""
    rng = np.random.default_rng(9)
    M, K, N = 40, 256, 64
    x, res, g = _acts(rng, M, K), _acts(rng, M, K), _weight(rng, K)
    _, n = O.fused.norm(x, g, 1e-6, res)
    wi = rng.integers(-127, 128, (N, K)).astype(np.int8)
    ws = rng.uniform(1e-3, 1e-2, N).astype(np.float32)
    q, s = w.rms_norm_quant(bf16_dev(x), bf16_dev(g), residual=bf16_dev(res))
    y = w.linear(q, s, w.prepack_weight(dev(wi)), dev(ws), N)
    sync()
    assert np.array_equal(bf16_host(y), O.linear(*O.dynamic_quant_f32(n), wi, ws)[0])
    cw = O.mx.e4m3_encode(np.clip(rng.standard_normal((N, K)) * 100.0, -448, 448))
    sw = rng.uniform(0.5e-2, 1.5e-2, (1, 2)).astype(np.float32)
    wp = w.fp8b_prepack_weight(dev(cw))
    q, s = w.fp8b_rms_norm_quant(bf16_dev(x), bf16_dev(g), residual=bf16_dev(res))
    y = w.fp8b_linear(q, wp, dev(sw), N, x_scale=s)
    y2 = w.fp8b_linear(dev(O.fp8b.quant_f32(n)[0]), wp, dev(sw), N, x_scale=dev(O.fp8b.quant_f32(n)[1]))
    pm, em = O.mx.mx_quant(rng.standard_normal((N, K)))
    mp = w.mx_prepack_weight(dev(pm), dev(em))
    q, s = w.mx_rms_norm_quant(bf16_dev(x), bf16_dev(g), residual=bf16_dev(res))
    z = w.mx_linear(q, mp, N, x_e8m0=s)
    qo, so = O.mx.mx_quant(n)
    z2 = w.mx_linear(dev(qo), mp, N, x_e8m0=dev(so))
    sync()
    assert np.array_equal(bf16_host(y), bf16_host(y2)) and np.array_equal(bf16_host(z), bf16_host(z2))


def test_norm_captured_and_replayed(w):
    rng = np.random.default_rng(5)
    M, K = 33, 1000
    g = bf16_dev(_weight(rng, K))
    x = bf16_dev(_acts(rng, M, K))
    res = bf16_dev(_acts(rng, M, K))
    h = torch.empty_like(x)
    q = torch.empty((M, K), dtype=torch.int8, device=DEV)
    s = torch.empty((M,), dtype=torch.float32, device=DEV)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        w.rms_norm_quant(x, g, residual=res, h=h, q=q, scale=s)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.rms_norm_quant(x, g, residual=res, h=h, q=q, scale=s)
    for i in range(3):
        xi, ri = _acts(rng, M, K), _acts(rng, M, K)
        x.copy_(bf16_dev(xi))
        res.copy_(bf16_dev(ri))
        q.fill_(1)
        graph.replay()
        sync()
        ho, n = O.fused.norm(xi, O.f32_to_bf16(host(g.float())), 1e-6, ri)
        qo, so = O.dynamic_quant_f32(n)
        assert np.array_equal(bf16_host(h), ho) and np.array_equal(host(q), qo) and np.array_equal(host(s), so)
