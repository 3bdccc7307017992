"""Products with bias, activation and residual in their epilogue, and the BF16 products,
dense and grouped by expert, through the C ABI against float64.

An output is held to 2^-8 (|y| + d) + d of its float64 value y (BF16: half a step; fp32
outputs: 2^-24 in its place), with d the fp32 errors in front of the output's rounding:
  v   the value in front of the activation. INT8: the sum is exact, its conversion, two
      products and the bias are four roundings: dv = 4 2^-24 (|acc x_s w_s| + |b|). FP8: the
      linear's own bound, cuts and (18 + B) 2^-23 A (A: the sum of absolute products, |b|
      among them). BF16: exact products; their fp32 sum within 6 sqrt(K) 2^-24 A
      (probabilistic, lambda = 6) and the bias's addition 2^-24 A more.
  act |act'| <= 1.13 for every activation here (the largest slope, of GELU), so 1.13 dv;
      and its own evaluation: v sigma(t) with t = v (silu) or within 4 2^-24 |t| of
      2 sqrt(2/pi) (v + 0.044715 v^3): the exponent's product and constant 2 2^-24 |t|, the
      exponential and the reciprocal 2^-23 each, the addition and the product 2^-24 each:
      at most (6 |t| + 8) 2^-24 |act| (|t| <= 90 before the result vanishes, so at most
      548 2^-24; a vanished result is below 90 e^-87 < 2^-118). GELU: erfc within 1.5e-7,
      halved, and roundings of 1 - tail: 2^-21 |v|.
      SwiGLU: |d(silu u)| <= 1.1 dg |u| + |silu| du + (6 |g| + 9) 2^-24 |silu u|.
  residual: one addition, 2^-24 (|act| + |r|).
"""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle as O
from tests.conftest import gpu_available
from tests.gpu_util import DEV, bf16_dev, bf16_host, dev, host, show, sync

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

F = O.fused
U = 2.0 ** -24


@pytest.fixture(scope="module")
def w():
    import moe_token_amax_amd as w
    return w


def _act_id(w, act):
    return getattr(w, "ACT_" + act.upper())


def _acts(rng, M, K, spread=0.0):
    x = rng.standard_normal((M, K)) * np.exp(spread * rng.standard_normal((M, 1)))
    x[rng.random((M, K)) < 0.01] *= 20.0
    return O.f32_to_bf16(x.astype(np.float32))


def _bf16(rng, *shape, scale=1.0):
    return O.f32_to_bf16((scale * rng.standard_normal(shape)).astype(np.float32))


def _f64(bits):
    return O.bf16_to_f32(bits).astype(np.float64)


def _epilogue(v, dv, act, res_bits=None):
    """(y, d) behind v with error dv."""
    if act == "swiglu":
        h = v.shape[1] // 2
        s, u = F.act64(v[:, :h], "silu"), v[:, h:]
        y = s * u
        d = 1.1 * dv[:, :h] * (np.abs(u) + dv[:, h:]) + np.abs(s) * dv[:, h:] + \
            (6 * np.minimum(np.abs(v[:, :h]), 90) + 9) * U * np.abs(y) + 2.0 ** -118 * np.abs(u)
    else:
        y = F.act64(v, act)
        t = {"silu": np.abs(v), "gelu_tanh": np.abs(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))}.get(act)
        own = 0.0
        if t is not None:
            own = (6 * np.minimum(t, 90) + 8) * U * np.abs(y) + 2.0 ** -118
        elif act == "gelu":
            own = 2.0 ** -21 * np.abs(v)
        d = 1.13 * dv + own
    if res_bits is not None:
        r = _f64(res_bits)
        d = d + U * (np.abs(y) + np.abs(r) + d)
        y = y + r
    return y, d


def _hold(got, y, d, what="", f32=False):
    off = np.abs((host(got).astype(np.float64) if f32 else _f64(bf16_host(got))) - y)
    tol = (2.0 ** -24 if f32 else 2.0 ** -8) * (np.abs(y) + d) + d + 1e-38
    bad = np.argwhere(~(off <= tol))
    assert bad.size == 0, f"{what}: {len(bad)} of {off.size}, first {bad[0].tolist()}: off {off[tuple(bad[0])]:.4g} " \
                          f"tol {tol[tuple(bad[0])]:.4g} y {y[tuple(bad[0])]:.4g}"
    return float((off / tol).max()) if off.size else 0.0


# ------------------------------------------------------------------ INT8
def _int8_operands(rng, M, N, K):
    q, s = O.dynamic_quant(_acts(rng, M, K, 1.0))
    wi = rng.integers(-127, 128, (N, K)).astype(np.int8)
    ws = (rng.uniform(0.5, 1.5, N) / (73.0 * math.sqrt(K))).astype(np.float32)
    return q, s, wi, ws


SIZES = [  # M, N, K
    (1, 16, 128), (1, 1, 16), (1, 5, 3), (2, 17, 65), (4, 256, 1024), (16, 100, 300), (17, 128, 256), (33, 130, 2000),
    (3, 40, 2048), (4, 48, 7168), (16, 64, 2050), (40, 40, 4200), (64, 512, 512), (65, 48, 384), (100, 333, 1000),
    (128, 256, 640), (200, 272, 128), (257, 300, 200), (300, 520, 1150), (1, 47, 8000), (1, 4200, 200), (1, 4101, 2601),
    (64, 4000, 300), (64, 4090, 3000), (33, 2100, 3903), (70, 2100, 1300), (100, 4100, 700), (130, 4100, 100),
    (1100, 300, 640), (1100, 270, 333), (1500, 64, 64), (1300, 130, 129)]


@pytest.mark.parametrize("act,bias,res", [("none", False, True), ("silu", True, True), ("gelu_tanh", True, False),
                                          ("gelu", False, True), ("relu", True, True)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_int8_linear(w, M, N, K, act, bias, res):
    show(f"int8 {M} x {N} x {K} {act} bias {bias} residual {res}")
    rng = np.random.default_rng(M + 7 * N + 11 * K)
    q, s, wi, ws = _int8_operands(rng, M, N, K)
    b, r = (_bf16(rng, N, scale=0.3) if bias else None), (_bf16(rng, M, N) if res else None)
    y = w.linear_fused(dev(q), dev(s), w.prepack_weight(dev(wi)), dev(ws), N, bias=bf16_dev(b) if bias else None,
                       act=_act_id(w, act), residual=bf16_dev(r) if res else None)
    sync()
    v = O.linear_ref64(O.int8_matmul_acc(q, wi), s, ws)
    dv = 4 * U * np.abs(v)
    if bias:
        v, dv = v + _f64(b), dv + 4 * U * np.abs(_f64(b))
    _hold(y, *_epilogue(v, dv, act, r), f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", SIZES)
def test_int8_without_activation_is_the_linear(w, M, N, K):
    rng = np.random.default_rng(M + 3 * N + 5 * K)
    q, s, wi, ws = _int8_operands(rng, M, N, K)
    b = _bf16(rng, N)
    wp = w.prepack_weight(dev(wi))
    y = w.linear_fused(dev(q), dev(s), wp, dev(ws), N, bias=bf16_dev(b))
    sync()
    assert np.array_equal(bf16_host(y), O.linear(q, s, wi, ws, b)[0])


# ------------------------------------------------------------------ FP8
@pytest.mark.parametrize("act,bias,res", [("none", False, True), ("silu", True, True), ("gelu_tanh", True, False),
                                          ("gelu", False, True), ("relu", True, True)])
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (1, 4200, 200), (2, 17, 65), (16, 100, 300), (17, 128, 256), (33, 130, 2000),
                                   (64, 512, 512), (64, 4000, 300), (128, 256, 640), (300, 520, 1152), (50, 7100, 2100),
                                   (130, 16400, 100), (1, 47, 8000), (100, 4100, 700)])
def test_fp8_linear(w, M, N, K, act, bias, res):
    show(f"fp8 {M} x {N} x {K} {act} bias {bias} residual {res}")
    rng = np.random.default_rng(M + 7 * N + 11 * K)
    x = _acts(rng, M, K, 1.0)
    cw = O.mx.e4m3_encode(np.clip(rng.standard_normal((N, K)) * 100.0, -448, 448))
    sw = (rng.uniform(0.5, 1.5, (O.fp8b.blocks(N), O.fp8b.blocks(K))) / (100 * math.sqrt(K))).astype(np.float32)
    b, r = (_bf16(rng, N, scale=0.3) if bias else None), (_bf16(rng, M, N) if res else None)
    kw = dict(bias=bf16_dev(b) if bias else None, act=_act_id(w, act))
    wp, xd, swd = w.fp8b_prepack_weight(dev(cw)), bf16_dev(x), dev(sw)
    rd = bf16_dev(r) if res else None
    y = w.fp8b_linear_fused(xd, wp, swd, N, residual=rd, **kw)
    qd, sd = w.fp8b_quant(xd)
    y2 = torch.empty_like(y) if rd is None else rd.clone()
    w.fp8b_linear_fused(qd, wp, swd, N, x_scale=sd, K=K, residual=None if rd is None else y2, y=y2, **kw)   # in place
    sync()
    assert np.array_equal(bf16_host(y), bf16_host(y2))
    q, s = O.fp8b.quant(x)
    v = O.fp8b.product64(q, s, cw, sw, b)
    A = np.abs(O.fp8b.dequant(q, s)) @ np.abs(O.fp8b.weight_dequant(cw, sw)).T
    if bias:
        A = A + np.abs(_f64(b))
    dv = O.fp8b.cut_bound(q, s, cw, sw) + (18 + O.fp8b.blocks(K)) * 2.0 ** -23 * A
    _hold(y, *_epilogue(v, dv, act, r), f"{M}x{N}x{K}")


def test_fp8_wide_tiles(w):
    """Tiles that a workgroup walks over, sampled rows."""
    M, N, K = 4100, 4100, 256
    rng = np.random.default_rng(1)
    x = _acts(rng, M, K, 1.0)
    cw = O.mx.e4m3_encode(np.clip(rng.standard_normal((N, K)) * 100.0, -448, 448))
    sw = (rng.uniform(0.5, 1.5, (O.fp8b.blocks(N), 2)) / (100 * math.sqrt(K))).astype(np.float32)
    b, r = _bf16(rng, N, scale=0.3), _bf16(rng, M, N)
    y = w.fp8b_linear_fused(bf16_dev(x), w.fp8b_prepack_weight(dev(cw)), dev(sw), N, bias=bf16_dev(b), act=w.ACT_SILU,
                            residual=bf16_dev(r))
    sync()
    pick = np.r_[0:3, 127:130, 254:258, M - 3:M]
    q, s = O.fp8b.quant(x[pick])
    v = O.fp8b.product64(q, s, cw, sw, b)
    A = np.abs(O.fp8b.dequant(q, s)) @ np.abs(O.fp8b.weight_dequant(cw, sw)).T + np.abs(_f64(b))
    dv = O.fp8b.cut_bound(q, s, cw, sw) + 20 * 2.0 ** -23 * A
    _hold(y[torch.from_numpy(pick).to(DEV)], *_epilogue(v, dv, "silu", r[pick]))


# ------------------------------------------------------------------ BF16
def _bf16_value(x, wt, b=None):
    v, A = F.product64(x, wt)
    dv = 6 * math.sqrt(x.shape[1]) * U * A
    if b is not None:
        v, dv = v + _f64(b), dv + U * (A + np.abs(_f64(b)))
    return v, dv


@pytest.mark.parametrize("act,bias,res,f32", [("none", False, False, True), ("none", True, True, False),
                                              ("swiglu", True, True, False), ("swiglu", False, False, True),
                                              ("silu", True, False, False), ("gelu", False, True, True),
                                              ("gelu_tanh", True, True, False), ("relu", False, True, False)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_bf16_linear(w, M, N, K, act, bias, res, f32):
    if act == "swiglu":
        N += N % 2
    width = N // 2 if act == "swiglu" else N
    show(f"bf16 {M} x {N} x {K} {act} bias {bias} residual {res} f32 {f32}")
    rng = np.random.default_rng(M + 7 * N + 11 * K)
    x, wt = _acts(rng, M, K, 1.0), _bf16(rng, N, K, scale=1 / math.sqrt(K))
    b, r = (_bf16(rng, N, scale=0.3) if bias else None), (_bf16(rng, M, width) if res else None)
    y = w.bf16_linear(bf16_dev(x), w.bf16_prepack_weight(bf16_dev(wt), act=_act_id(w, act)), N,
                      bias=bf16_dev(b) if bias else None, act=_act_id(w, act), residual=bf16_dev(r) if res else None,
                      out=w.OUT_F32 if f32 else w.OUT_BF16)
    sync()
    show(f"  share of the tolerance used: "
         f"{_hold(y, *_epilogue(*_bf16_value(x, wt, b), act, r), f'{M}x{N}x{K}', f32):.3f}")


@pytest.mark.parametrize("M,N,K,act", [(4100, 4100, 192, "silu"), (2304, 2048, 1100, "swiglu"), (3000, 2900, 133, "none"),
                                       (5000, 300, 512, "swiglu"), (1100, 9000, 256, "gelu")])
def test_bf16_wide_tiles(w, M, N, K, act):
    """Tiles that a workgroup walks over, ragged on every side, sampled rows; rows around untouched."""
    show(f"bf16 {M} x {N} x {K} {act}")
    rng = np.random.default_rng(M + N + K)
    width = N // 2 if act == "swiglu" else N
    x, wt = _acts(rng, M, K), _bf16(rng, N, K, scale=1 / math.sqrt(K))
    b, r = _bf16(rng, N, scale=0.3), _bf16(rng, M, width)
    room = torch.full((M + 2, width), 7.0, dtype=torch.bfloat16, device=DEV)
    w.bf16_linear(bf16_dev(x), w.bf16_prepack_weight(bf16_dev(wt), act=_act_id(w, act)), N, bias=bf16_dev(b),
                  act=_act_id(w, act), residual=bf16_dev(r), y=room[1:M + 1])
    sync()
    assert (room[0] == 7).all() and (room[M + 1] == 7).all()
    pick = np.unique(np.r_[0:3, 31:34, 127:130, 254:258, 1000:1003, M - 3:M])
    y = room[1:M + 1][torch.from_numpy(pick).to(DEV)]
    _hold(y, *_epilogue(*_bf16_value(x[pick], wt, b), act, r[pick]))


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("M", [3, 20, 50, 80, 260, 1200])
@pytest.mark.parametrize("N,K", [(200, 640), (41, 77), (64, 200)])
def test_exact_small_integers(w, M, N, K, kind):
    """Small integers and unit scales: every sum is exact, the output its BF16."""
    rng = np.random.default_rng(M)
    xi = rng.integers(-3, 4, (M, K)).astype(np.float32)
    wi = rng.integers(-2, 3, (N, K)).astype(np.float32)
    r = rng.integers(-4, 5, (M, N)).astype(np.float32)
    rd = bf16_dev(O.f32_to_bf16(r))
    if kind == "int8":
        y = w.linear_fused(dev(xi.astype(np.int8)), dev(np.ones(M, np.float32)), w.prepack_weight(dev(wi.astype(np.int8))),
                           dev(np.ones(N, np.float32)), N, residual=rd)
    else:
        y = w.bf16_linear(bf16_dev(O.f32_to_bf16(xi)), w.bf16_prepack_weight(bf16_dev(O.f32_to_bf16(wi))), N, residual=rd)
    sync()
    assert np.array_equal(bf16_host(y), O.f32_to_bf16((xi @ wi.T + r).astype(np.float32)))


@pytest.mark.parametrize("M", [1, 20, 50, 100, 1200])
@pytest.mark.parametrize("K,lo", [(72, 8), (77, 3), (128, 8), (1000, 16), (333, 5)])
def test_nothing_behind_a_row_takes_part(w, M, K, lo):
    """Rows inside wider ones full of NaN; outputs and residual in wider rows."""
    rng = np.random.default_rng(K)
    N = 70
    wide = np.full((M, K + 32), 0x7FC0, np.uint16)
    x = _acts(rng, M, K)
    wide[:, lo:lo + K] = x
    wt = _bf16(rng, N, K, scale=1 / math.sqrt(K))
    rw = np.full((M, N + 7), 0x7FC0, np.uint16)
    rw[:, 3:3 + N] = _bf16(rng, M, N)
    room = torch.full((M + 2, N + 9), 7.0, dtype=torch.bfloat16, device=DEV)
    w.bf16_linear(bf16_dev(wide)[:, lo:lo + K], w.bf16_prepack_weight(bf16_dev(wt)), N, act=w.ACT_SILU,
                  residual=bf16_dev(rw)[:, 3:3 + N], y=room[1:M + 1, 5:5 + N])
    sync()
    _hold(room[1:M + 1, 5:5 + N], *_epilogue(*_bf16_value(x, wt), "silu", rw[:, 3:3 + N]))
    room[1:M + 1, 5:5 + N] = 7.0
    assert (room == 7).all()
    # codes inside wider rows
    q, s = O.dynamic_quant(x)
    codes = np.full((M, K + 32), 99, np.int8)
    codes[:, lo:lo + K] = q
    wi = rng.integers(-127, 128, (N, K)).astype(np.int8)
    ws = (rng.uniform(0.5, 1.5, N) / 1000).astype(np.float32)
    w.linear_fused(dev(codes)[:, lo:lo + K], dev(s), w.prepack_weight(dev(wi)), dev(ws), N, y=room[1:M + 1, 5:5 + N])
    sync()
    assert np.array_equal(bf16_host(room[1:M + 1, 5:5 + N]), O.linear(q, s, wi, ws)[0])
    room[1:M + 1, 5:5 + N] = 7.0
    assert (room == 7).all()


@pytest.mark.parametrize("M", [1, 40, 100, 1100])
def test_non_finite_values_stay_in_their_row(w, M):
    rng = np.random.default_rng(M)
    N, K = 96, 200
    x, wt = _acts(rng, M, K), _bf16(rng, N, K, scale=0.1)
    x[0, 7] = 0x7F80
    if M > 2:
        x[2, 199] = 0x7FC0
    for act in ("none", "silu", "gelu", "gelu_tanh", "relu"):
        y = w.bf16_linear(bf16_dev(x), w.bf16_prepack_weight(bf16_dev(wt)), N, act=_act_id(w, act))
        sync()
        y = y.float().cpu().numpy()
        clean = np.delete(np.arange(M), [0, 2] if M > 2 else [0])
        assert np.isfinite(y[clean]).all()
        assert not np.isfinite(y[0, O.bf16_to_f32(wt)[:, 7] > 0]).any()
        if M > 2:
            assert np.isnan(y[2]).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_activations_over_their_range(w, act):
    """v itself through the products: one-hot rows times a column of values."""
    v = np.concatenate([np.linspace(-120, 120, 4001), np.linspace(-6, 6, 4001), [3e38, -3e38, 1e20, -1e20, 0.0, 1e-38]])
    vb = O.f32_to_bf16(v.astype(np.float32))
    wt = np.zeros((len(vb), 16), np.uint16)
    wt[:, 0] = vb
    x = np.zeros((1, 16), np.uint16)
    x[0, 0] = 0x3F80
    y = w.bf16_linear(bf16_dev(x), w.bf16_prepack_weight(bf16_dev(wt)), len(vb), act=_act_id(w, act), out=w.OUT_F32)
    sync()
    _hold(y, *_epilogue(_f64(vb)[None], np.zeros((1, len(vb))), act), f32=True)


# ------------------------------------------------------------------ grouped
def _grouped_value(x, rows, counts, wt, act):
    """float64 outputs and errors of the rows that the counts own."""
    ys, ds, first = [], [], 0
    for e, n in enumerate(counts):
        v, dv = _bf16_value(x[rows[first:first + n]], wt[e])
        y, d = _epilogue(v, dv, act)
        ys.append(y)
        ds.append(d)
        first += n
    return np.concatenate(ys), np.concatenate(ds)


COUNTS = [[12, 7, 0, 19], [0, 0, 1], [16, 17, 32, 33, 64, 65, 96, 97, 128, 129], [300, 0, 513, 1], [1] * 40, [700],
          [256, 512, 255, 257]]


@pytest.mark.parametrize("index", [False, True])
@pytest.mark.parametrize("act", ["none", "swiglu", "gelu"])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", [(48, 128), (300, 200), (530, 77)])
def test_grouped(w, counts, N, K, act, index):
    show(f"grouped {counts} {N} x {K} {act} index {index}")
    rng = np.random.default_rng(sum(counts) + N + K)
    E, R, T = len(counts), sum(counts) + 5, 37
    x = _acts(rng, T if index else R, K)
    rows = rng.integers(0, T, R).astype(np.int32) if index else np.arange(R)
    wt = _bf16(rng, E, N, K, scale=1 / math.sqrt(K))
    width = N // 2 if act == "swiglu" else N
    y = torch.full((R, width), 7.0, dtype=torch.bfloat16, device=DEV)
    w.bf16_grouped_gemm(bf16_dev(x), dev(np.array(counts, np.int64)), w.bf16_prepack_weight(bf16_dev(wt), act=_act_id(w, act)),
                        N, act=_act_id(w, act), row_index=dev(rows) if index else None, y=y)
    sync()
    n = sum(counts)
    assert (y[n:] == 7).all()                            # rows behind the last group
    _hold(y[:n], *_grouped_value(x, rows, counts, wt, act), f"{counts}")


def test_grouped_bad_indices_and_counts_stay_in_bounds(w):
    rng = np.random.default_rng(2)
    R, N, K, T = 40, 64, 128, 10
    x, wt = _acts(rng, T, K), _bf16(rng, 3, N, K, scale=0.1)
    wp = w.bf16_prepack_weight(bf16_dev(wt))
    rows = rng.integers(0, T, R).astype(np.int32)
    rows[3], rows[5] = -7, 1 << 30                       # clamped
    y = torch.full((R + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    w.bf16_grouped_gemm(bf16_dev(x), dev(np.array([20, -3, 100], np.int64)), wp, N, row_index=dev(rows), y=y[:R])
    sync()
    rows[3], rows[5] = 0, T - 1
    assert (y[R] == 7).all()
    _hold(y[:R], *_grouped_value(x, rows, [20, 0, 20], wt, "none"))


def test_grouped_strided_rows_and_none_at_all(w):
    rng = np.random.default_rng(3)
    x, wt = _acts(rng, 50, 300), _bf16(rng, 2, 64, 264, scale=0.1)
    wp = w.bf16_prepack_weight(bf16_dev(wt))
    y = w.bf16_grouped_gemm(bf16_dev(x)[:, 8:272], dev(np.array([21, 29], np.int64)), wp, 64)
    z = torch.full((50, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    w.bf16_grouped_gemm(bf16_dev(x)[:, 8:272], dev(np.array([0, 0], np.int64)), wp, 64, y=z)
    sync()
    _hold(y, *_grouped_value(x[:, 8:272], np.arange(50), [21, 29], wt, "none"))
    assert (z == 7).all()


def test_zero_rows(w):
    wp = w.bf16_prepack_weight(torch.zeros((32, 64), dtype=torch.bfloat16, device=DEV))
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    assert w.bf16_linear(x, wp, 32).shape == (0, 32)
    assert w.bf16_grouped_gemm(x, torch.zeros(1, dtype=torch.int64, device=DEV), wp, 32).shape == (0, 32)
    assert w.rms_norm(x, None).shape == (0, 64)


# ------------------------------------------------------------------ together
def test_block_of_a_layer_captured_and_replayed(w):
    """Norm -> INT8 projection with the residual behind it -> norm (FP8 codes and BF16) ->
    router logits in fp32 -> BF16 experts with SwiGLU, captured, replayed with other inputs
    and compared with the same calls made one by one."""
    rng = np.random.default_rng(11)
    T, H, I, E, k = 48, 256, 96, 8, 2
    g1, g2 = bf16_dev(_bf16(rng, H)), bf16_dev(_bf16(rng, H))
    wi = rng.integers(-127, 128, (H, H)).astype(np.int8)
    wo, wos = w.prepack_weight(dev(wi)), dev((rng.uniform(0.5, 1.5, H) / (73 * 16)).astype(np.float32))
    router = w.bf16_prepack_weight(bf16_dev(_bf16(rng, E, H, scale=0.2)))
    w13 = w.bf16_prepack_weight(bf16_dev(_bf16(rng, E, 2 * I, H, scale=0.06)), act=w.ACT_SWIGLU)
    w2 = w.bf16_prepack_weight(bf16_dev(_bf16(rng, E, H, I, scale=0.1)))
    x, stream = bf16_dev(_acts(rng, T, H)), bf16_dev(_acts(rng, T, H))
    ws = [torch.empty((w.bf16_grouped_workspace_bytes(T * k, E, 2 * I, H),), dtype=torch.uint8, device=DEV)
          for _ in range(2)]

    def layer(out):
        h = stream.clone()
        q, s = w.rms_norm_quant(x, g1, residual=h)
        w.linear_fused(q, s, wo, wos, H, residual=h, y=h)
        n = torch.empty_like(h)
        w.fp8b_rms_norm_quant(h, g2, y=n)
        logits = w.bf16_linear(n, router, E, out=w.OUT_F32)
        ids, wts = w.moe_gate(logits, k)
        gl, rt, pr = w.moe_route(ids, E)
        a = w.bf16_grouped_gemm(n, gl, w13, 2 * I, act=w.ACT_SWIGLU, row_index=rt, workspace=ws[0])
        y = w.bf16_grouped_gemm(a, gl, w2, H, workspace=ws[1])
        out[0].copy_(h)
        out[1].copy_(w.moe_combine(y, pr, wts))

    out = [torch.empty_like(x) for _ in range(2)]
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        layer(out)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(out)
    want = [torch.empty_like(x) for _ in range(2)]
    for _ in range(3):
        x.copy_(bf16_dev(_acts(rng, T, H)))
        stream.copy_(bf16_dev(_acts(rng, T, H)))
        layer(want)
        for o in out:
            o.fill_(7.0)
        graph.replay()
        sync()
        assert torch.isfinite(want[1].float()).all() and want[1].float().abs().max() > 0
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_at_once(w):
    rng = np.random.default_rng(12)
    M, N, K = 1200, 600, 1000
    x, wt = bf16_dev(_acts(rng, M, K)), bf16_dev(_bf16(rng, N, K, scale=0.03))
    wp = w.bf16_prepack_weight(wt)
    want = w.bf16_linear(x, wp, N)
    sync()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.empty_like(want) for _ in range(6)]
    room = [torch.empty((w.bf16_linear_workspace_bytes(M, N, K),), dtype=torch.uint8, device=DEV) for _ in range(2)]
    for i, y in enumerate(ys):
        with torch.cuda.stream(streams[i % 2]):
            w.bf16_linear(x, wp, N, y=y, workspace=room[i % 2])
    sync()
    assert all(torch.equal(y, want) for y in ys)


# ------------------------------------------------------------------ every kernel and split
PLANS = [  # M, N, K of BF16 (INT8: twice the K)
    (23, 22, 62), (107, 4, 4386), (38, 3440, 206), (52, 1984, 1172), (64, 4096, 3584), (103, 2662, 1546), (75, 22, 8540),
    (180, 302, 9000), (654, 942, 2031), (227, 20, 9528), (340, 1502, 3400), (700, 4134, 1000), (389, 8070, 1104), (4325, 134, 5911),
    (5629, 1438, 455), (2448, 5190, 67), (2500, 4202, 1111), (40001, 66, 130), (70000, 18, 30)]


def _sample(M):
    return np.unique(np.clip(np.r_[0:2, 15:18, 31:34, 63:66, 126:130, 255:258, M // 2:M // 2 + 3, M - 3:M], 0, M - 1))


@pytest.mark.parametrize("kind,act", [("bf16", "none"), ("bf16", "swiglu"), ("bf16", "gelu"), ("int8", "silu"), ("int8", "none")])
@pytest.mark.parametrize("M,N,K", PLANS)
def test_every_kernel(w, M, N, K, kind, act):
    """Low and high tiles, K whole and in parts, with and without the epilogue's operands;
    sampled rows against 64 bits."""
    show(f"{kind} {M} x {N} x {K} {act}")
    rng = np.random.default_rng(M + N + K)
    width = N // 2 if act == "swiglu" else N
    with_res = act != "gelu"
    b, r = _bf16(rng, N, scale=0.3), _bf16(rng, M, width)
    room = torch.full((M + 2, width), 7.0, dtype=torch.bfloat16, device=DEV)
    kw = dict(bias=bf16_dev(b), act=_act_id(w, act), residual=bf16_dev(r) if with_res else None)
    if act in ("swiglu", "silu"):                         # in place
        room[1:M + 1] = kw["residual"]
        kw["residual"] = room[1:M + 1]
    pick = _sample(M)
    if kind == "bf16":
        x, wt = _acts(rng, M, K), _bf16(rng, N, K, scale=1 / math.sqrt(K))
        w.bf16_linear(bf16_dev(x), w.bf16_prepack_weight(bf16_dev(wt), act=_act_id(w, act)), N, y=room[1:M + 1], **kw)
        v, dv = _bf16_value(x[pick], wt, b)
    else:
        q, s, wi, ws = _int8_operands(rng, M, N, 2 * K)
        w.linear_fused(dev(q), dev(s), w.prepack_weight(dev(wi)), dev(ws), N, y=room[1:M + 1], **kw)
        v = (q[pick].astype(np.float64) @ wi.T.astype(np.float64)) * s[pick].astype(np.float64)[:, None] * ws.astype(np.float64)
        dv = 3.1 * U * np.abs(v)                          # acc to fp32, two products
        v = v + _f64(b)
        dv = dv + U * (np.abs(v) + dv)
    sync()
    assert (room[0] == 7).all() and (room[M + 1] == 7).all()
    y = room[1:M + 1]
    _hold(y[torch.from_numpy(pick).to(DEV)], *_epilogue(v, dv, act, r[pick] if with_res else None), f"{M}x{N}x{K}")
    assert torch.isfinite(y.float()).all()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("M,N,K,lo", [(700, 4134, 1001, 1), (300, 1000, 5761, 3), (2500, 4202, 1111, 1), (340, 1502, 3403, 5)])
def test_rows_at_odd_addresses(w, M, N, K, lo, kind):
    """As they are, and copied (wide tiles); NaN (INT8: codes) around them."""
    rng = np.random.default_rng(K)
    pick = _sample(M)
    if kind == "bf16":
        x, wt = _acts(rng, M, K), _bf16(rng, N, K, scale=1 / math.sqrt(K))
        wide = torch.full((M, K + 6), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, lo:lo + K] = bf16_dev(x)
        y = w.bf16_linear(wide[:, lo:lo + K], w.bf16_prepack_weight(bf16_dev(wt)), N)
        sync()
        _hold(y[torch.from_numpy(pick).to(DEV)], *_epilogue(*_bf16_value(x[pick], wt), "none"))
        return
    q, s, wi, ws = _int8_operands(rng, M, N, K)
    wide = torch.full((M, K + 6), 99, dtype=torch.int8, device=DEV)
    wide[:, lo:lo + K] = dev(q)
    wp = w.prepack_weight(dev(wi))
    a = w.linear_fused(wide[:, lo:lo + K], dev(s), wp, dev(ws), N)
    b = w.linear(dev(q), dev(s), wp, dev(ws), N)
    sync()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("act,index,lo", [("none", True, 0), ("swiglu", False, 0), ("gelu", True, 3)])
@pytest.mark.parametrize("counts,N,K", [([900, 0, 513, 161, 160, 1466], 4130, 700), ([2700, 300], 4200, 1000)])
def test_grouped_of_many_rows(w, counts, N, K, act, index, lo):
    """Tiles of 128 and of 256 rows; rows through an index, rows at odd addresses."""
    rng = np.random.default_rng(N + K)
    E, R, T = len(counts), sum(counts) + 5, 777
    x = _acts(rng, T if index else R, K)
    wide = torch.full((len(x), K + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, lo:lo + K] = bf16_dev(x)
    rows = rng.integers(0, T, R).astype(np.int32) if index else np.arange(R)
    wt = _bf16(rng, E, N, K, scale=1 / math.sqrt(K))
    width = N // 2 if act == "swiglu" else N
    y = torch.full((R, width), 7.0, dtype=torch.bfloat16, device=DEV)
    w.bf16_grouped_gemm(wide[:, lo:lo + K], dev(np.array(counts, np.int64)),
                        w.bf16_prepack_weight(bf16_dev(wt), act=_act_id(w, act)), N, act=_act_id(w, act),
                        row_index=dev(rows) if index else None, y=y)
    sync()
    assert (y[sum(counts):] == 7).all() and torch.isfinite(y.float()).all()
    first = 0
    for e, n in enumerate(counts):
        if n:
            pick = first + _sample(n)
            v, dv = _bf16_value(x[rows[pick]], wt[e])
            _hold(y[torch.from_numpy(pick).to(DEV)], *_epilogue(v, dv, act), f"expert {e}")
        first += n


def test_split_sums_captured_and_replayed(w):
    """A product whose K is split, in a graph that is replayed with new rows and its own
    workspace, with eager work on the same stream between."""
    rng = np.random.default_rng(9)
    M, N, K = 340, 1502, 3400
    wt = _bf16(rng, N, K, scale=1 / math.sqrt(K))
    wp = w.bf16_prepack_weight(bf16_dev(wt))
    assert w.bf16_linear_workspace_bytes(M, N, K) >= 2 * M * N * 4
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    room = torch.empty((w.bf16_linear_workspace_bytes(M, N, K),), dtype=torch.uint8, device=DEV)
    w.bf16_linear(x, wp, N, y=y, workspace=room)
    sync()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.bf16_linear(x, wp, N, y=y, workspace=room)
    for i in range(4):
        x.copy_(bf16_dev(_acts(rng, M, K)))
        room.fill_(255)                                   # nothing of the call before is used
        g.replay()
        eager = w.bf16_linear(x, wp, N)
        sync()
        assert torch.equal(y.view(torch.int16), eager.view(torch.int16)), i


@pytest.mark.parametrize("M,N,K,act", [(2500, 4202, 1112, "gelu"), (1037, 530, 1111, "none")])
def test_offsets_past_32_bits(w, M, N, K, act):
    """Rows 4 MB apart: x, residual and y are columns of one buffer of 4 to 10 GB."""
    show(f"{M} rows 4 MB apart")
    rng = np.random.default_rng(M)
    big = torch.empty((M, 1 << 21), dtype=torch.bfloat16, device=DEV)
    x, wt, r = _acts(rng, M, K), _bf16(rng, N, K, scale=1 / math.sqrt(K)), _bf16(rng, M, N)
    xs, rs, ys = big[:, 8:8 + K], big[:, 20001:20001 + N], big[:, 40000:40000 + N]
    xs.copy_(bf16_dev(x))
    rs.copy_(bf16_dev(r))
    wp = w.bf16_prepack_weight(bf16_dev(wt))
    w.bf16_linear(xs, wp, N, act=_act_id(w, act), residual=rs, y=ys)
    rows = rng.integers(0, M, M + 3).astype(np.int32)
    counts = [M // 2, 0, M - M // 2]
    g = w.bf16_grouped_gemm(xs, dev(np.array(counts, np.int64)), torch.cat([wp, wp, wp]), N, act=_act_id(w, act),
                            row_index=dev(rows))
    n, hn = w.rms_norm(xs, None, 1e-6), big[:, 60000:60000 + K]
    w.rms_norm(xs, None, 1e-6, y=hn)
    sync()
    pick = _sample(M)
    at = torch.from_numpy(pick).to(DEV)
    _hold(ys[at], *_epilogue(*_bf16_value(x[pick], wt), act, r[pick]))
    _hold(g[at], *_epilogue(*_bf16_value(x[rows[pick]], wt), act))
    same = w.rms_norm(xs.contiguous(), None, 1e-6)
    assert torch.equal(n.view(torch.int16), same.view(torch.int16)) and torch.equal(hn.contiguous().view(torch.int16),
                                                                                 same.view(torch.int16))


def test_eager_calls_beside_a_replayed_graph_on_another_stream(w):
    """Two products at once, each with its own workspace."""
    rng = np.random.default_rng(4)
    M, N, K = 340, 1502, 3400
    wp = w.bf16_prepack_weight(bf16_dev(_bf16(rng, N, K, scale=1 / math.sqrt(K))))
    xs = [bf16_dev(_acts(rng, M, K)) for _ in range(2)]
    want = [w.bf16_linear(x, wp, N) for x in xs]
    y = torch.empty_like(want[0])
    room = torch.empty((w.bf16_linear_workspace_bytes(M, N, K),), dtype=torch.uint8, device=DEV)
    sync()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.bf16_linear(xs[0], wp, N, y=y, workspace=room)
    side = torch.cuda.Stream()
    for _ in range(5):
        y.zero_()
        sync()
        g.replay()
        with torch.cuda.stream(side):
            z = w.bf16_linear(xs[1], wp, N)
        sync()
        assert torch.equal(y.view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(z.view(torch.int16), want[1].view(torch.int16))
