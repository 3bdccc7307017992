"""The kernels of the fused linears and of the BF16 products that only large or ragged
sizes reach, each shown to be the one that runs, against float64. Tolerances as in
test_gpu_fused.py."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle as O
from tests.conftest import gpu_available
from tests.gpu_util import DEV, bf16_dev, dev, show, sync
from tests.test_gpu_fused import F, U, _act_id, _acts, _bf16, _bf16_value, _epilogue, _f64, _hold, _int8_operands

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


def _rows_of_tiles(M):
    """A row of every 128, in turn the first, the last and one between, and the last rows."""
    at = np.arange(0, M, 128)
    return np.unique(np.clip(np.r_[at + np.resize([0, 127, 37, 64], len(at)), M - 2:M], 0, M - 1))


# 256 x 256 with more tiles than workgroups and last tiles of 1, 4 and 150 rows; blocks of
# K even, odd and two; columns that end inside a wavefront's 64 or 16. 128 x 256.
FP8 = [(8193, 4100, 512, "silu", True, True, True), (8193, 4100, 512, "none", False, True, False),
       (4100, 4130, 640, "gelu", True, False, False), (4100, 4130, 640, "relu", True, True, True),
       (8342, 4161, 200, "gelu_tanh", False, True, True), (8342, 4161, 200, "none", True, True, False),
       (4097, 8200, 900, "silu", False, False, False), (4097, 8200, 900, "gelu", False, True, True)]
FP8_128 = [(2000, 3000, 1000, "silu", True, True, True), (2000, 3000, 1000, "relu", False, False, False),
           (1930, 2890, 1000, "gelu_tanh", True, True, False), (1930, 2890, 1000, "none", False, True, True)]


@pytest.mark.parametrize("M,N,K,act,bias,res,place,tile", [(*c, (256, 256)) for c in FP8] + [(*c, (128, 256)) for c in FP8_128])
def test_fp8_high_tiles_with_an_epilogue(w, M, N, K, act, bias, res, place, tile):
    """The wide tiles that a workgroup walks over and the 128-row tiles, the residual in
    place or beside; rows around the output untouched; codes given and quantized inside."""
    show(f"fp8 {M} x {N} x {K} {act} bias {bias} residual {res} in place {place}")
    rng = np.random.default_rng(M + 7 * N + 11 * K)
    x = _acts(rng, M, K, 1.0)
    cw = O.mx.e4m3_encode(np.clip(rng.standard_normal((N, K)) * 100.0, -448, 448))
    sw = (rng.uniform(0.5, 1.5, (O.fp8b.blocks(N), O.fp8b.blocks(K))) / (100 * math.sqrt(K))).astype(np.float32)
    b, r = (_bf16(rng, N, scale=0.3) if bias else None), (_bf16(rng, M, N) if res else None)
    wp, xd, swd = w.fp8b_prepack_weight(dev(cw)), bf16_dev(x), dev(sw)
    qd, sd = w.fp8b_quant(xd)
    plan = w.fp8b_linear_plan(qd, N, x_scale=sd, K=K)
    assert (plan.tile_rows, plan.tile_cols) == tile
    assert tile[0] == 128 or plan.tiles > 256            # more than a workgroup a CU
    assert w.fp8b_linear_plan(xd, N).tile_rows == tile[0]
    room = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    y, rd = room[1:M + 1], bf16_dev(r) if res else None
    if place:
        y.copy_(rd)
        rd = y
    kw = dict(bias=bf16_dev(b) if bias else None, act=_act_id(w, act), y=y)
    w.fp8b_linear_fused(qd, wp, swd, N, x_scale=sd, K=K, residual=rd, **kw)
    sync()
    assert (room[0] == 7).all() and (room[M + 1] == 7).all()
    first = y.clone()
    if place:
        y.copy_(bf16_dev(r))
    w.fp8b_linear_fused(xd, wp, swd, N, residual=rd, **kw)
    sync()
    assert torch.equal(first.view(torch.int16), y.view(torch.int16))
    pick = _rows_of_tiles(M)
    q, s = O.fp8b.quant(x[pick])
    v = O.fp8b.product64(q, s, cw, sw, b)
    A = np.abs(O.fp8b.dequant(q, s)) @ np.abs(O.fp8b.weight_dequant(cw, sw)).T
    if bias:
        A = A + np.abs(_f64(b))
    dv = O.fp8b.cut_bound(q, s, cw, sw) + (18 + O.fp8b.blocks(K)) * 2.0 ** -23 * A
    _hold(y[torch.from_numpy(pick).to(DEV)], *_epilogue(v, dv, act, r[pick] if res else None), f"{M}x{N}x{K}")
    assert torch.isfinite(y.float()).all()


# K in elements of BF16 (INT8: twice as many): steps of 128 bytes odd, even and two, ragged
# and whole; last tiles of 8, 1, 77 and 120 rows
WALKED = [(8200, 4100, 520), (8193, 4100, 512), (8269, 8150, 96), (8312, 4354, 712)]


@pytest.mark.parametrize("kind,act,bias,res,place", [("bf16", "none", False, True, False), ("bf16", "swiglu", True, True, True),
                                                     ("bf16", "silu", True, False, False), ("int8", "gelu", True, True, True),
                                                     ("int8", "none", True, False, False), ("int8", "relu", False, True, False)])
@pytest.mark.parametrize("M,N,K", WALKED)
def test_wide_tiles_that_a_workgroup_walks_over(w, M, N, K, kind, act, bias, res, place):
    """More tiles than workgroups: the next tile's rows and weights land while one is
    stored. Rows of every tile against float64, rows around the output untouched."""
    show(f"{kind} {M} x {N} x {K} {act} bias {bias} residual {res} in place {place}")
    rng = np.random.default_rng(M + 7 * N + 11 * K)
    width = N // 2 if act == "swiglu" else N
    b, r = (_bf16(rng, N, scale=0.3) if bias else None), (_bf16(rng, M, width) if res else None)
    room = torch.full((M + 2, width), 7.0, dtype=torch.bfloat16, device=DEV)
    y, rd = room[1:M + 1], bf16_dev(r) if res else None
    if place:
        y.copy_(rd)
        rd = y
    kw = dict(bias=bf16_dev(b) if bias else None, act=_act_id(w, act), residual=rd, y=y)
    pick = _rows_of_tiles(M)
    if kind == "bf16":
        x, wt = _acts(rng, M, K), _bf16(rng, N, K, scale=1 / math.sqrt(K))
        xd, wp = bf16_dev(x), w.bf16_prepack_weight(bf16_dev(wt), act=_act_id(w, act))
        plan = w.bf16_linear_plan(xd, N, _act_id(w, act))
        w.bf16_linear(xd, wp, N, **kw)
        v, dv = _bf16_value(x[pick], wt, b)
    else:
        q, s, wi, ws = _int8_operands(rng, M, N, 2 * K)
        qd = dev(q)
        plan = w.linear_fused_plan(qd, N)
        w.linear_fused(qd, dev(s), w.prepack_weight(dev(wi)), dev(ws), N, **kw)
        v = (q[pick].astype(np.float64) @ wi.T.astype(np.float64)) * s[pick].astype(np.float64)[:, None] * ws.astype(np.float64)
        dv = 4 * U * np.abs(v)
        if bias:
            v, dv = v + _f64(b), dv + 4 * U * np.abs(_f64(b))
    sync()
    assert (plan.tile_rows, plan.tile_cols, plan.copied) == (256, 256, 0) and plan.tiles > 512
    assert (room[0] == 7).all() and (room[M + 1] == 7).all()
    _hold(y[torch.from_numpy(pick).to(DEV)], *_epilogue(v, dv, act, r[pick] if res else None), f"{M}x{N}x{K}")
    assert torch.isfinite(y.float()).all()


# experts whose rows end in every height of the low tiles, behind wide tiles and alone; and
# with so many tiles (columns in 17 and in 16 groups) that they are spread over the XCDs
HEIGHTS = [65, 80, 96, 97, 128, 129, 326, 608, 3, 17, 40, 0, 1700]
MANY = [4000, 70, 4890]
WIDE = [9000, 8070]


@pytest.mark.parametrize("counts,N,K,lo,index,act,rows", [
    (HEIGHTS, 4130, 1400, 0, False, "none", 256), (HEIGHTS, 4130, 1400, 0, True, "swiglu", 256),
    (HEIGHTS, 4130, 1400, 3, False, "swiglu", 128), (HEIGHTS, 4130, 1401, 0, True, "gelu", 128),
    (MANY, 4130, 700, 0, False, "none", 128), (MANY, 4000, 701, 1, True, "swiglu", 128),
    (MANY, 4000, 1000, 0, True, "silu", 256), (WIDE, 2000, 1000, 0, True, "none", 256), (WIDE, 2100, 1000, 0, True, "gelu", 256)])
def test_grouped_heights(w, counts, N, K, lo, index, act, rows):
    """Tiles of up to 128 rows and wide ones, each shown to be there by the plan; an
    expert's first rows, its last ones and the borders of its tiles."""
    show(f"grouped {counts} {N} x {K} from column {lo} index {index} {act}")
    rng = np.random.default_rng(N + K + lo)
    E, R, T = len(counts), sum(counts) + 5, 777
    x = _acts(rng, T if index else R, K)
    wide = torch.full((len(x), K + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, lo:lo + K] = bf16_dev(x)
    xd, at = wide[:, lo:lo + K], rng.integers(0, T, R).astype(np.int32) if index else np.arange(R)
    ad = dev(at) if index else None
    plan = w.bf16_grouped_plan(xd, E, N, row_index=ad)
    assert (plan.tile_rows, plan.tile_cols) == (rows, 256)
    wt = _bf16(rng, E, N, K, scale=1 / math.sqrt(K))
    width = N // 2 if act == "swiglu" else N
    y = torch.full((R, width), 7.0, dtype=torch.bfloat16, device=DEV)
    w.bf16_grouped_gemm(xd, dev(np.array(counts, np.int64)), w.bf16_prepack_weight(bf16_dev(wt), act=_act_id(w, act)), N,
                        act=_act_id(w, act), row_index=ad, y=y)
    sync()
    assert (y[sum(counts):] == 7).all() and torch.isfinite(y.float()).all()
    first = 0
    for e, n in enumerate(counts):
        if n:
            step = np.arange(0, n, 128)
            pick = first + np.unique(np.clip(np.r_[step, step + 16, step + 63, step + 95, step + 127, n - 2:n], 0, n - 1))
            v, dv = _bf16_value(x[at[pick]], wt[e])
            _hold(y[torch.from_numpy(pick).to(DEV)], *_epilogue(v, dv, act), f"expert {e}")
        first += n


def _activated(w, v_bits, act):
    """fp32 outputs of the values themselves: a one-hot row times a column of them."""
    wt = np.zeros((len(v_bits), 16), np.uint16)
    wt[:, 0] = v_bits
    x = np.zeros((1, 16), np.uint16)
    x[0, 0] = 0x3F80
    y = w.bf16_linear(bf16_dev(x), w.bf16_prepack_weight(bf16_dev(wt)), len(v_bits), act=_act_id(w, act), out=w.OUT_F32)
    sync()
    return y.cpu().numpy()[0].astype(np.float64)


def test_gelu_tail_is_the_published_formula(w):
    """v < 0: relative to 0.5 v t s(t) e^(-z^2) in 64 bits, z = |v| / sqrt 2, t = 1 / (1 + p z), s
    the polynomial of the Handbook's 7.1.26, however small the value. Roundings (units of
    2^-24): z 1.3 (constant 0.3, product 1); t: 3.3 of its divisor and 2 of the reciprocal;
    a term a_k t^k of s: its coefficient, k + 1 additions at most five, 5.3 k, so at most 28 of
    sum |a_k| t^k; the exponent z^2 log2 e: 2.6 + 1 + 2 of it, so 5.6 v^2 / 2 of the result, and 2
    of the exponential; the products 4."""
    v = O.f32_to_bf16(np.unique(np.r_[-np.linspace(0.01, 13, 4000), -np.geomspace(1e-30, 0.01, 300)]).astype(np.float32))
    v = np.unique(v)
    y, x = _activated(w, v, "gelu"), _f64(v)
    z = -x / math.sqrt(2.0)
    t = 1.0 / (1.0 + 0.3275911 * z)
    a = [0.254829592, -0.284496736, 1.421413741, -1.453152027, 1.061405429]
    s = sum(c * t ** k for k, c in enumerate(a))
    size = sum(abs(c) * t ** k for k, c in enumerate(a))
    want = 0.5 * x * t * s * np.exp(-z * z)
    tol = 1.01 * (28.0 * size / s + 11.3 + 2.8 * x * x) * U * np.abs(want)
    off = np.abs(y - want)
    show(f"{len(v)} values, share of the tolerance used {float((off / tol).max()):.3f}")
    assert (off <= tol).all(), x[off > tol][:3]
    true = F.act64(x, "gelu")                             # and that formula, of the function
    assert (np.abs(want - true) <= 0.75e-7 * np.abs(x)).all()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_sigmoid_tails_hold_their_relative_bound_until_they_vanish(w, act):
    """Down to an exponent's argument of -87 within (6 |t| + 8) 2^-24 of the value; behind that
    0 or the value, which is below 90 e^-87 (the reciprocal of 2^126 and the exponential's
    overflow)."""
    v = np.unique(O.f32_to_bf16(np.r_[-np.linspace(0.001, 110, 4000), np.linspace(0.001, 110, 1000)].astype(np.float32)))
    y, x = _activated(w, v, act), _f64(v)
    want = F.act64(x, act)
    t = x if act == "silu" else 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    off = np.abs(y - want)
    near = t >= -87.0
    assert near.any() and (~near).any()
    assert (off <= (6 * np.minimum(np.abs(t), 90) + 8) * U * np.abs(want))[near].all()
    assert (off[~near] <= 2.0 ** -118).all() and (y[~near] <= 0).all()


@pytest.mark.parametrize("M,K", [(1, 4224), (1, 8192), (2, 300), (4, 2048), (16, 512), (17, 512), (200, 640)])
def test_fp8_linear_over_its_rows(w, M, K):
    """x, the residual and y are one buffer: x is quantized before any of y is written."""
    show(f"fp8 {M} x {K} x {K} over its rows")
    rng = np.random.default_rng(M + K)
    x = _acts(rng, M, K)
    cw = O.mx.e4m3_encode(np.clip(rng.standard_normal((K, K)) * 100.0, -448, 448))
    sw = (rng.uniform(0.5, 1.5, (O.fp8b.blocks(K), O.fp8b.blocks(K))) / (100 * math.sqrt(K))).astype(np.float32)
    wp, swd, xd = w.fp8b_prepack_weight(dev(cw)), dev(sw), bf16_dev(x)
    want = w.fp8b_linear_fused(xd, wp, swd, K, act=w.ACT_SILU, residual=xd)
    for _ in range(3):
        h = bf16_dev(x)
        w.fp8b_linear_fused(h, wp, swd, K, act=w.ACT_SILU, residual=h, y=h)
        sync()
        assert torch.equal(h.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("E", [1021, 1023, 1024])
def test_grouped_with_as_many_experts_as_there_can_be(w, E):
    """The list's four experts a thread: the last ones among them, most of them empty."""
    rng = np.random.default_rng(E)
    N, K = 40, 72
    counts = rng.integers(0, 3, E) * (rng.random(E) < 0.4)
    counts[[0, E - 3, E - 1]] = 70, 5, 33
    R = int(counts.sum()) + 3
    x, wt = _acts(rng, R, K), _bf16(rng, E, N, K, scale=1 / math.sqrt(K))
    y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    w.bf16_grouped_gemm(bf16_dev(x), dev(counts.astype(np.int64)), w.bf16_prepack_weight(bf16_dev(wt)), N, y=y)
    sync()
    assert (y[R - 3:] == 7).all()
    e = np.repeat(np.arange(E), counts)
    xs, ws = _f64(x[:R - 3]), _f64(wt)[e]
    v, A = (ws * xs[:, None]).sum(2), np.abs(ws * xs[:, None]).sum(2)
    _hold(y[:R - 3], v, 6 * math.sqrt(K) * U * A)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activations_of_infinities(w, act):
    """inf stays, -inf times 0 is NaN (ReLU: 0), NaN stays; zeros stay zeros."""
    v = np.array([0x7F80, 0xFF80, 0x7FC0, 0x0000, 0x8000] * 16, np.uint16)
    wt = np.zeros((len(v), 16), np.uint16)
    wt[:, 0] = v
    wp = w.bf16_prepack_weight(bf16_dev(wt))
    for M in (1, 40, 200):
        x = np.zeros((M, 16), np.uint16)
        x[:, 0] = 0x3F80
        y = w.bf16_linear(bf16_dev(x), wp, len(v), act=_act_id(w, act), out=w.OUT_F32)
        sync()
        y = y.cpu().numpy().reshape(M, 16, 5)
        assert (y[..., 0] == np.inf).all() and np.isnan(y[..., 2]).all() and (y[..., 3:] == 0).all()
        assert (y[..., 1] == 0).all() if act == "relu" else np.isnan(y[..., 1]).all()
