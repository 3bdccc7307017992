"""Block-scaled FP8 through the C ABI against the oracle.

Codes and scales are compared exactly. A product is held to
  2^-8 (|y| + d) + d,   d = c + (18 + B) 2^-23 A
of the float64 value y, with c the oracle's bound of the matrix unit's cuts, A the sum
of |s_x q_x s_w q_w| over K and B the number of 128-blocks: 2^-8 is half a step of
BF16; a block's 16 groups of 8 products are added in fp32 (16 roundings at most of
partial sums below A), the two scales are multiplied (1), and the B blocks and the bias
are added (B + 1), each within 2^-23.
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

F = O.fp8b


@pytest.fixture(scope="module")
def w():
    import moe_token_amax_amd as w
    return w


def _acts(rng, M, K, spread=0.0):
    x = rng.standard_normal((M, K)) * np.exp(spread * rng.standard_normal((M, 1)))
    x[rng.random((M, K)) < 0.01] *= 20.0
    return O.f32_to_bf16(x.astype(np.float32))


def _weight(rng, *shape):
    """codes [..., N, K] and scales [..., ceil(N/128), ceil(K/128)]"""
    c = O.mx.e4m3_encode(np.clip(rng.standard_normal(shape) * 100.0, -448, 448))
    s = rng.uniform(0.5, 1.5, (*shape[:-2], F.blocks(shape[-2]), F.blocks(shape[-1]))) * 0.01
    return c, s.astype(np.float32)


def _hold(got_bits, q, sx, cw, sw, bias_bits=None, what="", exact=False):
    """exact: products that are not cut, c = 0"""
    y = F.product64(q, sx, cw, sw, bias_bits)
    A = np.abs(F.dequant(q, sx)) @ np.abs(F.weight_dequant(cw, sw)).T
    if bias_bits is not None:
        A = A + np.abs(O.bf16_to_f32(bias_bits)).astype(np.float64)
    d = (0.0 if exact else F.cut_bound(q, sx, cw, sw)) + (18 + F.blocks(cw.shape[1])) * 2.0 ** -23 * A
    off = np.abs(O.bf16_to_f32(got_bits).astype(np.float64) - y)
    tol = 2.0 ** -8 * (np.abs(y) + d) + d + 1e-38
    bad = np.argwhere(~(off <= tol))
    assert bad.size == 0, f"{what}: {len(bad)} of {off.size}, first {bad[0].tolist()}: off {off[tuple(bad[0])]:.4g} " \
                          f"tol {tol[tuple(bad[0])]:.4g} y {y[tuple(bad[0])]:.4g}"
    return float((off / tol).max())


# ------------------------------------------------------------------ quant
@pytest.mark.parametrize("alg", [0, 1])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 7168), (3, 128), (16, 129), (17, 37), (33, 1412), (100, 704), (257, 2048)])
def test_quant_bit_exact(w, M, K, act, alg):
    show(f"quant {M} x {K} act {act} alg {alg}")
    rng = np.random.default_rng(M * 1000 + K)
    x = _acts(rng, M, K * (1 + act), 2.0)
    if M > 2:
        x[1, : K // 2] = 0               # blocks of zeros
        x[2, 0] = 0x8000                 # -0
    q, s = w.fp8b_quant(bf16_dev(x), act=act, scale_alg=alg)
    sync()
    qo, so = F.quant(x, act, alg)
    assert np.array_equal(host(s), so)
    assert np.array_equal(host(q), qo)


def test_quant_ties_and_small_values(w):
    # every BF16 magnitude from 2^-133 up, next to maxima that make ties and subnormal codes
    rng = np.random.default_rng(0)
    rows = []
    for top in (448.0, 224.0, 1.0, 1.75, 3.0e38, 1e-30, 2.0 ** -126, 2.0 ** -133):
        v = top * np.sort(rng.random(127)) ** rng.integers(1, 12, 127)
        rows.append(np.concatenate([[top], v * rng.choice([-1, 1], 127)]))
    rows.append(np.concatenate([[448.0], np.arange(127) * 0.5]))
    x = O.f32_to_bf16(np.array(rows, np.float32))
    for alg in (0, 1):
        q, s = w.fp8b_quant(bf16_dev(x), scale_alg=alg)
        sync()
        qo, so = F.quant(x, 0, alg)
        assert np.array_equal(host(s), so) and np.array_equal(host(q), qo)


def test_quant_every_bf16_value_against_random_maxima(w):
    # all finite BF16 values in rows of 127 below a maximum of their own binade
    v = np.arange(0, 0x7F80, dtype=np.uint16)
    rng = np.random.default_rng(4)
    v = rng.permutation(v)[: 127 * 256].reshape(256, 127)
    top = np.minimum(v.max(1) + rng.integers(0, 4, 256), 0x7F7F).astype(np.uint16)
    x = np.concatenate([top[:, None], v | (rng.integers(0, 2, v.shape).astype(np.uint16) << 15)], 1)
    q, s = w.fp8b_quant(bf16_dev(x))
    sync()
    qo, so = F.quant(x)
    assert np.array_equal(host(s), so) and np.array_equal(host(q), qo)


def test_quant_strided_rows_and_untouched_surroundings(w):
    rng = np.random.default_rng(8)
    x = _acts(rng, 20, 700)
    for lo, hi in ((8, 8 + 392), (3, 403)):      # 16-byte aligned rows, odd ones
        view = bf16_dev(x)[:, lo:hi]
        room = torch.full((22, 512), 0xEE, dtype=torch.uint8, device=DEV)
        q, s = w.fp8b_quant(view, q=room[1:21])
        sync()
        qo, so = F.quant(x[:, lo:hi])
        assert np.array_equal(host(s), so) and np.array_equal(host(q), qo)
        assert (host(room)[[0, 21]] == 0xEE).all()


def test_quant_non_finite_values_show_in_the_scale(w):
    x = np.zeros((3, 256), np.uint16)
    x[0, 5], x[1, 200], x[2, 0] = 0x7F80, 0x7FC0, 0x3F80
    q, s = w.fp8b_quant(bf16_dev(x))
    sync()
    s = host(s)
    assert np.isinf(s[0, 0]) and s[1, 0] == 0 and np.isnan(s[1, 1]) and s[0, 1] == 0 and s[0, 2] > 0


# ------------------------------------------------------------------ linear
LINEAR = [  # M, N, K
    (1, 16, 128), (1, 1, 1), (2, 17, 65), (4, 256, 1024), (16, 100, 300), (17, 128, 256), (33, 130, 2000),
    (3, 40, 2048), (4, 48, 7168), (5, 48, 7168), (16, 64, 2048), (9, 33, 3000), (40, 40, 4200),
    (64, 512, 512), (65, 48, 384), (100, 333, 1000), (128, 256, 640), (200, 272, 128), (257, 300, 200), (300, 520, 1152),
    (1, 47, 3000), (1, 47, 8000), (1, 4200, 200), (1, 4101, 2600), (1, 4101, 6000), (5, 4200, 200), (16, 4200, 2100),
    (7, 4101, 5000), (64, 4000, 300), (64, 4000, 1500), (64, 4090, 3000), (33, 2100, 3900), (70, 2100, 1300),
    (64, 5000, 1500), (50, 7100, 2100), (100, 4100, 700), (5, 16400, 100), (100, 9000, 100), (130, 16400, 100),
]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(w, M, N, K, bias):
    show(f"linear {M} x {N} x {K} bias {bias}")
    rng = np.random.default_rng(M + 7 * N + 11 * K)
    x = _acts(rng, M, K, 1.0)
    cw, sw = _weight(rng, N, K)
    b = O.f32_to_bf16(rng.standard_normal(N).astype(np.float32)) if bias else None
    wp = w.fp8b_prepack_weight(dev(cw))
    xd, swd = bf16_dev(x), dev(sw)
    bd = None if b is None else bf16_dev(b)
    y = w.fp8b_linear(xd, wp, swd, N, bias=bd)
    q, s = w.fp8b_quant(xd)
    y2 = w.fp8b_linear(q, wp, swd, N, x_scale=s, K=K, bias=bd)
    sync()
    got = bf16_host(y)
    assert np.array_equal(got, bf16_host(y2))
    show(f"  share of the tolerance used: {_hold(got, *F.quant(x), cw, sw, b, f'{M}x{N}x{K}'):.3f}")


@pytest.mark.parametrize("M,N,K", [(2100, 3900, 256), (3000, 2900, 130), (4096, 2048, 640), (2050, 4100, 1100),
                                   (1024, 4000, 1024), (600, 4000, 1024), (150, 4096, 2000), (150, 200, 7000),
                                   (4100, 4100, 128), (333, 16400, 600), (2000, 300, 2000)])
def test_linear_many_tiles(w, M, N, K):
    """Sizes of every tile height, ragged on every side: every output of sampled rows."""
    show(f"linear {M} x {N} x {K}")
    rng = np.random.default_rng(M + N + K)
    x = _acts(rng, M, K, 1.0)
    cw, sw = _weight(rng, N, K)
    b = O.f32_to_bf16(rng.standard_normal(N).astype(np.float32))
    room = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    w.fp8b_linear(bf16_dev(x), w.fp8b_prepack_weight(dev(cw)), dev(sw), N, bias=bf16_dev(b), y=room[1:M + 1])
    sync()
    assert (room[0] == 7).all() and (room[M + 1] == 7).all()
    pick = np.unique(np.r_[0:3, 14:18, 127:130, 254:258, 1000:1003, M - 3:M])
    pick = pick[pick < M]
    q, s = F.quant(x[pick])
    _hold(bf16_host(room[1:M + 1])[pick], q, s, cw, sw, b)
    # and the product of the codes is the same row by row as in a small call
    y2 = w.fp8b_linear(bf16_dev(x)[M - 5:], w.fp8b_prepack_weight(dev(cw)), dev(sw), N, bias=bf16_dev(b))
    sync()
    _hold(bf16_host(y2), *F.quant(x[M - 5:]), cw, sw, b)


@pytest.mark.parametrize("M", [1, 8, 40, 70, 300])
def test_linear_rows_do_not_depend_on_the_batch(w, M):
    """Row 0 alone and inside a batch: held to the same tolerance, and rows past M stay as they are."""
    rng = np.random.default_rng(M)
    N, K = 144, 896
    x = _acts(rng, M, K)
    cw, sw = _weight(rng, N, K)
    wp = w.fp8b_prepack_weight(dev(cw))
    room = torch.full((M + 2, N + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    w.fp8b_linear(bf16_dev(x), wp, dev(sw), N, y=room[1:M + 1, 8:8 + N])
    sync()
    r = room.float().cpu().numpy()
    assert (r[0] == 7).all() and (r[-1] == 7).all() and (r[:, :8] == 7).all() and (r[:, 8 + N:] == 7).all()
    _hold(bf16_host(room[1:M + 1, 8:8 + N]), *F.quant(x), cw, sw)


def test_linear_strided_input_and_scale_alg(w):
    rng = np.random.default_rng(12)
    x = _acts(rng, 70, 1000)
    cw, sw = _weight(rng, 80, 520)
    wp = w.fp8b_prepack_weight(dev(cw))
    for lo in (16, 5):
        for alg in (0, 1):
            y = w.fp8b_linear(bf16_dev(x)[:, lo:lo + 520], wp, dev(sw), 80, scale_alg=alg)
            sync()
            _hold(bf16_host(y), *F.quant(x[:, lo:lo + 520], 0, alg), cw, sw)
    # codes inside wider rows
    q, s = F.quant(x[:, :520])
    wide = torch.zeros((70, 640 + 64), dtype=torch.uint8, device=DEV)
    wide[:, 32:32 + 640] = dev(q)
    y = w.fp8b_linear(wide[:, 32:32 + 640], wp, dev(sw), 80, x_scale=dev(s), K=520)
    sync()
    _hold(bf16_host(y), q, s, cw, sw)


@pytest.mark.parametrize("M", [3, 80, 260])
def test_linear_exact_small_integers(w, M):
    """Codes that are small integers and unit scales: every sum is exact, the output its BF16."""
    rng = np.random.default_rng(M)
    N, K = 200, 640
    xi = rng.integers(-3, 4, (M, K)).astype(np.float32)
    wi = rng.integers(-2, 3, (N, K)).astype(np.float32)
    q = O.mx.e4m3_encode(xi)
    s = np.ones((5, M), np.float32)
    y = w.fp8b_linear(dev(q), w.fp8b_prepack_weight(dev(O.mx.e4m3_encode(wi))), dev(np.ones((2, 5), np.float32)), N,
                      x_scale=dev(s))
    sync()
    assert np.array_equal(bf16_host(y), O.f32_to_bf16((xi @ wi.T).astype(np.float32)))


@pytest.mark.parametrize("M,N", [(1, 300), (80, 300), (260, 300), (5000, 2000)])
def test_linear_every_scale_belongs_to_its_block(w, M, N):
    """One code per block, scales that are distinct powers of two: a scale of a wrong block shows."""
    K = 512
    q = np.zeros((M, K), np.uint8)
    cw = np.zeros((N, K), np.uint8)
    for b in range(4):
        q[:, 128 * b + 17 * b] = 0x38
        cw[:, 128 * b + 17 * b] = 0x38
    s = 2.0 ** (np.arange(4)[:, None] + 4.0 * (np.arange(M) % 3)[None])
    sw = 2.0 ** (-8.0 * (np.arange(-(-N // 128)) % 3)[:, None] + 2.0 * np.arange(4)[None])
    s, sw = s.astype(np.float32), sw.astype(np.float32)
    y = w.fp8b_linear(dev(q), w.fp8b_prepack_weight(dev(cw)), dev(sw), N, x_scale=dev(s))
    sync()
    want = F.product64(q, s, cw, sw)
    assert np.array_equal(bf16_host(y), O.f32_to_bf16(want.astype(np.float32)))


def test_linear_non_finite_values_stay_in_their_row_and_column(w):
    rng = np.random.default_rng(1)
    for M in (5, 90):
        x = _acts(rng, M, 256)
        x[3, 200] = 0x7FC0
        x[4, 10] = 0x7F80
        cw, sw = _weight(rng, 40, 256)
        cw[7, 3] = 0x7F
        y = w.fp8b_linear(bf16_dev(x), w.fp8b_prepack_weight(dev(cw)), dev(sw), 40)
        sync()
        v = y.float().cpu().numpy()
        # a NaN makes the block's scale NaN; an infinity makes it infinite, times a finite
        # sum of codes: an infinity, or NaN where that sum is 0
        nan = ~np.isfinite(v)
        assert np.isnan(v[3]).all() and nan[4].all() and np.isnan(v[:4, 7]).all() and nan[:, 7].all()
        keep = np.ones((M, 40), bool)
        keep[[3, 4]] = False
        keep[:, 7] = False
        assert not nan[keep].any()


# ------------------------------------------------------------------ grouped
GROUPED = [  # counts, N, K
    ([12, 7, 0, 19], 64, 64), ([1], 16, 128), ([0, 0, 5, 0], 130, 300), ([64, 65, 1, 0, 16, 17], 272, 256),
    ([129, 0, 300, 3], 144, 384), ([1] * 40, 48, 200), ([0] * 31 + [70], 80, 128), ([256, 257, 511], 520, 640),
    # 64 tiles and more, of one, two and three column groups; 63
    ([2] * 70, 130, 200), ([3, 0, 1] * 33, 272, 128), ([1, 129] * 22, 600, 130), ([1] * 63, 272, 128), ([1] * 64, 530, 100),
]


@pytest.mark.parametrize("exact", [False, True])
@pytest.mark.parametrize("indexed", [False, True])
@pytest.mark.parametrize("counts,N,K", GROUPED)
def test_grouped(w, counts, N, K, indexed, exact):
    show(f"grouped {counts if len(counts) < 9 else len(counts)} {N} x {K} indexed {indexed} exact {exact}")
    rng = np.random.default_rng(len(counts) + N + K)
    g = np.array(counts, np.int64)
    used, E = int(g.sum()), len(g)
    R = used + 5                                  # rows past the counts stay as they are
    T = 23 if indexed else R
    x = _acts(rng, T, K, 1.0)
    idx = rng.integers(0, T, R).astype(np.int32) if indexed else np.arange(R, dtype=np.int32)
    cw, sw = _weight(rng, E, N, K)
    q, s = w.fp8b_quant(bf16_dev(x))
    y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    w.fp8b_grouped_gemm(q, s, dev(g), w.fp8b_prepack_weight(dev(cw)), dev(sw), N, K=K,
                        row_index=dev(idx) if indexed else None, y=y, exact=exact)
    sync()
    got = bf16_host(y)
    assert (y[used:] == 7).all()
    qo, so = F.quant(x)
    r = 0
    for e in range(E):
        i = idx[r:r + g[e]]
        if len(i):
            _hold(got[r:r + g[e]], qo[i], np.ascontiguousarray(so[:, i]), cw[e], sw[e], what=f"expert {e}",
                  exact=exact)
        r += int(g[e])


def test_grouped_index_is_clamped(w):
    rng = np.random.default_rng(3)
    x = _acts(rng, 9, 128)
    cw, sw = _weight(rng, 2, 32, 128)
    idx = np.array([0, -1, 8, 9, 1 << 30, -(1 << 31), 4], np.int32)
    q, s = w.fp8b_quant(bf16_dev(x))
    wp = w.fp8b_prepack_weight(dev(cw))
    g = dev(np.array([3, 4], np.int64))
    y = w.fp8b_grouped_gemm(q, s, g, wp, dev(sw), 32, row_index=dev(idx))
    z = w.fp8b_grouped_gemm(q, s, g, wp, dev(sw), 32, row_index=dev(np.clip(idx, 0, 8).astype(np.int32)))
    sync()
    assert torch.equal(y, z)


def test_grouped_bad_counts_stay_in_bounds(w):
    """Counts past R or negative: rows [0, R) may be anything, nothing outside is written."""
    rng = np.random.default_rng(6)
    x = _acts(rng, 40, 128)
    cw, sw = _weight(rng, 3, 48, 128)
    q, s = w.fp8b_quant(bf16_dev(x))
    wp = w.fp8b_prepack_weight(dev(cw))
    for counts in ([30, 30, 30], [-5, 20, 90], [0, 0, 1000], [70, 1, 1]):
        room = torch.full((44, 48), 7.0, dtype=torch.bfloat16, device=DEV)
        w.fp8b_grouped_gemm(q, s, dev(np.array(counts, np.int64)), wp, dev(sw), 48, y=room[2:42])
        sync()
        assert (room[:2] == 7).all() and (room[42:] == 7).all()


# ------------------------------------------------------------------ chain and layer
MOE = [  # counts, H, I
    ([12, 7, 0, 19], 64, 32), ([3, 0, 1], 200, 100), ([70, 130, 0, 2, 33], 384, 256), ([1] * 9, 130, 68),
    ([300, 20, 80], 256, 192),
]


def _experts(w, rng, E, H, I):
    c13, s13 = _weight(rng, E, 2 * I, H)
    c2, s2 = _weight(rng, E, H, I)
    return (c13, s13, c2, s2), (w.fp8b_prepack_weight(dev(c13)), dev(s13), w.fp8b_prepack_weight(dev(c2)), dev(s2))


@pytest.mark.parametrize("counts,H,I", MOE)
def test_chain(w, counts, H, I):
    show(f"chain {counts} H {H} I {I}")
    rng = np.random.default_rng(H + I)
    g = np.array(counts, np.int64)
    R, E = int(g.sum()), len(g)
    x = _acts(rng, R, H)
    (c13, s13, c2, s2), W = _experts(w, rng, E, H, I)
    gl, xd = dev(g), bf16_dev(x)
    y = w.fp8b_moe_grouped(xd, gl, *W, I)
    q, s = w.fp8b_quant(xd)
    y2 = w.fp8b_moe_grouped(q, gl, *W, I, H=H, x_scale=s)
    # the chain equals its stages, and every stage is held on the GPU's own input
    h = w.fp8b_grouped_gemm(q, s, gl, W[0], W[1], 2 * I, K=H, exact=True)
    q2, sc2 = w.fp8b_quant(h, act=w.ACT_SWIGLU)
    y3 = w.fp8b_grouped_gemm(q2, sc2, gl, W[2], W[3], H, K=I)
    sync()
    assert torch.equal(y, y2) and torch.equal(y, y3)
    qo, so = F.quant(x)
    q2o, s2o = F.quant(bf16_host(h), 1)
    assert np.array_equal(host(q2), q2o) and np.array_equal(host(sc2), s2o)
    r = 0
    for e in range(E):
        a, b = r, r + int(g[e])
        if b > a:
            _hold(bf16_host(h)[a:b], qo[a:b], np.ascontiguousarray(so[:, a:b]), c13[e], s13[e], what=f"W13 {e}",
                  exact=True)
            _hold(bf16_host(y)[a:b], q2o[a:b], np.ascontiguousarray(s2o[:, a:b]), c2[e], s2[e], what=f"W2 {e}")
        r = b


@pytest.mark.parametrize("T,k,E,H,I,G,keep", [(1, 2, 4, 64, 32, 1, 1), (16, 8, 32, 256, 128, 4, 2), (130, 4, 16, 200, 72, 2, 1),
                                              (257, 6, 48, 384, 192, 8, 4), (600, 2, 3, 128, 128, 1, 1)])
def test_router_to_layer(w, T, k, E, H, I, G, keep):
    """The operators one after the other as a server runs them; the layer equals its stages."""
    show(f"layer T {T} k {k} E {E} H {H} I {I}")
    rng = np.random.default_rng(T + E)
    x = _acts(rng, T, H)
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[0, :E - 1] = -np.inf                        # one expert only: the other slots are dropped
    _, W = _experts(w, rng, E, H, I)
    xd = bf16_dev(x)
    ids, wts = w.moe_gate(dev(l), k, scoring=w.GATE_SIGMOID, n_group=G, topk_group=keep, scale=1.5)
    out = w.fp8b_moe_layer(xd, ids, wts, *W, I)
    gl, rt, pr = w.moe_route(ids, E)
    q, s = w.fp8b_quant(xd)
    h = w.fp8b_grouped_gemm(q, s, gl, W[0], W[1], 2 * I, K=H, row_index=rt, exact=True)
    q2, sc2 = w.fp8b_quant(h, act=w.ACT_SWIGLU)
    y = w.fp8b_grouped_gemm(q2, sc2, gl, W[2], W[3], H, K=I)
    out2 = w.moe_combine(y, pr, wts)
    sync()
    assert torch.equal(out, out2)
    # an oracle of the whole: gate in float64, then the combine over the GPU's own expert rows
    want, ww = O.fp8b.gate(l, k, None, "sigmoid", G, keep, True, 1.5)
    assert np.array_equal(host(ids), want) and (want[0, 1:] == -1).all()
    assert np.array_equal(bf16_host(out), O.moe_io.combine(bf16_host(y), host(pr), host(wts)))


def test_layer_workspace_is_rewritten(w):
    """A smaller call in a larger call's workspace, filled with NaN first."""
    rng = np.random.default_rng(2)
    E, H, I, k = 8, 256, 128, 2
    _, W = _experts(w, rng, E, H, I)
    ws = torch.full((w.fp8b_moe_layer_workspace_bytes(64, k, E, H, I),), 0xFF, dtype=torch.uint8, device=DEV)
    for T in (64, 5, 33):
        xd = bf16_dev(_acts(rng, T, H))
        ids, wts = w.moe_gate(dev(rng.standard_normal((T, E)).astype(np.float32)), k)
        a = w.fp8b_moe_layer(xd, ids, wts, *W, I, workspace=ws)
        b = w.fp8b_moe_layer(xd, ids, wts, *W, I)
        sync()
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()


def test_group_check_refuses_bad_counts(w, monkeypatch):
    monkeypatch.setenv("W8A8_CHECK", "1")
    rng = np.random.default_rng(0)
    q, s = w.fp8b_quant(bf16_dev(_acts(rng, 8, 128)))
    cw, sw = _weight(rng, 2, 16, 128)
    wp = w.fp8b_prepack_weight(dev(cw))
    w.fp8b_grouped_gemm(q, s, dev(np.array([3, 5], np.int64)), wp, dev(sw), 16)
    for counts in ([-1, 5], [8, 1]):
        with pytest.raises(w.W8A8Error) as err:
            w.fp8b_grouped_gemm(q, s, dev(np.array(counts, np.int64)), wp, dev(sw), 16)
        assert err.value.status == 2


# ------------------------------------------------------------------ graphs and streams
def test_gate_and_layer_in_a_graph(w):
    rng = np.random.default_rng(9)
    T, k, E, H, I = 40, 4, 16, 256, 128
    _, W = _experts(w, rng, E, H, I)
    x = [bf16_dev(_acts(rng, T, H)) for _ in range(3)]
    l = [dev(rng.standard_normal((T, E)).astype(np.float32)) for _ in range(3)]
    xin, lin = x[0].clone(), l[0].clone()
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    wts = torch.empty((T, k), device=DEV)
    out = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty((w.fp8b_moe_layer_workspace_bytes(T, k, E, H, I),), dtype=torch.uint8, device=DEV)

    def step(xi, li, o, room):
        w.moe_gate(li, k, scoring=w.GATE_SIGMOID, n_group=4, topk_group=2, ids=ids, weights=wts)
        w.fp8b_moe_layer(xi, ids, wts, *W, I, out=o, workspace=room)

    step(xin, lin, out, ws)
    sync()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(xin, lin, out, ws)
    for r in range(4):
        xin.copy_(x[r % 3])
        lin.copy_(l[r % 3])
        out.fill_(3.0)
        ws.fill_(0xFF)
        g.replay()
        sync()
        got = out.clone()
        ref = torch.empty_like(out)
        step(x[r % 3], l[r % 3], ref, torch.empty_like(ws))
        sync()
        assert torch.equal(got, ref)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_linear_in_a_graph(w, M):
    rng = np.random.default_rng(M)
    N, K = 272, 1024
    cw, sw = _weight(rng, N, K)
    wp, swd = w.fp8b_prepack_weight(dev(cw)), dev(sw)
    x = [bf16_dev(_acts(rng, M, K)) for _ in range(3)]
    xin = x[0].clone()
    y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty((w.fp8b_linear_workspace_bytes(M, N, K),), dtype=torch.uint8, device=DEV)
    w.fp8b_linear(xin, wp, swd, N, y=y, workspace=ws)
    sync()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.fp8b_linear(xin, wp, swd, N, y=y, workspace=ws)
    for r in range(4):
        xin.copy_(x[r % 3])
        y.fill_(3.0)
        ws.fill_(0xFF)
        g.replay()
        sync()
        got = y.clone()
        ref = w.fp8b_linear(x[r % 3], wp, swd, N)
        sync()
        assert torch.equal(got, ref)


def test_two_streams_with_their_own_workspaces(w):
    rng = np.random.default_rng(10)
    T, k, E, H, I = 64, 2, 8, 512, 256
    _, W = _experts(w, rng, E, H, I)
    x = [bf16_dev(_acts(rng, T, H)) for _ in range(2)]
    l = [dev(rng.standard_normal((T, E)).astype(np.float32)) for _ in range(2)]
    want = []
    for i in range(2):
        want.append(w.fp8b_moe_layer(x[i], *w.moe_gate(l[i], k), *W, I))
    sync()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(w.fp8b_moe_layer(x[i], *w.moe_gate(l[i], k), *W, I))
    sync()
    for i in range(2):
        assert all(torch.equal(want[i], g) for g in got[i])


# ------------------------------------------------------------------ infinities
@pytest.mark.parametrize("alg", [0, 1])
@pytest.mark.parametrize("sign", [0x0000, 0x8000])
def test_quant_infinity_is_a_nan_code(w, sign, alg):
    """An infinite value makes its block's scale infinite: v / scale is NaN for it and 0 for the
    finite values of the block. A block with a NaN has scale NaN and codes 0."""
    rng = np.random.default_rng(7)
    x = _acts(rng, 5, 300)
    x[1, 130] = 0x7F80 | sign
    x[2, [0, 9]] = 0x7F80 | sign
    x[3, 299] = 0x7FC0 | sign
    for act, xs in ((0, x), (1, np.concatenate([x, np.full((5, 300), 0x3F80, np.uint16)], 1))):
        q, s = w.fp8b_quant(bf16_dev(xs), act=act, scale_alg=alg)
        sync()
        q, s = host(q), host(s)
        qo, so = F.quant(xs, act, alg)
        if not (act and sign):                           # silu(-inf) is NaN in the fixed sequence
            assert np.isinf(s[1, 1]) and (q[1, 130] & 0x7F) == 0x7F and not (np.delete(q[1, 128:256], 2) & 0x7F).any()
            assert np.isinf(s[0, 2]) and (q[2, [0, 9]] & 0x7F == 0x7F).all() and not (q[2, 1:9] & 0x7F).any()
        assert np.isnan(s[2, 3]) and not (q[3, 256:] & 0x7F).any()
        nan = (qo & 0x7F) == 0x7F
        assert np.array_equal(s, so, equal_nan=True) and np.array_equal((q & 0x7F) == 0x7F, nan)
        assert np.array_equal(q[~nan], qo[~nan])


@pytest.mark.parametrize("M", [5, 40, 300])
def test_linear_infinite_activation_gives_nan(w, M):
    """The codes of an infinity are NaN, and so is every output of its row; no other row feels it."""
    rng = np.random.default_rng(M)
    x = _acts(rng, M, 256)
    cw, sw = _weight(rng, 40, 256)
    wp, swd = w.fp8b_prepack_weight(dev(cw)), dev(sw)
    clean = w.fp8b_linear(bf16_dev(x), wp, swd, 40)
    x[3, 10], x[4, 200] = 0x7F80, 0xFF80
    y = w.fp8b_linear(bf16_dev(x), wp, swd, 40)
    q, s = w.fp8b_quant(bf16_dev(x))
    z = w.fp8b_grouped_gemm(q, s, dev(np.array([M], np.int64)), wp, swd[None], 40, exact=True)
    sync()
    for v in (y, z):
        v = v.float().cpu().numpy()
        assert np.isnan(v[[3, 4]]).all()
        assert np.isfinite(np.delete(v, [3, 4], 0)).all()
    keep = np.delete(np.arange(M), [3, 4])
    assert np.array_equal(bf16_host(y)[keep], bf16_host(clean)[keep])


# ------------------------------------------------------------------ the wide tiles' walk
WIDE = [(8192, 8192, 256), (8200, 8100, 384), (12300, 8192, 200), (9000, 12300, 512)]  # M, N, K


@pytest.mark.parametrize("M,N,K", WIDE)
def test_linear_wide_tiles_one_after_the_other(w, M, N, K):
    """More 256 x 256 tiles than workgroups, so that each walks over four to seven, at two to four
    blocks of K: one code per block and scales that are powers of two, different from tile to
    tile, so that a block, scale or row of another tile shows. Every output is exact."""
    show(f"linear {M} x {N} x {K}")
    B = -(-K // 128)
    q = torch.zeros((M, 128 * B), dtype=torch.uint8, device=DEV)
    cw = torch.zeros((N, K), dtype=torch.uint8, device=DEV)
    for b in range(B):
        # 1.0 on one column of the block for the rows, on the same one for the columns
        q[:, 128 * b + 17 * b] = 0x38
        cw[:, 128 * b + 17 * b] = 0x38
    m = torch.arange(M, device=DEV)
    n = torch.arange(-(-N // 128), device=DEV)
    b = torch.arange(B, device=DEV)
    # exponents of the blocks' terms lie within the 8 bits of a BF16, and move with the row, the
    # row's tile, the column's block and the block of K
    ea = (b[:, None] + (m % 7 + m // 256 % 5)[None]) % 4
    eb = 2 * ((b[None] + n[:, None]) % 2) + (n // 2 % 3)[:, None] * 8
    s, sw = (2.0 ** ea).float().contiguous(), (2.0 ** eb).float().contiguous()
    y = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    w.fp8b_linear(q, w.fp8b_prepack_weight(cw), sw, N, x_scale=s, K=K, y=y[:M])
    sync()
    want = s.t() @ sw.t()                                # exact in float32
    want = want.repeat_interleave(128, 1)[:, :N].to(torch.bfloat16)
    bad = (y[:M] != want).nonzero()
    assert bad.numel() == 0, (len(bad), bad[:4].tolist())
    assert (y[M] == 7).all()


def test_linear_wide_tiles_of_random_values(w):
    """Four tiles a workgroup, ragged on every side: every output of two rows of every row of tiles."""
    M, N, K = 8200, 8200, 400
    rng = np.random.default_rng(1)
    x = _acts(rng, M, K, 1.0)
    cw, sw = _weight(rng, N, K)
    b = O.f32_to_bf16(rng.standard_normal(N).astype(np.float32))
    y = w.fp8b_linear(bf16_dev(x), w.fp8b_prepack_weight(dev(cw)), dev(sw), N, bias=bf16_dev(b))
    sync()
    first = np.arange(0, M, 256)
    pick = np.unique(np.r_[first + rng.integers(0, 8, len(first)), np.minimum(first + rng.integers(8, 256, len(first)), M - 1)])
    _hold(bf16_host(y)[pick], *F.quant(x[pick]), cw, sw, b)


# ------------------------------------------------------------------ offsets past 32 bits
def test_quant_and_linear_past_32_bit_offsets(w):
    """More than 2^32 bytes of codes and elements of x: rows on either side of every 2^32."""
    M, N, K = 1 << 19 | 4097, 40, 8200
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn((M, K), generator=g, device=DEV, dtype=torch.bfloat16)
    cw, sw = _weight(np.random.default_rng(0), N, K)
    wp, swd = w.fp8b_prepack_weight(dev(cw)), dev(sw)
    Kp = 128 * F.blocks(K)
    pick = np.unique([0, 1, (1 << 31) // K, (1 << 32) // K, (1 << 32) // K + 1, (1 << 32) // Kp, (1 << 32) // Kp + 1, M - 2, M - 1])
    rows = torch.from_numpy(pick).to(DEV)
    xh = bf16_host(x[rows])
    y = w.fp8b_linear(x, wp, swd, N)
    q, s = w.fp8b_quant(x)
    z = w.fp8b_linear(q, wp, swd, N, x_scale=s, K=K)
    sync()
    qo, so = F.quant(xh)
    assert np.array_equal(host(q[rows]), qo) and np.array_equal(host(s[:, rows]), so)
    _hold(bf16_host(y[rows]), qo, so, cw, sw)
    assert torch.equal(y, z)
