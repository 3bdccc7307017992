"""Plans and workspace sizes of the fused linears and the BF16 expert products (CPU
only): queries, and calls that fail their checks before anything is launched."""

from __future__ import annotations

import ctypes
import random

import pytest

OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4, 5
P = 256                       # an address that is never read


@pytest.fixture(scope="module")
def w():
    import moe_token_amax_amd as w
    return w


def _plan(w, kind, M, N, K, at=P, ld=None, act=0):
    p = w.Plan()
    ld = K if ld is None else ld
    if kind == "int8":
        st = w.lib.w8a8_linear_fused_plan(at, ld, M, N, K, ctypes.byref(p))
    else:
        st = w.lib.w8a8_bf16_linear_plan(at, ld, M, N, K, act, ctypes.byref(p))
    assert st == OK, w.lib.w8a8_last_error()
    return p


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_aligned_rows_need_no_room_for_a_copy(w, kind):
    """Prompts on wide tiles: their rows are copied, and room for that is asked for, only
    where an address, a stride or a width keeps the tiles from loading them."""
    p = _plan(w, kind, 8192, 4096, 7168)
    assert (p.tile_rows, p.tile_cols, p.k_parts, p.copied, p.tiles) == (256, 256, 1, 0, 512)
    assert p.workspace_bytes == 0
    bytes_row = 7168 * (1 if kind == "int8" else 2)
    for kw in (dict(at=P + 2), dict(ld=7170)):
        p = _plan(w, kind, 8192, 4096, 7168, **kw)
        assert p.copied == 1 and p.workspace_bytes == 8192 * bytes_row
    p = _plan(w, kind, 8192, 4096, 7168, ld=1 << 24)                  # past 32-bit offsets in a tile
    assert p.copied == 1 and p.workspace_bytes == 8192 * bytes_row
    p = _plan(w, kind, 8192, 4096, 7166)
    assert p.copied == 1 and p.workspace_bytes == 8192 * bytes_row    # to whole steps of 128 bytes


@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_a_call_asks_for_what_its_plan_says(w, kind):
    """One byte less than the plan's is refused, and the size query covers every plan."""
    rng = random.Random(3)
    size = w.linear_fused_workspace_bytes if kind == "int8" else w.bf16_linear_workspace_bytes
    asked = 0
    for _ in range(3000):
        M, N, K = (int(2 ** rng.uniform(0, b)) for b in (14, 14, 14))
        act = rng.choice([0, 1]) if kind == "bf16" and N % 2 == 0 else 0
        p = _plan(w, kind, M, N, K, P + rng.choice([0, 2]), K + rng.choice([0, 1, 8]), act)
        assert 0 <= p.workspace_bytes <= size(M, N, K)
        assert (p.k_parts > 1 or p.copied == 1) == (p.workspace_bytes > 0)
        p = _plan(w, kind, M, N, K, act=act)
        if not p.workspace_bytes:
            continue
        asked += 1
        a, n = ctypes.c_void_p(P), p.workspace_bytes - 1
        if kind == "int8":
            st = w.lib.w8a8_linear_fused(a, K, a, M, K, a, a, N, None, 0, None, 0, a, N, a, n, None)
        else:
            st = w.lib.w8a8_bf16_linear(a, K, M, K, a, N, None, act, None, 0, a, N, 0, a, n, None)
        assert st == WORKSPACE and b"%d workspace bytes" % p.workspace_bytes in w.lib.w8a8_last_error()
    assert asked > 200


def test_plan_refusals(w):
    L, p = w.lib, w.Plan()
    at = ctypes.byref(p)
    assert L.w8a8_linear_fused_plan(P, 64, -1, 8, 64, at) == SHAPE
    assert L.w8a8_linear_fused_plan(P, 63, 4, 8, 64, at) == SHAPE
    assert L.w8a8_linear_fused_plan(P, 64, 4, 8, 64, None) == NULL
    assert L.w8a8_bf16_linear_plan(P, 64, 4, 0, 64, 0, at) == SHAPE
    assert L.w8a8_bf16_linear_plan(P, 63, 4, 8, 64, 0, at) == SHAPE
    assert L.w8a8_bf16_linear_plan(P, 64, 4, 8, 64, 6, at) == UNSUPPORTED
    assert L.w8a8_bf16_linear_plan(P, 64, 4, 8, 64, 0, None) == NULL
    assert L.w8a8_fp8b_linear_plan(None, 63, 4, 8, 64, at) == SHAPE
    assert L.w8a8_fp8b_linear_plan(P, 64, 4, 8, 64, at) == SHAPE      # codes: rows of 128
    assert L.w8a8_fp8b_linear_plan(None, 64, 4, 8, 64, None) == NULL
    assert L.w8a8_bf16_grouped_plan(P, 63, 4, None, 4, 2, 16, 64, at) == SHAPE
    assert L.w8a8_bf16_grouped_plan(P, 64, 4, None, 4, 0, 16, 64, at) == SHAPE
    assert L.w8a8_bf16_grouped_plan(P, 64, 4, None, 4, 1025, 16, 64, at) == UNSUPPORTED
    assert L.w8a8_bf16_grouped_plan(P, 64, 4, None, 4, 2, 16, 64, None) == NULL
    for st in (L.w8a8_linear_fused_plan(None, 64, 0, 8, 64, at), L.w8a8_bf16_linear_plan(None, 64, 0, 8, 64, 0, at),
               L.w8a8_fp8b_linear_plan(None, 64, 0, 8, 64, at), L.w8a8_bf16_grouped_plan(None, 64, 0, None, 0, 2, 8, 64, at)):
        assert st == OK and p.tiles == p.workspace_bytes == 0


def test_output_over_the_rows_is_refused(w):
    """The workgroups of other columns still read the rows that one has written."""
    L, a, b = w.lib, ctypes.c_void_p(P), ctypes.c_void_p(2 * P)
    for M in (1, 64, 8192):
        assert L.w8a8_bf16_linear(a, 4096, M, 4096, b, 4096, None, 0, a, 4096, a, 4096, 0, b, 1 << 30, None) == UNSUPPORTED
        assert b"y lies over the rows" in L.w8a8_last_error()
        assert L.w8a8_linear_fused(a, 4096, b, M, 4096, b, b, 64, None, 0, None, 0, a, 64, b, 1 << 30, None) == UNSUPPORTED
    assert L.w8a8_bf16_grouped_gemm(a, 256, 8, None, b, 8, 2, 256, 256, b, 0, a, b, 1 << 20, None) == UNSUPPORTED


def test_fp8_plan(w):
    p = w.Plan()
    for M, N, K, codes, tile in [(1, 4096, 7168, False, (16, 16)), (1, 16384, 7168, False, (16, 32)),
                                 (333, 1000, 2000, True, (64, 32)), (8192, 4096, 7168, True, (256, 256)),
                                 (8192, 4096, 7168, False, (256, 256))]:
        assert w.lib.w8a8_fp8b_linear_plan(P if codes else None, -(-K // 128) * 128, M, N, K, ctypes.byref(p)) == OK
        assert (p.tile_rows, p.tile_cols, p.k_parts, p.copied) == (*tile, 1, 0)
        assert p.tiles == -(-M // tile[0]) * -(-N // tile[1])
        assert p.workspace_bytes == (0 if codes else w.fp8b_linear_workspace_bytes(M, N, K))


def test_grouped_plan(w):
    p, a = w.Plan(), ctypes.c_void_p(P)
    for at, ld, rows, index, R, E, N, K, tile in [
            (P, 1000, 1003, None, 1003, 7, 1412, 1000, (64, 128)), (P, 1400, 3600, None, 3600, 8, 4130, 1400, (256, 256)),
            (P, 1401, 3600, None, 3600, 8, 4130, 1401, (128, 256)), (P + 2, 1400, 3600, None, 3600, 8, 4130, 1400, (128, 256)),
            (P, 1400, 777, a, 3600, 8, 4130, 1400, (256, 256)), (P, 1 << 20, 4096, a, 3600, 8, 4130, 1400, (128, 256)),
            (P, 1 << 20, 4096, None, 3600, 8, 4130, 1400, (256, 256))]:
        assert w.lib.w8a8_bf16_grouped_plan(at, ld, rows, index, R, E, N, K, ctypes.byref(p)) == OK
        assert (p.tile_rows, p.tile_cols, p.k_parts, p.copied) == (*tile, 1, 0)
        assert 256 < p.workspace_bytes <= w.bf16_grouped_workspace_bytes(R, E, N, K)


KERNELS = [(16, 16), (16, 32), (32, 32), (64, 32), (32, 128), (64, 128), (64, 256), (128, 256), (256, 256)]
SPLITS = [(32, 128), (64, 128), (128, 256)]


@pytest.mark.parametrize("kind,act", [("bf16", 0), ("bf16", 1), ("int8", 0)])
def test_the_sizes_of_the_gpu_tests_reach_every_kernel_and_split(w, kind, act):
    """test_every_kernel and the linears' sizes: pinned, so that another cost of a kernel
    cannot move them off one unseen."""
    from tests.test_gpu_fused import PLANS, SIZES
    double = 2 if kind == "int8" else 1
    plans = [_plan(w, kind, M, N + N % 2 if act else N, K * double, act=act) for M, N, K in PLANS] + \
        [_plan(w, kind, M, N + N % 2 if act else N, K, act=act) for M, N, K in SIZES]
    whole = {(p.tile_rows, p.tile_cols) for p in plans if p.k_parts == 1}
    split = {(p.tile_rows, p.tile_cols) for p in plans if p.k_parts > 1}
    assert whole == set(KERNELS[act:]) and split == set(SPLITS)      # SwiGLU: pairs of 16 columns


# rows at the borders of the tiles, one by one to 600, then up to prompts
ROWS = sorted(set(range(600)) | {16 * i + d for i in range(38, 300, 3) for d in (-1, 0, 1)} |
              {8191, 8192, 8193, 32767, 32769, 65536, 1 << 20})


@pytest.mark.parametrize("kind", ["int8", "bf16"])
@pytest.mark.parametrize("N,K", [(4096, 7168), (4122, 6000), (1776, 7549), (16, 16384), (100, 130), (7168, 2048), (20, 15),
                                 (30000, 100)])
def test_linear_workspace_never_falls_as_rows_grow(w, kind, N, K):
    """A room made for the largest batch serves every smaller one."""
    size = w.linear_fused_workspace_bytes if kind == "int8" else w.bf16_linear_workspace_bytes
    sizes = [size(M, N, K) for M in ROWS]
    assert sizes[0] == 0
    falls = [(ROWS[i], sizes[i], ROWS[i + 1], sizes[i + 1]) for i in range(len(ROWS) - 1) if sizes[i] > sizes[i + 1]]
    assert not falls, falls[:3]


@pytest.mark.parametrize("E,N,K", [(2, 5346, 1499), (8, 4096, 7168), (64, 8192, 4096), (256, 4096, 4096), (7, 1412, 1000),
                                   (16, 2048, 2048), (1, 300, 200), (40, 30000, 512)])
def test_grouped_workspace_never_falls_as_rows_grow(w, E, N, K):
    sizes = [w.bf16_grouped_workspace_bytes(R, E, N, K) for R in ROWS]
    assert sizes[0] == 0
    falls = [(ROWS[i], sizes[i], ROWS[i + 1], sizes[i + 1]) for i in range(len(ROWS) - 1) if sizes[i] > sizes[i + 1]]
    assert not falls, falls[:3]


def test_grouped_workspace_covers_every_call(w):
    """A call that is given a byte less than it needs says how much that is."""
    rng = random.Random(4)
    a = ctypes.c_void_p(P)
    for _ in range(2000):
        R, E, N, K = int(2 ** rng.uniform(0, 15)), int(2 ** rng.uniform(0, 10)), int(2 ** rng.uniform(0, 13)), \
            int(2 ** rng.uniform(3, 13))
        st = w.lib.w8a8_bf16_grouped_gemm(a, K, R, None, a, R, E, N, K, a, 0, a, a, 0, None)
        assert st == WORKSPACE
        need = int(w.lib.w8a8_last_error().split(b"needs ")[1].split()[0])
        assert 256 < need <= w.bf16_grouped_workspace_bytes(R, E, N, K)
