"""Refusals and sizes of the router and the block-scaled FP8 entry points (CPU only):
every call fails its checks before anything is launched, or does nothing."""

from __future__ import annotations

import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

from tests.test_kernel_resources import CSRC, MAX_SCRATCH, _flags, _hipcc, _innermost_mfma_loops

OK, NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4, 5
P = ctypes.c_void_p(256)      # never dereferenced: the checks fail first
ODD = ctypes.c_void_p(257)


@pytest.fixture(scope="module")
def w():
    import moe_token_amax_amd as w
    return w


def _gate(L, logits=P, dtype=0, T=4, E=64, ld=64, bias=None, scoring=1, n_group=1, topk_group=1, top_k=2, renorm=1,
          scale=1.0, ids=P, weights=P):
    return L.w8a8_moe_gate(logits, dtype, T, E, ld, bias, scoring, n_group, topk_group, top_k, renorm, scale, ids,
                           weights, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(ld=63), SHAPE), (dict(top_k=0), SHAPE),
    (dict(T=1 << 30, top_k=2), SHAPE), (dict(T=1 << 26), SHAPE), (dict(T=1 << 25, top_k=64, E=64), SHAPE), (dict(dtype=3), UNSUPPORTED), (dict(scoring=2), UNSUPPORTED),
    (dict(E=1025, ld=1025), UNSUPPORTED), (dict(n_group=0), SHAPE), (dict(n_group=3), SHAPE),
    (dict(E=130, ld=130, n_group=65), SHAPE), (dict(n_group=4, topk_group=5), SHAPE), (dict(topk_group=0), SHAPE),
    (dict(top_k=65, E=128, ld=128), SHAPE), (dict(n_group=8, topk_group=1, top_k=9), SHAPE),
    (dict(scale=math.inf), SHAPE), (dict(scale=math.nan), SHAPE), (dict(logits=None), NULL), (dict(ids=None), NULL),
    (dict(weights=None), NULL), (dict(logits=ODD), ALIGN), (dict(bias=ODD), ALIGN), (dict(ids=ODD), ALIGN),
    (dict(T=0, logits=None, ids=None, weights=None), OK)])
def test_gate_refusals(w, kw, status):
    assert _gate(w.lib, **kw) == status
    assert (w.lib.w8a8_last_error() == b"") == (status == OK)


def _quant(L, x=P, M=4, K=64, ldx=64, act=0, alg=0, q=P, s=P):
    return L.w8a8_fp8b_quant(x, M, K, ldx, act, alg, q, s, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=200000, ldx=200000), SHAPE), (dict(M=1 << 30), SHAPE), (dict(M=(1 << 28) - 16), SHAPE),
    (dict(ldx=63), SHAPE), (dict(act=1, ldx=127), SHAPE), (dict(act=2), UNSUPPORTED), (dict(alg=2), UNSUPPORTED),
    (dict(x=None), NULL), (dict(q=None), NULL), (dict(s=None), NULL), (dict(x=ODD), ALIGN),
    (dict(q=ctypes.c_void_p(264)), ALIGN), (dict(s=ODD), ALIGN), (dict(M=0, x=None, q=None, s=None), OK)])
def test_quant_refusals(w, kw, status):
    assert _quant(w.lib, **kw) == status


def _linear(L, x=P, ldx=64, xs=None, M=4, K=64, wp=P, ws=P, N=8, bias=None, y=P, ldy=8, alg=0, room=P, n=1 << 20):
    return L.w8a8_fp8b_linear(x, ldx, xs, M, K, wp, ws, N, bias, y, ldy, alg, room, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(M=1 << 28), SHAPE), (dict(N=0), SHAPE), (dict(N=(1 << 22) + 1, ldy=1 << 23), SHAPE), (dict(ldx=63), SHAPE),
    (dict(ldy=7), SHAPE), (dict(xs=P, ldx=64), SHAPE), (dict(alg=-1), UNSUPPORTED), (dict(x=None), NULL),
    (dict(wp=None), NULL), (dict(ws=None), NULL), (dict(y=None), NULL), (dict(wp=ctypes.c_void_p(264)), ALIGN),
    (dict(x=ODD), ALIGN), (dict(bias=ODD), ALIGN), (dict(xs=P, ldx=136), ALIGN),
    (dict(xs=P, ldx=128, x=ctypes.c_void_p(264)), ALIGN), (dict(n=100), WORKSPACE), (dict(room=None), WORKSPACE),
    (dict(room=ctypes.c_void_p(128)), WORKSPACE), (dict(M=0, x=None, wp=None, ws=None, y=None), OK)])
def test_linear_refusals(w, kw, status):
    assert _linear(w.lib, **kw) == status


def _grouped(L, a=P, s=P, rows=8, index=None, gl=P, R=8, E=4, N=16, K=64, wp=P, ws=P, y=P, room=P, n=1 << 20):
    return L.w8a8_fp8b_grouped_gemm(a, s, rows, index, gl, R, E, N, K, wp, ws, y, 0, room, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), UNSUPPORTED),
    (dict(R=1 << 28, rows=1 << 28, N=1 << 14), SHAPE),
    (dict(R=1 << 27, rows=1 << 27, N=1 << 14), UNSUPPORTED), (dict(R=1 << 27, rows=1 << 27, N=1 << 12), UNSUPPORTED), (dict(K=0), SHAPE), (dict(rows=7), SHAPE),
    (dict(rows=0, index=P), SHAPE), (dict(gl=None), NULL), (dict(a=None), NULL), (dict(gl=ctypes.c_void_p(260)), ALIGN),
    (dict(a=ctypes.c_void_p(264)), ALIGN), (dict(index=ODD), ALIGN), (dict(n=8), WORKSPACE), (dict(room=None), WORKSPACE),
    (dict(R=0, a=None, gl=None), OK)])
def test_grouped_refusals(w, kw, status):
    assert _grouped(w.lib, **kw) == status


def test_chain_and_layer_refusals(w):
    L = w.lib

    def chain(x=P, xs=None, gl=P, R=16, E=4, H=64, I=32, wp=P, alg=0, y=P, room=P, n=1 << 24):
        return L.w8a8_fp8b_moe_grouped(x, xs, gl, R, E, H, I, wp, P, wp, P, alg, y, room, n, None)

    def layer(x=P, T=4, H=64, ids=P, wts=P, k=2, E=4, I=32, wp=P, alg=0, out=P, room=P, n=1 << 24):
        return L.w8a8_fp8b_moe_layer(x, T, H, ids, wts, k, E, I, wp, P, wp, P, alg, out, room, n, None)

    assert chain(E=0) == SHAPE and chain(I=0) == SHAPE and chain(R=-1) == SHAPE and chain(E=2000) == UNSUPPORTED
    assert chain(alg=7) == UNSUPPORTED and chain(x=None) == NULL and chain(wp=ctypes.c_void_p(264)) == ALIGN
    assert chain(xs=P, x=ctypes.c_void_p(264)) == ALIGN and chain(n=64) == WORKSPACE and chain(room=None) == WORKSPACE
    assert chain(R=0, x=None) == OK
    assert layer(T=1 << 24, k=1) == SHAPE
    assert layer(T=-1) == SHAPE and layer(k=0) == SHAPE and layer(E=1025) == UNSUPPORTED and layer(H=0) == SHAPE
    assert layer(alg=2) == UNSUPPORTED and layer(ids=None) == NULL and layer(out=ODD) == ALIGN
    assert layer(n=64) == WORKSPACE and layer(room=ODD) == WORKSPACE and layer(T=0, x=None) == OK
    assert L.w8a8_fp8b_prepack_weight(P, 0, 16, 64, P, None) == SHAPE
    assert L.w8a8_fp8b_prepack_weight(None, 1, 16, 64, P, None) == NULL
    assert L.w8a8_fp8b_prepack_weight(P, 1, 16, 64, ctypes.c_void_p(264), None) == ALIGN


def test_sizes(w):
    assert w.fp8b_packed_bytes(1, 128, 256) == 128 * 256
    assert w.fp8b_packed_bytes(3, 17, 129) == 3 * 32 * 256       # N to 16, K to 128
    assert w.fp8b_linear_workspace_bytes(3, 16, 200) == 3 * 256 + 256
    assert w.fp8b_linear_workspace_bytes(0, 16, 200) == 0
    assert w.fp8b_moe_workspace_bytes(0, 4, 64, 32) == 0
    assert w.fp8b_moe_layer_workspace_bytes(4, 2, 4, 64, 32) > w.fp8b_moe_workspace_bytes(8, 4, 64, 32) - 8 * 128


def test_binding_refusals_without_a_gpu(w):
    t = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        w.moe_gate(t, 2)                                         # not on a GPU
    with pytest.raises(TypeError):
        w.moe_gate(torch.zeros((4, 64), dtype=torch.float64), 2)
    with pytest.raises(TypeError):
        w.fp8b_quant(t)
    with pytest.raises(TypeError):
        w.fp8b_linear(t, t, t, 8)
    b, u = t.to(torch.bfloat16), t.to(torch.uint8)
    with pytest.raises(ValueError):
        w.fp8b_quant(b)                                          # not on a GPU
    with pytest.raises(ValueError):
        w.fp8b_grouped_gemm(torch.zeros((4, 100), dtype=torch.uint8), t, torch.zeros(2, dtype=torch.int64), u, t, 8)
    with pytest.raises(ValueError):
        w.fp8b_moe_layer(b, torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2)), u, t[None], u, t[None], 32)


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not available")
@pytest.mark.parametrize("src", ["fp8b.hip", "gate.hip"])
def test_kernels_keep_out_of_scratch(src, tmp_path):
    out = tmp_path / "k.s"
    r = subprocess.run([_hipcc(), *_flags(), "-S", os.path.join(CSRC, src), "-o", str(out),
                        "-Rpass-analysis=kernel-resource-usage"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    names = re.findall(r"Function Name: (\S+)", r.stderr)
    scratch = [int(v) for v in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", r.stderr)]
    assert names and len(names) == len(scratch)
    assert not {n: s for n, s in zip(names, scratch) if s > MAX_SCRATCH}
    lines = out.read_text().split("\n")
    assert not any("v_pk_fma_f32" in x or "v_pk_mul_f32" in x or "v_pk_add_f32" in x for x in lines)
    if src == "fp8b.hip":
        loops = _innermost_mfma_loops(lines)
        assert loops
        assert not [1 for a, b in loops for x in lines[a:b + 1] if "scratch_" in x]


def test_one_workgroup_too_many_is_refused(w):
    """Sizes whose launch would have exactly 2^32 threads; one less passes this check (and fails a
    later one: nothing is launched here)."""
    assert _gate(w.lib, T=(1 << 26) - 3, logits=None) == SHAPE and _gate(w.lib, T=(1 << 26) - 1, logits=None) == SHAPE
    assert _gate(w.lib, T=(1 << 26) - 4, logits=None) == NULL

    def chain(R, xs=None):
        return w.lib.w8a8_fp8b_moe_grouped(P, xs, P, R, 4, 64, 32, P, P, P, P, 0, P, P, 64, None)

    assert chain((1 << 28) - 17) == SHAPE and chain((1 << 28) - 31) == SHAPE
    assert chain((1 << 28) - 32) == WORKSPACE and chain((1 << 28) - 17, xs=P) == WORKSPACE
    assert _quant(w.lib, M=(1 << 28) - 17, q=None) == NULL


# ------------------------------------------------------------------ which kernel a linear's sizes take
def _costs():
    """The table of dense_kernel, as the source has it."""
    with open(os.path.join(CSRC, "fp8b.hip")) as f:
        src = f.read()
    rows = re.findall(r"\{(k\w+), (\d+), (\d+), ([\d.]+), ([\d.]+), ([\d.]+), ([\d.]+), (true|false)\}", src)
    names = re.search(r"enum DenseKernel \{([^}]*)\}", src).group(1).replace(",", " ").split()
    assert [r[0] for r in rows] == names
    return rows


def _dense_kernel(M, N, K):
    KB, best, least = -(-K // 128), None, 1e30
    for name, rows, cols, launch, per, first, full, two in _costs():
        rows, cols, launch, per, first, full = int(rows), int(cols), float(launch), float(per), float(first), float(full)
        if (name == "kTile256" and KB < 2) or ("Decode" in name and M > 65535 * 16):
            continue
        n = -(-M // rows) * -(-N // cols)
        rounds = n / 512.0 if two == "true" else float(-(-n // 256))
        us = launch + rounds * per + KB * max(first, rounds * full)
        if us < least:
            best, least = name, us
    return best


def _decode_sets(M, N, K):
    """Register sets of a decode kernel, None for a tile."""
    most = {"kDecode16": 8, "kDecode16x32": 8, "kDecode32": 4, "kDecode64": 2}.get(_dense_kernel(M, N, K))
    blocks = -(-(-(-K // 128)) // 8)
    return most and (min(2, most) if blocks <= 2 else min(4, most) if blocks <= 4 else most)


def test_linear_tests_reach_every_kernel():
    from tests import test_gpu_fp8b as g
    many = next(m for m in g.test_linear_many_tiles.pytestmark if m.name == "parametrize").args[1]
    sizes = [*g.LINEAR, *many, *g.WIDE]
    got = {}
    for s in sizes:
        got.setdefault((_dense_kernel(*s), _decode_sets(*s)), []).append(s)
    want = {("kDecode16", 2), ("kDecode16", 4), ("kDecode16", 8), ("kDecode16x32", 2), ("kDecode16x32", 4),
            ("kDecode16x32", 8), ("kDecode32", 2), ("kDecode32", 4), ("kDecode64", 2), ("kTile32", None), ("kTile64", None),
            ("kTile64x256", None), ("kTile128", None), ("kTile256", None)}
    assert set(got) == want, (want - set(got), set(got) - want)


def test_wide_tests_walk_over_several_tiles():
    """256 workgroups share the tiles: past 512 some have three, at two blocks of K and more."""
    from tests import test_gpu_fp8b as g
    for M, N, K in [*g.WIDE, (8200, 8200, 400)]:
        assert _dense_kernel(M, N, K) == "kTile256" and -(-M // 256) * -(-N // 256) > 512
    assert {-(-K // 128) for _, _, K in g.WIDE} >= {2, 3, 4}
