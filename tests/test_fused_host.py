"""Refusals and sizes of the RMS norm, the fused epilogues and the BF16 products (CPU
only): every call fails its checks before anything is launched, or does nothing."""

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
P8 = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def w():
    import moe_token_amax_amd as w
    return w


def _norm(L, fmt, x=P, ldx=64, res=None, ldr=64, h=P, ldh=64, weight=P, eps=1e-6, M=4, K=64, y=None, ldy=64, q=P,
          ldq=64, s=P, alg=0):
    lead = (x, ldx, res, ldr, h, ldh, weight, eps, M, K, y, ldy)
    if fmt == "bf16":
        return L.w8a8_rms_norm(*lead, None)
    if fmt == "int8":
        return L.w8a8_rms_norm_quant(*lead, q, ldq, s, None)
    return {"fp8": L.w8a8_fp8b_rms_norm_quant, "mx": L.w8a8_mx_rms_norm_quant}[fmt](*lead, alg, q, s, None)


@pytest.mark.parametrize("fmt,kw,status", [
    ("int8", dict(M=-1), SHAPE), ("int8", dict(M=1 << 31), SHAPE), ("int8", dict(K=0), SHAPE),
    ("int8", dict(K=133145, ldx=1 << 20, ldq=1 << 20), SHAPE), ("int8", dict(ldx=63), SHAPE),
    ("int8", dict(res=P, ldr=63), SHAPE), ("int8", dict(res=P, ldh=63), SHAPE), ("int8", dict(y=P, ldy=63), SHAPE),
    ("int8", dict(ldq=63), SHAPE), ("int8", dict(eps=-1e-9), SHAPE), ("int8", dict(eps=math.nan), SHAPE),
    ("int8", dict(eps=math.inf), SHAPE), ("int8", dict(x=None), NULL), ("int8", dict(q=None), NULL),
    ("int8", dict(s=None), NULL), ("int8", dict(res=P, h=None), NULL), ("int8", dict(x=ODD), ALIGN),
    ("int8", dict(weight=ODD), ALIGN), ("int8", dict(res=ODD), ALIGN), ("int8", dict(res=P, h=ODD), ALIGN),
    ("int8", dict(y=ODD), ALIGN), ("int8", dict(s=ctypes.c_void_p(258)), ALIGN),
    ("int8", dict(M=0, x=None, q=None, s=None), OK), ("bf16", dict(y=None), NULL), ("bf16", dict(M=0), OK),
    ("fp8", dict(alg=2), UNSUPPORTED), ("fp8", dict(q=P8), ALIGN), ("fp8", dict(q=None), NULL),
    ("mx", dict(K=48), UNSUPPORTED), ("mx", dict(alg=-1), UNSUPPORTED), ("mx", dict(q=ctypes.c_void_p(260)), ALIGN),
    ("mx", dict(s=None), NULL), ("mx", dict(M=0, x=None), OK)])
def test_norm_refusals(w, fmt, kw, status):
    assert _norm(w.lib, fmt, **kw) == status
    assert (w.lib.w8a8_last_error() == b"") == (status == OK)


def _int8(L, q=P, ldq=64, xs=P, M=4, K=64, wp=P, ws=P, N=8, bias=None, act=0, res=None, ldr=8, y=P, ldy=8, room=P, n=0):
    return L.w8a8_linear_fused(q, ldq, xs, M, K, wp, ws, N, bias, act, res, ldr, y, ldy, room, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(M=1 << 28), SHAPE), (dict(N=0), SHAPE), (dict(N=(1 << 22) + 1, ldy=1 << 23), SHAPE),
    (dict(K=0), SHAPE), (dict(ldq=63), SHAPE), (dict(ldy=7), SHAPE), (dict(res=P, ldr=7), SHAPE),
    (dict(act=1), UNSUPPORTED), (dict(act=6), UNSUPPORTED), (dict(act=-1), UNSUPPORTED), (dict(q=None), NULL),
    (dict(xs=None), NULL), (dict(wp=None), NULL), (dict(ws=None), NULL), (dict(y=None), NULL), (dict(wp=P8), ALIGN),
    (dict(xs=ODD), ALIGN), (dict(ws=ODD), ALIGN), (dict(bias=ODD), ALIGN), (dict(res=ODD), ALIGN), (dict(y=ODD), ALIGN),
    (dict(K=15, n=4 * 128 - 1), WORKSPACE), (dict(K=15, room=None, n=1 << 20), WORKSPACE),
    (dict(K=15, room=P8, n=1 << 20), WORKSPACE), (dict(M=0, q=None, xs=None, wp=None, ws=None, y=None), OK)])
def test_int8_refusals(w, kw, status):
    assert _int8(w.lib, **kw) == status


def _fp8(L, x=P, ldx=128, xs=P, M=4, K=64, wp=P, ws=P, N=8, bias=None, act=0, res=None, ldr=8, y=P, ldy=8, room=None,
         n=0):
    return L.w8a8_fp8b_linear_fused(x, ldx, xs, M, K, wp, ws, N, bias, act, res, ldr, y, ldy, 0, room, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(act=1), UNSUPPORTED), (dict(act=9), UNSUPPORTED), (dict(res=P, ldr=7), SHAPE), (dict(res=ODD), ALIGN),
    (dict(ldy=7), SHAPE), (dict(xs=None, ldx=64), WORKSPACE), (dict(x=None), NULL),
    (dict(M=0, x=None, xs=None, wp=None, ws=None, y=None), OK)])
def test_fp8_refusals(w, kw, status):
    assert _fp8(w.lib, **kw) == status


def _bf16(L, x=P, ldx=64, M=4, K=64, wp=P, N=8, bias=None, act=0, res=None, ldr=8, y=P, ldy=8, out=0, room=P, n=0):
    return L.w8a8_bf16_linear(x, ldx, M, K, wp, N, bias, act, res, ldr, y, ldy, out, room, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(ldx=63), SHAPE), (dict(ldy=7), SHAPE), (dict(res=P, ldr=7), SHAPE),
    (dict(act=1, ldy=3), SHAPE), (dict(act=1, N=7), SHAPE), (dict(act=7), UNSUPPORTED), (dict(out=1), UNSUPPORTED),
    (dict(out=4), UNSUPPORTED), (dict(x=None), NULL), (dict(wp=None), NULL), (dict(y=None), NULL), (dict(wp=P8), ALIGN),
    (dict(x=ODD), ALIGN), (dict(y=ODD), ALIGN), (dict(y=ctypes.c_void_p(258), out=2), ALIGN), (dict(bias=ODD), ALIGN),
    (dict(res=ODD), ALIGN), (dict(K=7, n=511), WORKSPACE), (dict(K=7, room=None, n=1 << 20), WORKSPACE),
    (dict(M=0, x=None, wp=None, y=None), OK)])
def test_bf16_refusals(w, kw, status):
    assert _bf16(w.lib, **kw) == status


def _grouped(L, x=P, ldx=64, rows=8, index=None, gl=P, R=8, E=4, N=16, K=64, wp=P, act=0, y=P, room=P, n=1 << 20):
    return L.w8a8_bf16_grouped_gemm(x, ldx, rows, index, gl, R, E, N, K, wp, act, y, room, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), UNSUPPORTED), (dict(K=7), UNSUPPORTED), (dict(K=0), SHAPE),
    (dict(R=1 << 28, rows=1 << 28), SHAPE), (dict(R=1 << 27, rows=1 << 27, N=1 << 14), UNSUPPORTED),
    (dict(ldx=63), SHAPE), (dict(act=1, N=15), SHAPE), (dict(act=8), UNSUPPORTED), (dict(rows=7), SHAPE),
    (dict(rows=0, index=P), SHAPE), (dict(x=None), NULL), (dict(gl=None), NULL), (dict(wp=None), NULL),
    (dict(y=None), NULL), (dict(gl=ctypes.c_void_p(260)), ALIGN), (dict(x=ODD), ALIGN), (dict(index=ODD), ALIGN),
    (dict(wp=P8), ALIGN), (dict(y=ODD), ALIGN), (dict(n=8), WORKSPACE), (dict(room=None), WORKSPACE),
    (dict(room=P8), WORKSPACE), (dict(R=0, x=None, gl=None), OK)])
def test_grouped_refusals(w, kw, status):
    assert _grouped(w.lib, **kw) == status


def test_prepack_refusals_and_sizes(w):
    L = w.lib
    assert L.w8a8_bf16_prepack_weight(P, 0, 16, 64, 0, P, None) == SHAPE
    assert L.w8a8_bf16_prepack_weight(P, 1, 15, 64, 1, P, None) == SHAPE       # [gate | up] of 15 rows
    assert L.w8a8_bf16_prepack_weight(P, 1, 16, 64, 9, P, None) == UNSUPPORTED
    assert L.w8a8_bf16_prepack_weight(None, 1, 16, 64, 0, P, None) == NULL
    assert L.w8a8_bf16_prepack_weight(P, 1, 16, 64, 0, P8, None) == ALIGN
    assert w.bf16_packed_bytes(1, 4096, 7168) == 4096 * 7168 * 2
    assert w.bf16_packed_bytes(3, 17, 65) == 3 * 32 * 128 * 2                    # N to 32, K to 64
    assert w._bf16_packed(3, 17, 65) == w.bf16_packed_bytes(3, 17, 65)
    assert w.linear_fused_workspace_bytes(3, 16, 200) == w.bf16_linear_workspace_bytes(3, 16, 200) == 0
    assert w.linear_fused_workspace_bytes(3, 16, 15) == w.bf16_linear_workspace_bytes(3, 16, 7) == 512  # rows copied
    assert w.bf16_linear_workspace_bytes(8192, 4096, 7169) >= 8192 * 2 * 7232
    assert w.bf16_linear_workspace_bytes(300, 300, 16000) >= 2 * 300 * 300 * 4  # sums of the parts of K
    assert w.bf16_linear_workspace_bytes(0, 16, 200) == 0
    assert w.bf16_grouped_workspace_bytes(0, 4, 16, 64) == 0


def test_binding_refusals_without_a_gpu(w):
    b = torch.zeros((4, 64), dtype=torch.bfloat16)
    u, q = torch.zeros((4096,), dtype=torch.uint8), torch.zeros((4, 64), dtype=torch.int8)
    for call in (lambda: w.rms_norm(b, None), lambda: w.rms_norm_quant(b, b[0]), lambda: w.fp8b_rms_norm_quant(b, None),
                 lambda: w.mx_rms_norm_quant(b, None), lambda: w.linear_fused(q, b[0], u, b[0], 8),
                 lambda: w.bf16_linear(b, u, 8), lambda: w.bf16_prepack_weight(b),
                 lambda: w.bf16_grouped_gemm(b, torch.zeros(2, dtype=torch.int64), u, 8)):
        with pytest.raises(ValueError):
            call()                                               # not on a GPU
    for call in (lambda: w.rms_norm(b.float(), None), lambda: w.linear_fused(b, b[0], u, b[0], 8),
                 lambda: w.bf16_linear(q, u, 8), lambda: w.bf16_prepack_weight(q)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not available")
@pytest.mark.parametrize("src", ["norm.hip", "fused.hip"])
def test_kernels_keep_out_of_scratch(src, tmp_path):
    out = tmp_path / "k.s"
    r = subprocess.run([_hipcc(), *_flags(), "-S", os.path.join(CSRC, src), "-o", str(out),
                        "-Rpass-analysis=kernel-resource-usage"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    names = re.findall(r"Function Name: (\S+)", r.stderr)
    scratch = [int(v) for v in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", r.stderr)]
    assert names and len(names) == len(scratch)
    assert not {n: s for n, s in zip(names, scratch) if s > MAX_SCRATCH}
    asm = out.read_text()
    for m in re.finditer(r"^(_Z\S+):\s*(?:;.*)?$", asm, re.M):
        if m.group(1) not in names:
            continue
        lines = asm[m.end():].split(".Lfunc_end")[0].split("\n")
        for a, b in _innermost_mfma_loops(lines):
            assert not any("scratch_" in x for x in lines[a:b + 1]), m.group(1)
