"""NumPy oracle of the block-scaled FP8 path and of the expert router. TEST
INFRASTRUCTURE ONLY: only ``tests/`` may import it. It shares no code or tables
with the HIP library.

Sources: "Qwen3.8-FP8 on Ascend 950: Why Weights Become MXFP8 at Load Time",
Deep Dive 1 (E4M3 weights with one fp32 scale per 128 x 128 tile); the quantizer
of the activations, the sum over blocks and the router are this library's own
definitions (parity unpinned beyond them).

  quant    per row and 128 columns: s = fl32(amax / 448), code = E4M3(fl32(v / s)),
           half to even, saturating, NaN of NaN; zeros for s = 0 and s NaN.
           scale_alg 1: a finite s rounded up to a power of two, at least 2^-126.
  product  float64: sum over blocks of s_x s_w times the exact sum of code products.
  gate     see ``gate``; everything in float64.

The matrix unit adds the products of 8 consecutive k after cutting each towards
zero to a multiple of 2^(E - 13), E the largest sum of the two codes' exponents in
the group (subnormal codes have exponent -6). ``cut_bound`` is the resulting bound
of every output, used by the tests' tolerance.
"""

from __future__ import annotations

import numpy as np

from .mx_ref import e4m3_decode, e4m3_encode
from .w8a8_ref import bf16_to_f32, swiglu

__all__ = ["BLOCK", "blocks", "quant", "quant_f32", "dequant", "weight_dequant", "product64", "cut_bound", "gate"]

BLOCK = 128


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def quant(x_bits, act: int = 0, scale_alg: int = 0):
    """BF16 bits [M, K] (or [M, 2K] with act 1) -> codes [M, 128 B], scales [B, M]."""
    if act:
        v = swiglu(x_bits, x_bits.shape[1] // 2)
    else:
        v = bf16_to_f32(x_bits)
    return quant_f32(v, scale_alg)


def quant_f32(v, scale_alg: int = 0):
    """float32 [M, K] -> codes [M, 128 B], scales [B, M]."""
    v = np.asarray(v, np.float32)
    M, K = v.shape
    B = blocks(K)
    full = np.zeros((M, B * BLOCK), np.float32)
    full[:, :K] = v
    full = full.reshape(M, B, BLOCK)
    s = (np.abs(full).max(2) / np.float32(448.0)).astype(np.float32)
    if scale_alg == 1:
        m, e = np.frexp(s.astype(np.float64))            # s = m 2^e, m in [0.5, 1)
        e = np.where(m == 0.5, e - 1, e)
        up = np.where(s > 0, np.ldexp(1.0, np.maximum(e, -126)), 0.0).astype(np.float32)
        s = np.where(np.isfinite(s), up, s)
    with np.errstate(divide="ignore", invalid="ignore"):
        t = (full / s[..., None]).astype(np.float32)
    t = np.where(s[..., None] > 0, t, np.float32(0.0))
    codes = np.where(np.isnan(t), np.uint8(0x7F), e4m3_encode(t))   # an infinity over its infinite scale
    return codes.reshape(M, B * BLOCK), np.ascontiguousarray(s.T)


def dequant(q, s):
    """codes [M, 128 B], scales [B, M] -> float64 [M, 128 B]."""
    M = q.shape[0]
    return (e4m3_decode(q).reshape(M, -1, BLOCK) * s.T.astype(np.float64)[..., None]).reshape(M, -1)


def weight_dequant(w, s):
    """codes [N, K], scales [ceil(N/128), ceil(K/128)] -> float64 [N, 128 B]."""
    N, K = w.shape
    v = np.zeros((N, blocks(K) * BLOCK))
    v[:, :K] = e4m3_decode(w)
    r = np.arange(N) // BLOCK
    c = np.arange(v.shape[1]) // BLOCK
    return v * s.astype(np.float64)[r][:, c]


def product64(q, sx, w, sw, bias_bits=None):
    y = dequant(q, sx) @ weight_dequant(w, sw).T
    return y if bias_bits is None else y + bf16_to_f32(bias_bits).astype(np.float64)


def _exponent(codes):
    """floor(log2) of the code's value, -6 for subnormals; a zero takes no part (-99)."""
    c = np.asarray(codes, np.int64)
    e = np.maximum((c >> 3) & 15, 1) - 7
    return np.where((c & 0x7F) == 0, -99, e)


def cut_bound(q, sx, w, sw):
    """Bound of |product - product64| from the cuts alone, float64 [M, N]: at most 7 of 8
    products of a group lose less than 2^(E - 13) each."""
    M, N = q.shape[0], w.shape[0]
    Kp = q.shape[1]
    wp = np.zeros((N, Kp), np.uint8)
    wp[:, :w.shape[1]] = w
    ex = _exponent(q).reshape(M, Kp // 8, 8)
    ew = _exponent(wp).reshape(N, Kp // 8, 8)
    out = np.zeros((M, N))
    rows = np.arange(N) // BLOCK
    for g in range(Kp // 8):
        top = (ex[:, None, g] + ew[None, :, g]).max(2).astype(np.float64)
        b = g * 8 // BLOCK
        cut = np.where(top > -50, 7.0 * 2.0 ** (top - 13.0), 0.0)
        out += cut * np.abs(sx[b].astype(np.float64))[:, None] * np.abs(sw[rows, b].astype(np.float64))[None]
    return out


def gate(logits, top_k, bias=None, scoring="softmax", n_group=1, topk_group=1, renormalize=True, scale=1.0):
    """float64 restatement, token by token: (ids int32 [T, k], weights float64 [T, k])."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    ids = np.full((T, top_k), -1, np.int32)
    wts = np.zeros((T, top_k))
    big = float(np.finfo(np.float32).max)
    for t in range(T):
        v = np.minimum(l[t], big)
        ok = ~np.isnan(v) & (v > -np.inf)
        s = np.zeros(E)
        if scoring == "sigmoid":
            with np.errstate(over="ignore"):
                s[ok] = 1.0 / (1.0 + np.exp(-v[ok]))
        elif ok.any():
            s[ok] = np.exp(v[ok] - v[ok].max())
            s /= s.sum()
        key = s + (0.0 if bias is None else np.asarray(bias, np.float64))
        key = np.where(ok & ~np.isnan(key), key, -np.inf)
        if n_group > 1:
            per = E // n_group
            marks = []
            for g in range(n_group):
                two = sorted((x for x in key[g * per:(g + 1) * per] if x > -np.inf), reverse=True)[:2]
                marks.append(sum(two) if two else -np.inf)
            best = sorted(range(n_group), key=lambda g: (-marks[g], g))[:topk_group]
            for g in range(n_group):
                if g not in best:
                    key[g * per:(g + 1) * per] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -np.inf][:top_k]
        ids[t, :len(order)] = order
        w = s[order]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else 0.0 * w
        wts[t, :len(order)] = w * scale
    return ids, wts
