"""Block-scaled FP8 products, the expert router in front of them, and their plain forms.

Four operators, as a serving program calls them:

  gate    router logits -> the top-k experts of every token and their weights
  quant   BF16 rows, or silu(gate) * up of BF16 [gate | up] rows -> E4M3 codes with one
          fp32 scale per row and 128 columns
  linear  BF16 rows x E4M3 weight with one fp32 scale per 128 x 128 block -> BF16
  layer   gate, then the whole expert layer: the tokens quantized, the rows of
          every expert through W13 -> SwiGLU -> requant -> W2, weighted sum

Definitions (s: the fp32 scale of a block; code: rounding to E4M3, ties to even):
  quant   s = max|x| / 448 over the block; q = code(x / s), 0 where s = 0 (both quotients
          are fp32 numbers)
  linear  y = BF16(sum over blocks b of s_x[m, b] s_w[n / 128, b] sum_k q_x q_w + bias)
  gate    score = sigmoid(l) or softmax(l); key = score + bias; experts whose logit is
          -inf or NaN are out; of the groups the best by the sum of their two largest
          keys stay; the k largest keys win, lowest index first among equals; the
          weight is the score, over the sum of the k where asked, times a factor
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
DEV = "cuda:0"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 16 sequences: scores of 256 experts, 4 of 8 groups, top 8
        dict(name="gate step", op="gate", T=16, E=256, k=8, scoring="sigmoid", groups=8, keep=4, bias=True,
             dtype="float32", masked=0.0),
        # a batch of prompts through the same router
        dict(name="gate prompts", op="gate", T=16384, E=256, k=8, scoring="sigmoid", groups=8, keep=4, bias=True,
             dtype="float32", masked=0.0),
        # softmax scores of BF16 logits over an odd number of experts, some of them off for some tokens
        dict(name="gate softmax odd", op="gate", T=5003, E=99, k=6, scoring="softmax", groups=1, keep=1, bias=False,
             dtype="bfloat16", masked=0.1),
        # the activation of a long prefill
        dict(name="quant prompt", op="quant", M=8192, K=7168, act="none"),
        # the W13 output of 2048 tokens at top 8
        dict(name="quant swiglu", op="quant", M=16384, K=2048, act="swiglu"),
        # rows of a width that fills neither a block nor a 16-byte chunk
        dict(name="quant swiglu odd", op="quant", M=1237, K=1412, act="swiglu"),
        # one token through a projection: the weight's stream from memory
        dict(name="linear token", op="linear", M=1, N=4096, K=7168, bias=False),
        # a decode batch
        dict(name="linear batch", op="linear", M=64, N=4096, K=7168, bias=False),
        # a short ragged prompt through a narrow projection, partial blocks on every side
        dict(name="linear odd", op="linear", M=333, N=1000, K=2000, bias=True),
        # a long prefill
        dict(name="linear prompt", op="linear", M=8192, N=4096, K=7168, bias=True),
        # a decode step of 16 sequences through an expert layer: about 100 experts own a row
        dict(name="layer step", op="layer", T=16, E=256, k=8, H=4096, I=2048, groups=8, keep=4, skew=0.5),
        # 2048 prompt tokens through the same layer
        dict(name="layer prompt", op="layer", T=2048, E=256, k=8, H=4096, I=2048, groups=8, keep=4, skew=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "quant", "linear", "linear", "layer", "layer"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 4, 512 // groups)
        keep = rng.randint(1, groups)
        k = min(rng.randint(1, 16), keep * (E // groups))
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, scoring=rng.choice(["sigmoid", "softmax"]), groups=groups,
                    keep=keep, bias=rng.random() < 0.6, dtype=rng.choice(["float32", "bfloat16", "float16"]),
                    masked=rng.choice([0.0, 0.05]))
    if op == "quant":
        if rng.random() < 0.5:
            return dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 32, 7168), act="none")
        return dict(op=op, M=_log(rng, 1, 16384), K=_log(rng, 32, 2048), act="swiglu")
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 16, 4096), K=_log(rng, 64, 7168), bias=rng.random() < 0.5)
    groups = rng.choice([1, 2, 4])
    E = groups * rng.randint(2, 32)
    keep = rng.randint(1, groups)
    k = min(rng.randint(1, 8), keep * (E // groups))
    return dict(op=op, T=_log(rng, 1, 2048), E=E, k=k, H=_log(rng, 128, 4096), I=_log(rng, 64, 2048), groups=groups,
                keep=keep, skew=round(rng.uniform(0.0, 1.0), 3))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _blocks(n):
    return -(-n // BLOCK)


def _activations(g, M, K):
    """N(0, 1) with one value in 200 twenty times as large, as activations have."""
    x = torch.randn((M, K), generator=g, device=DEV)
    x = torch.where(torch.rand((M, K), generator=g, device=DEV) < 0.005, x * 20.0, x)
    return x.to(torch.bfloat16)


def _weight(g, E, N, K):
    """E4M3 codes uint8 [E, N, K] and scales float32 [E, ceil(N / 128), ceil(K / 128)]
    of weights of deviation about 1 / sqrt(K)."""
    w = torch.empty((E, N, K), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        part = torch.randn((min(step, E - e), N, K), generator=g, device=DEV).mul_(112.0).clamp_(-E4M3_MAX, E4M3_MAX)
        w[e:e + step] = part.to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.rand((E, _blocks(N), _blocks(K)), generator=g, device=DEV).mul_(0.6).add_(0.7)
    return w, s.mul_(1.0 / (112.0 * math.sqrt(K)))


def _router(g, T, E, dtype, bias, masked, skew):
    l = torch.randn((T, E), generator=g, device=DEV) + skew * torch.randn((E,), generator=g, device=DEV)
    if masked:
        l = torch.where(torch.rand((T, E), generator=g, device=DEV) < masked, -math.inf, l)
    b = 0.05 * torch.randn((E,), generator=g, device=DEV) if bias else None
    return l.to(getattr(torch, dtype)), b


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c, op = dict(case), case["op"]
    if op == "gate":
        c["logits"], c["b"] = _router(g, c["T"], c["E"], c["dtype"], c["bias"], c["masked"], 0.5)
    elif op == "quant":
        c["x"] = _activations(g, c["M"], c["K"] * (2 if c["act"] == "swiglu" else 1))
    elif op == "linear":
        c["x"] = _activations(g, c["M"], c["K"])
        w, s = _weight(g, 1, c["N"], c["K"])
        c["w"], c["ws"] = w[0], s[0]
        c["b"] = torch.randn((c["N"],), generator=g, device=DEV).mul_(0.1).to(torch.bfloat16) if c["bias"] else None
    else:
        c["x"] = _activations(g, c["T"], c["H"])
        c["logits"], c["b"] = _router(g, c["T"], c["E"], "float32", True, 0.0, c["skew"])
        c["w13"], c["s13"] = _weight(g, c["E"], 2 * c["I"], c["H"])
        c["w2"], c["s2"] = _weight(g, c["E"], c["H"], c["I"])
    if own:
        # what a serving program keeps: the weights laid out once at load time,
        # outputs and workspaces
        import moe_token_amax_amd as W
        c["W"] = W

        def room(n):
            return torch.empty((max(n, 1),), dtype=torch.uint8, device=DEV)

        if op in ("gate", "layer"):
            c["ids"] = torch.empty((c["T"], c["k"]), dtype=torch.int32, device=DEV)
            c["weights"] = torch.empty((c["T"], c["k"]), dtype=torch.float32, device=DEV)
            c["scoring"] = {"sigmoid": W.GATE_SIGMOID, "softmax": W.GATE_SOFTMAX}[c.get("scoring", "sigmoid")]
        if op == "quant":
            c["kind"] = {"none": W.ACT_NONE, "swiglu": W.ACT_SWIGLU}[c["act"]]
            c["q"] = torch.empty((c["M"], BLOCK * _blocks(c["K"])), dtype=torch.uint8, device=DEV)
            c["scale"] = torch.empty((_blocks(c["K"]), c["M"]), dtype=torch.float32, device=DEV)
        if op == "linear":
            c["w"] = W.fp8b_prepack_weight(c["w"])
            c["y"] = torch.empty((c["M"], c["N"]), dtype=torch.bfloat16, device=DEV)
            c["work"] = room(W.fp8b_linear_workspace_bytes(c["M"], c["N"], c["K"]))
        if op == "layer":
            c["w13"], c["w2"] = W.fp8b_prepack_weight(c["w13"]), W.fp8b_prepack_weight(c["w2"])
            c["out"] = torch.empty((c["T"], c["H"]), dtype=torch.bfloat16, device=DEV)
            c["work"] = room(W.fp8b_moe_layer_workspace_bytes(c["T"], c["k"], c["E"], c["H"], c["I"]))
    return c


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _pad(t, dim, to):
    n = t.shape[dim]
    if n == to:
        return t
    shape = list(t.shape)
    shape[dim] = to - n
    return torch.cat([t, t.new_zeros(shape)], dim)


def _plain_quant(v):
    """float32 [M, K] -> E4M3 codes [M, 128 B], scales float32 [B, M], B blocks."""
    M, B = v.shape[0], _blocks(v.shape[1])
    v = _pad(v, 1, B * BLOCK).view(M, B, BLOCK)
    s = (v.abs().amax(2).double() / E4M3_MAX).float()  # torch multiplies fp32 by a rounded 1 / 448
    q = torch.where(s[..., None] > 0, v / s[..., None], 0.0).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn).view(M, B * BLOCK), s.t().contiguous()


def _plain_values(q, s):
    return (q.float().view(q.shape[0], -1, BLOCK) * s.t()[..., None]).view(q.shape[0], -1)


def _plain_weight(w, s):
    """float32 [E, N, 128 B]: codes uint8 [E, N, K] times their blocks' scales."""
    E, N, K = w.shape
    v = _pad(_pad(w.view(torch.float8_e4m3fn).float(), 2, _blocks(K) * BLOCK), 1, _blocks(N) * BLOCK)
    v.view(E, _blocks(N), BLOCK, _blocks(K), BLOCK).mul_(s[:, :, None, :, None])
    return v[:, :N]


def _plain_silu(h):
    gate, up = h.float().chunk(2, 1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_gate(logits, b, c):
    """In 64 bits: which of two close keys is larger decides the expert."""
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = logits.double().clamp(max=torch.finfo(torch.float32).max)
    inside = ~(l.isnan() | (l == -math.inf))
    low = torch.where(inside, l, -math.inf)
    if c.get("scoring", "sigmoid") == "sigmoid":
        score = torch.where(inside, 1.0 / (1.0 + torch.exp(-l)), 0.0)
    else:
        top = low.amax(1, keepdim=True)
        e = torch.where(inside, torch.exp(low - torch.where(top == -math.inf, 0.0, top)), 0.0)
        total = e.sum(1, keepdim=True)
        score = e / torch.where(total > 0, total, 1.0)
    key = torch.where(inside, score if b is None else score + b.double(), -math.inf)
    if G > 1:
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True)[0]
        first = best[..., 0]
        second = best[..., 1] if E // G > 1 else torch.full_like(first, -math.inf)
        order = torch.sort(torch.where(second == -math.inf, first, first + second), dim=1, descending=True, stable=True)[1]
        stays = torch.zeros((T, G), dtype=torch.bool, device=key.device).scatter(1, order[:, :c["keep"]], True)
        key = torch.where(stays.repeat_interleave(E // G, 1), key, -math.inf)
    value, ids = torch.sort(key, dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    w = torch.where(value > -math.inf, score.gather(1, ids), 0.0)
    total = w.sum(1, keepdim=True)
    w = 2.5 * w / torch.where(total > 0, total, 1.0)
    return torch.where(value > -math.inf, ids, -1).to(torch.int32), w.float()


def _plain_linear(x, w, s, b):
    y = _plain_values(*_plain_quant(x.float())) @ _plain_weight(w[None], s[None])[0].t()
    return (y if b is None else y + b.float()).to(torch.bfloat16)


def _plain_layer(c):
    ids, weights = _plain_gate(c["logits"], c["b"], c)
    T, k, E = c["T"], c["k"], c["E"]
    expert = torch.where(ids < 0, E, ids).flatten().long()
    order = torch.sort(expert, stable=True)[1]
    e = expert[order]
    counts = (e[:, None] == torch.arange(E + 1, device=e.device)).sum(0)
    place = torch.arange(T * k, device=e.device) - (counts.cumsum(0) - counts)[e]
    most = int(counts.max())  # rows of the busiest expert: every expert gets as many

    def experts(rows, w, s):
        batch = rows.new_zeros((E + 1, most, rows.shape[1]))
        batch[e, place] = rows
        y = torch.bmm(_plain_weight(w, s), batch[:E].transpose(1, 2).contiguous())
        return y.transpose(1, 2)[e.clamp(max=E - 1), place].to(torch.bfloat16)

    x = _plain_values(*_plain_quant(c["x"].float()))
    h = experts(x[order // k], c["w13"], c["s13"])
    y = experts(_plain_values(*_plain_quant(_plain_silu(h))), c["w2"], c["s2"]).float()
    pairs = torch.empty_like(y)
    pairs[order] = torch.where(e[:, None] < E, y, 0.0)
    out = (weights[..., None] * pairs.view(T, k, -1)).sum(1)
    return ids, weights, out.to(torch.bfloat16)


def run(state):
    c, op = state, state["op"]
    if not own:
        if op == "gate":
            return _plain_gate(c["logits"], c["b"], c)
        if op == "quant":
            return _plain_quant(c["x"].float() if c["act"] == "none" else _plain_silu(c["x"]))
        if op == "linear":
            return _plain_linear(c["x"], c["w"], c["ws"], c["b"])
        return _plain_layer(c)
    W = c["W"]
    if op in ("gate", "layer"):
        W.moe_gate(c["logits"], c["k"], bias=c["b"], scoring=c["scoring"], n_group=c["groups"], topk_group=c["keep"],
                   renormalize=True, scale=2.5, ids=c["ids"], weights=c["weights"])
        if op == "gate":
            return c["ids"], c["weights"]
        W.fp8b_moe_layer(c["x"], c["ids"], c["weights"], c["w13"], c["s13"], c["w2"], c["s2"], c["I"], out=c["out"],
                         workspace=c["work"])
        return c["ids"], c["weights"], c["out"]
    if op == "quant":
        q, s = W.fp8b_quant(c["x"], act=c["kind"], q=c["q"], scale=c["scale"])
        return q.view(torch.float8_e4m3fn), s
    return W.fp8b_linear(c["x"], c["w"], c["ws"], c["N"], bias=c["b"], y=c["y"], workspace=c["work"])


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    if op == "gate":
        size = 4 if c["dtype"] == "float32" else 2
        # a score, a comparison with the bias added: about ten operations a logit
        return {"bytes": c["T"] * c["E"] * size + 8 * c["T"] * c["k"] + (4 * c["E"] if c["bias"] else 0),
                "flops": 10 * c["T"] * c["E"]}
    if op == "quant":
        M, K, n = c["M"], c["K"], 2 if c["act"] == "swiglu" else 1
        return {"bytes": 2 * n * M * K + M * BLOCK * _blocks(K) + 4 * M * _blocks(K), "flops": (3 + 5 * (n - 1)) * M * K}
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": 2 * M * K + N * K + 4 * _blocks(N) * _blocks(K) + 2 * M * N, "flops": 2 * M * N * K}
    T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
    hit = E * (1.0 - (1.0 - k / E) ** T)  # experts that own a row, were they equally likely
    weights = hit * (3 * H * I + 4 * (_blocks(2 * I) * _blocks(H) + _blocks(H) * _blocks(I)))
    return {"bytes": weights + 4 * T * H + 4 * T * E + 8 * T * k, "flops": 6 * T * k * H * I}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _code64(v):
    """The nearest E4M3 value, ties to the even code: 3 bits below the leading one,
    steps of 2^-9 under 2^-6."""
    a = v.abs().clamp(max=E4M3_MAX)
    step = torch.ldexp(torch.ones_like(a), torch.frexp(a.clamp(min=2.0 ** -6))[1] - 4)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _blocks64(v):
    """(x / s, s) of float64 [M, K], the scale and the quotient as the fp32 numbers that
    the codes are defined by: BF16 values and a BF16 maximum often meet a tie exactly."""
    M, K = v.shape
    full = torch.zeros((M, _blocks(K), BLOCK), dtype=torch.float64, device=v.device)
    full.view(M, -1)[:, :K] = v
    s = (full.abs().max(2)[0] / E4M3_MAX).float().double()
    t = torch.where(s[..., None] > 0, full / s.clamp(min=1e-300)[..., None], 0.0)
    return t.float().double(), s


def _product64(v, codes, s):
    """float64 [M, K] quantized, times one weight [N, K]."""
    N, K = codes.shape
    t, sx = _blocks64(v)
    a = (_code64(t) * sx[..., None]).view(v.shape[0], -1)[:, :K]
    rows = torch.arange(N, device=s.device) // BLOCK
    cols = torch.arange(K, device=s.device) // BLOCK
    w = codes.view(torch.float8_e4m3fn).double() * s.double()[rows][:, cols]
    return a @ w.t()


def _gate64(logits, b, c):
    l = logits.double()
    on = l > -math.inf
    p = torch.sigmoid(l) if c.get("scoring", "sigmoid") == "sigmoid" else torch.softmax(l, 1)
    key = p + (0.0 if b is None else b.double())
    key = key.masked_fill(~on, -math.inf)
    if c["groups"] > 1:
        split = key.unflatten(1, (c["groups"], -1))
        two = split.topk(min(2, split.shape[2]), 2)[0]
        mark = two.masked_fill(two == -math.inf, 0.0).sum(2).masked_fill(two[..., 0] == -math.inf, -math.inf)
        chosen = torch.zeros_like(mark).scatter_(1, mark.topk(c["keep"], 1)[1], 1.0)
        key = split.masked_fill(chosen[..., None] == 0, -math.inf).flatten(1)
    value, ids = key.topk(c["k"], 1)
    w = p.gather(1, ids).masked_fill(value == -math.inf, 0.0)
    return ids.masked_fill(value == -math.inf, -1), 2.5 * w / w.sum(1, keepdim=True).clamp(min=1e-300)


def _silu64(h):
    h = h.double()
    n = h.shape[1] // 2
    return h[:, :n] * torch.sigmoid(h[:, :n]) * h[:, n:]


def exact(case, seed):
    global own
    before, own = own, False
    try:
        c = prepare(case, seed)
    finally:
        own = before
    op = c["op"]
    if op == "gate":
        return None, _gate64(c["logits"], c["b"], c)[1]
    if op == "quant":
        t, s = _blocks64(c["x"].double() if c["act"] == "none" else _silu64(c["x"]))
        return _code64(t).view(c["M"], -1), s.t().contiguous()
    if op == "linear":
        y = _product64(c["x"].double(), c["w"], c["ws"])
        return y if c["b"] is None else y + c["b"].double()
    ids, weights = _gate64(c["logits"], c["b"], c)
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        t, j = torch.where(ids == e)
        if len(t):
            h = _product64(c["x"][t].double(), c["w13"][e], c["s13"][e]).to(torch.bfloat16)
            y = _product64(_silu64(h), c["w2"][e], c["s2"][e]).to(torch.bfloat16)
            out.index_add_(0, t, weights[t, j][:, None] * y)
    return None, weights, out
