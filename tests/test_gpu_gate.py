"""The expert router through the C ABI against the float64 oracle.

Ids are compared exactly. Weights: a softmax that is not renormalized divides by a
sum of up to 1024 float32 exponentials and is held to 2^-20 relative; every other
weight to 2^-23 (one rounding to float32 and one of the factor).
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from tests.conftest import gpu_available
from tests.gpu_util import DEV, dev, host, show, sync

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def w():
    import moe_token_amax_amd as w
    return w


def _check(w, l, k, bias=None, scoring="sigmoid", G=1, keep=1, renorm=True, scale=1.0, ids=None, wts=None):
    """l: CPU tensor of logits in the type under test"""
    show(f"gate {tuple(l.shape)} {l.dtype} k={k} {scoring} groups={G}/{keep} bias={bias is not None}")
    b = None if bias is None else dev(bias.astype(np.float32))
    got_i, got_w = w.moe_gate(l.to(DEV), k, bias=b, scoring=w.GATE_SIGMOID if scoring == "sigmoid" else w.GATE_SOFTMAX,
                              n_group=G, topk_group=keep, renormalize=renorm, scale=scale, ids=ids, weights=wts)
    sync()
    want_i, want_w = O.fp8b.gate(l.double().numpy(), k, None if bias is None else bias.astype(np.float32), scoring, G,
                                 keep, renorm, np.float64(np.float32(scale)))
    gi = host(got_i)
    bad = np.argwhere(gi != want_i)
    assert bad.size == 0, (bad[:4].tolist(), gi[bad[0][0]], want_i[bad[0][0]])
    tol = 2.0 ** (-20 if scoring == "softmax" and not renorm else -23)
    off = np.abs(host(got_w).astype(np.float64) - want_w)
    assert (off <= tol * np.abs(want_w) + 1e-38).all(), float((off / np.maximum(np.abs(want_w), 1e-38)).max())


def _logits(T, E, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn((T, E), generator=g)).to(dtype)


CASES = [  # T, E, k, scoring, groups, keep, dtype
    (1, 1, 1, "softmax", 1, 1, torch.float32), (3, 8, 2, "softmax", 1, 1, torch.bfloat16),
    (5, 60, 4, "softmax", 1, 1, torch.float16), (7, 64, 6, "sigmoid", 1, 1, torch.bfloat16),
    (16, 256, 8, "sigmoid", 8, 4, torch.float32), (65, 256, 8, "sigmoid", 8, 4, torch.bfloat16),
    (33, 160, 6, "softmax", 8, 3, torch.float32), (9, 99, 5, "sigmoid", 3, 2, torch.float32),
    (130, 384, 8, "sigmoid", 1, 1, torch.float32), (17, 513, 16, "softmax", 1, 1, torch.float32),
    (4, 1024, 64, "sigmoid", 64, 40, torch.float32), (6, 1000, 9, "softmax", 5, 2, torch.float16),
    (11, 64, 3, "sigmoid", 64, 7, torch.float32), (2, 12, 12, "sigmoid", 4, 4, torch.float32),
    (257, 128, 8, "sigmoid", 4, 1, torch.bfloat16), (70, 32, 32, "softmax", 2, 2, torch.bfloat16),
]


@pytest.mark.parametrize("renorm,scale", [(True, 2.5), (False, 1.0)])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,scoring,G,keep,dtype", CASES)
def test_gate(w, T, E, k, scoring, G, keep, dtype, with_bias, renorm, scale):
    bias = 0.1 * np.random.default_rng(E).standard_normal(E) if with_bias else None
    _check(w, _logits(T, E, dtype, 7 * T + E), k, bias, scoring, G, keep, renorm, scale)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,keep", [(1, 1), (4, 2), (16, 3)])
def test_gate_ties_go_to_the_lowest_index(w, scoring, G, keep):
    # three distinct logits over 64 experts: nearly every comparison is a tie
    l = torch.from_numpy(np.random.default_rng(5).integers(0, 3, (40, 64)).astype(np.float32))
    _check(w, l, 8, None, scoring, G, keep)
    _check(w, l.to(torch.bfloat16), 8, np.zeros(64), scoring, G, keep)
    _check(w, torch.zeros((3, 64)), 8, np.repeat([0.5, 0.25], 32), scoring, G, keep)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,keep", [(1, 1), (4, 2)])
@pytest.mark.parametrize("E", [32, 256])
def test_gate_masks_and_specials(w, scoring, G, keep, E):
    rng = np.random.default_rng(E)
    l = rng.standard_normal((24, E)).astype(np.float32)
    l[0] = -np.inf                       # nothing left
    l[1, 1:] = -np.inf                   # one expert
    l[2] = np.nan
    l[3, ::2] = np.nan
    l[4, 3] = np.inf
    l[5] = np.inf
    l[6] = np.finfo(np.float32).min
    l[7, : E // 2] = -np.inf             # half of the groups have no expert
    l[8] = 1e30
    l[9, 5] = -1e30
    l[10] *= 200.0                       # sigmoids at 0 and 1
    l[11, : E - 3] = -np.inf             # fewer experts than slots
    b = 0.1 * rng.standard_normal(E)
    b[7], b[9] = -np.inf, np.inf         # an expert switched off, one forced
    for bias in (None, b):
        for renorm in (True, False):
            _check(w, torch.from_numpy(l), 5, bias, scoring, G, keep, renorm)


def _nudge(x, n):
    """x moved by n float32 steps"""
    return (x.view(np.int32) + np.asarray(n, np.int32)).view(np.float32)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,keep", [(1, 1), (8, 3)])
def test_gate_close_keys(w, scoring, G, keep):
    """Logits a few float32 steps apart: the scores differ by less than a float32 step."""
    rng = np.random.default_rng(11)
    base = rng.uniform(2.0, 6.0, (64, 1)).astype(np.float32)
    l = _nudge(np.repeat(base, 128, 1), rng.integers(-3, 4, (64, 128)))
    _check(w, torch.from_numpy(l), 8, None, scoring, G, keep)
    # keys close through the bias: score + bias of two experts meet within 1e-9
    l2 = rng.uniform(-1.0, 1.0, (64, 128)).astype(np.float32)
    b = np.zeros(128)
    l2[:, 64:] = l2[:, :64]
    b[64:] = 2.0 ** -31 * rng.integers(-2, 3, 64)
    _check(w, torch.from_numpy(l2), 8, b, scoring, G, keep)


MANY = [  # T, E, k, scoring, groups, keep, dtype, bias: four tokens a wavefront
    (5121, 256, 8, "sigmoid", 8, 4, torch.float32, True), (5126, 256, 8, "sigmoid", 8, 4, torch.bfloat16, True),
    (5120, 64, 6, "softmax", 1, 1, torch.bfloat16, False), (5123, 160, 6, "softmax", 10, 3, torch.float32, False),
    (5197, 99, 6, "softmax", 1, 1, torch.bfloat16, False), (5122, 128, 15, "sigmoid", 4, 2, torch.float16, True),
    (5195, 256, 16, "softmax", 16, 5, torch.float32, False), (5136, 32, 4, "sigmoid", 8, 3, torch.float32, False),
    (5129, 17, 5, "softmax", 1, 1, torch.float32, True), (5125, 256, 8, "sigmoid", 2, 1, torch.float32, False),
    (5121, 3, 2, "sigmoid", 1, 1, torch.float32, True),
]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,scoring,G,keep,dtype,with_bias", MANY)
def test_gate_four_tokens_a_wavefront(w, T, E, k, scoring, G, keep, dtype, with_bias, renorm):
    """Random tokens, and among them ties, masks, specials and keys that are too close
    for floats, so that a wavefront holds tokens of every kind."""
    rng = np.random.default_rng(T)
    l = rng.standard_normal((T, E)).astype(np.float32)
    b = 0.1 * rng.standard_normal(E).astype(np.float32)
    l[0::7] = rng.integers(0, 3, l[0::7].shape)                      # ties
    l[1::9] = np.where(rng.random(l[1::9].shape) < 0.5, -np.inf, l[1::9])
    l[2::11] = -np.inf
    l[3::13, 0] = np.nan
    l[4::17] = _nudge(np.full_like(l[4::17], 2.5), rng.integers(-3, 4, l[4::17].shape))
    l[5::19] *= 300.0
    l[6::23, -1] = np.inf
    if E > 1:
        b[1] = -np.inf
    _check(w, torch.from_numpy(l).to(dtype), k, b if with_bias else None, scoring, G, keep, renorm, 1.5)


@pytest.mark.parametrize("T", [64, 5200])
@pytest.mark.parametrize("k", [1, 2, 8, 13, 14, 20])
def test_gate_pairs_in_float_order_and_double_order_differ(w, T, k):
    """Keys that agree in about 22 bits: pairs that floats put in the wrong order, at every
    place of the list and across its end, singly and in chains."""
    rng = np.random.default_rng(k)
    E = 64
    l = rng.uniform(-2.0, 2.0, (T, E))
    b = rng.uniform(-0.2, 0.2, E)
    # bias of expert e + 32 such that its key is within some 2^-24 of expert e's in token 0's logits
    s = 1 / (1 + np.exp(-l.astype(np.float32).astype(np.float64)))
    for t in range(T):
        n = rng.integers(1, 4)
        top = np.argsort(-(s[t] + b))[rng.integers(0, min(k + 2, 12))]
        for j in range(n):
            e = (top + 7 * (j + 1)) % E
            want = s[t, top] + b[top] - b[e] + rng.integers(-8, 9) * 2.0 ** -26
            if 0.01 < want < 0.99:
                l[t, e] = np.log(want / (1 - want))
    _check(w, torch.from_numpy(l.astype(np.float32)), k, b, "sigmoid", 1, 1, True, 1.0)


@pytest.mark.parametrize("T", [64, 5200])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("k", [1, 2, 5, 8, 14, 17])
def test_gate_equal_pairs_next_to_a_closer_one(w, T, scoring, k):
    """Two experts of one logit and bias at the end of the list, and a third, of another
    logit and bias, within some 2^-24 of both: on either side of them in doubles."""
    rng = np.random.default_rng(100 + k)
    E, h = 64, 16
    l = rng.uniform(-2.0, 2.0, (T, E))
    b = rng.uniform(-0.2, 0.2, E)
    l[:, h:2 * h], b[h:2 * h] = l[:, :h], b[:h]
    if scoring == "sigmoid":
        s = 1 / (1 + np.exp(-l[:, :h].astype(np.float32).astype(np.float64)))
        want = np.clip(s + b[:h] - b[2 * h:3 * h] + rng.integers(-6, 7, (T, h)) * 2.0 ** -26, 0.01, 0.99)
        l[:, 2 * h:3 * h] = np.log(want / (1 - want))
    l[:, 3 * h:] = -9.0
    _check(w, torch.from_numpy(l.astype(np.float32)), k, b, scoring, 1, 1, True, 1.0)


@pytest.mark.parametrize("T", [64, 5200])
@pytest.mark.parametrize("E,G,keep,third", [(256, 8, 4, False), (256, 8, 4, True), (128, 16, 1, False), (64, 2, 1, False),
                                            (96, 3, 2, False), (256, 4, 3, True)])
def test_gate_groups_whose_marks_nearly_tie(w, T, E, G, keep, third):
    """The last group that stays and the first that goes (and one more) have marks that agree
    in some 24 bits, from other logits and biases."""
    rng = np.random.default_rng(E + G + T)
    per = E // G
    l = rng.uniform(-2.0, 2.0, (T, E))
    b = rng.uniform(-0.1, 0.1, E)
    s = 1 / (1 + np.exp(-l.astype(np.float32).astype(np.float64)))
    key = (s + b).reshape(T, G, per)
    top = np.argsort(-key, axis=2)[:, :, :2]
    order = np.argsort(-np.take_along_axis(key, top, 2).sum(2), axis=1)
    t = np.arange(T)
    a = order[:, keep - 1]
    for o in [keep] + ([keep + 1] if third and keep + 1 < G else []):
        c = order[:, o]
        for j in range(2):
            e_a, e_c = a * per + top[t, a, j], c * per + top[t, c, j]
            want = s[t, e_a] + b[e_a] - b[e_c] + rng.integers(-6, 7, T) * 2.0 ** -26
            l[t, e_c] = np.log(np.clip(want, 0.01, 0.99) / (1 - np.clip(want, 0.01, 0.99)))
    _check(w, torch.from_numpy(l.astype(np.float32)), 6, b, "sigmoid", G, keep, True, 1.0)


def test_gate_many_tokens(w):
    # more tokens than one pass of the chip; every token exact against the oracle on a sample
    T, E, k = 9001, 256, 8
    l = _logits(T, E, torch.float32, 3)
    b = 0.05 * np.random.default_rng(0).standard_normal(E).astype(np.float32)
    ids, wts = w.moe_gate(l.to(DEV), k, bias=dev(b), scoring=w.GATE_SIGMOID, n_group=8, topk_group=4, scale=2.5)
    sync()
    pick = np.r_[0:40, 4480:4520, T - 41:T]
    want, ww = O.fp8b.gate(l.double().numpy()[pick], k, b, "sigmoid", 8, 4, True, 2.5)
    assert np.array_equal(host(ids)[pick], want)
    assert np.abs(host(wts)[pick] - ww).max() <= 2.0 ** -23 * 2.5


def test_gate_strided_rows_and_given_outputs(w):
    wide = _logits(21, 300, torch.bfloat16, 1).to(DEV)
    view = wide[:, 3:131]                 # rows of 128 inside 300, not 16-byte aligned
    ids = torch.full((21, 4), 77, dtype=torch.int32, device=DEV)
    wts = torch.full((21, 4), 9.0, device=DEV)
    w.moe_gate(view, 4, scoring=w.GATE_SIGMOID, n_group=4, topk_group=2, ids=ids, weights=wts)
    sync()
    want, ww = O.fp8b.gate(view.double().cpu().numpy(), 4, None, "sigmoid", 4, 2)
    assert np.array_equal(host(ids), want) and np.abs(host(wts) - ww).max() <= 2.0 ** -23
    i, x = w.moe_gate(torch.empty((0, 64), device=DEV), 4)
    assert i.shape == (0, 4) and x.shape == (0, 4)


def test_gate_on_another_stream(w):
    l = _logits(300, 256, torch.float32, 2).to(DEV)
    a = w.moe_gate(l, 8, scoring=w.GATE_SIGMOID, n_group=8, topk_group=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = w.moe_gate(l, 8, scoring=w.GATE_SIGMOID, n_group=8, topk_group=4)
    sync()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------ logits that doubles cannot tell apart
TINY = np.array([0.0, -0.0, 1e-17, -1e-17, 2e-17, 3e-18, -5e-20, 1e-30, 1.4e-45])  # 1 + exp(-x) = 2 for each


@pytest.mark.parametrize("T", [64, 5200])
@pytest.mark.parametrize("G,keep", [(1, 1), (4, 2), (4, 4)])
@pytest.mark.parametrize("k", [1, 2, 8, 16])
def test_gate_distinct_logits_of_equal_sigmoids(w, T, k, G, keep):
    """Without a bias the order of keys is that of the logits only as far as doubles tell
    their sigmoids apart: past 23 or so, and next to 0, distinct logits have equal scores,
    which go to the lower index, inside the list and across its end."""
    rng = np.random.default_rng(1000 * k + G + keep)
    E = 64
    l = rng.standard_normal((T, E)).astype(np.float32)
    for r in range(T):
        n = int(rng.integers(1, E + 1))
        at = rng.permutation(E)[:n]
        kind = r % 6
        if kind == 0:                                    # anywhere in the range where they start to meet
            l[r, at] = rng.uniform(18.0, 38.0, n)
        elif kind == 1:                                  # neighbours of one value
            l[r, at] = _nudge(np.full(n, rng.uniform(19.0, 37.0), np.float32), rng.integers(-4, 5, n))
        elif kind == 2:                                  # steps of BF16 in that range
            l[r, at] = 30.0 + 0.25 * rng.integers(0, 28, n)
        elif kind == 3:                                  # one alone, the rest far below
            l[r, at[0]] = rng.uniform(20.0, 40.0)
        elif kind == 4:                                  # next to 0, everything else below
            l[r] = -1.0 - np.abs(l[r])
            l[r, at] = rng.choice(TINY, n)
        else:                                            # next to 0 below a few others
            l[r, at] = rng.choice(TINY, n)
    _check(w, torch.from_numpy(l), k, None, "sigmoid", G, keep)
    _check(w, torch.from_numpy(l), k, None, "sigmoid", G, keep, False, 2.5)
    _check(w, torch.from_numpy(l).to(torch.bfloat16), k, None, "sigmoid", G, keep)


@pytest.mark.parametrize("T", [64, 5200])
@pytest.mark.parametrize("G,keep", [(1, 1), (4, 2)])
@pytest.mark.parametrize("k", [1, 2, 8, 16])
def test_gate_distinct_logits_of_equal_softmax_scores(w, T, k, G, keep):
    """Logits that the difference to the maximum absorbs, as the maximum and below it."""
    rng = np.random.default_rng(2000 * k + G)
    E = 64
    l = -1.0 - np.abs(rng.standard_normal((T, E))).astype(np.float32)
    for r in range(T):
        n = int(rng.integers(1, E + 1))
        at = rng.permutation(E)[:n]
        l[r, at] = rng.choice(TINY, n)
        if r % 3 == 1:
            l[r, at[0]] = rng.uniform(1.0, 90.0)
        if r % 3 == 2:
            l[r] = np.where(np.isin(np.arange(E), at), l[r], -np.inf)
    for renorm in (True, False):
        _check(w, torch.from_numpy(l), k, None, "softmax", G, keep, renorm)
    _check(w, torch.from_numpy(l).to(torch.bfloat16), k, None, "softmax", G, keep)


@pytest.mark.parametrize("T", [1, 5120])
def test_gate_saturated_pair_goes_to_the_lower_index(w, T):
    """sigmoid(34) and sigmoid(34.01) are one double: expert 3, whatever else decides the path taken."""
    l = np.full((T, 64), -1.0, np.float32)
    l[:, 3], l[:, 7] = 34.0, 34.01
    for k in (1, 2):
        ids, wts = w.moe_gate(dev(l), k, scoring=w.GATE_SIGMOID)
        zero, _ = w.moe_gate(dev(l), k, scoring=w.GATE_SIGMOID, bias=torch.zeros(64, device=DEV))
        sync()
        assert (host(ids) == np.array([3, 7])[:k]).all() and torch.equal(ids, zero)
        assert (host(wts) == np.float32(1.0 / k)).all()


@pytest.mark.parametrize("T", [64, 5200])
@pytest.mark.parametrize("keep", [1, 2, 3])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_gate_group_marks_past_the_float_range(w, T, scoring, keep):
    """Two keys whose sum a float does not hold: a group of them is in, below groups whose
    sum is larger and above groups that have no expert."""
    rng = np.random.default_rng(keep)
    E, G, per = 64, 4, 16
    low = float(np.finfo(np.float32).min)
    for order in ([-3e38, -2e38, low, 0.0], [low, low, -3e38, -2.5e38], [0.0, low, -2e38, -3e38], [-2e38, 3e38, low, 3e38]):
        b = np.repeat(np.array(order), per)
        l = rng.standard_normal((T, E)).astype(np.float32)
        for g in range(G):                               # groups without an expert, and with one
            l[g::7, g * per:(g + 1) * per] = -np.inf
            l[g + 1::9, g * per:(g + 1) * per - 1] = -np.inf
        _check(w, torch.from_numpy(l), 5, b, scoring, G, keep)


@pytest.mark.parametrize("T", [64, 5200])
@pytest.mark.parametrize("G,keep", [(1, 1), (4, 2)])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_softmax_chosen_by_the_bias_far_below_the_maximum(w, T, G, keep, renorm):
    """The bias moves the choice to experts whose scores are 0 or next to it: their sum is 0, and
    so are the weights."""
    rng = np.random.default_rng(G)
    E, k = 64, 4
    l = rng.standard_normal((T, E)).astype(np.float32)
    b = 0.1 * rng.standard_normal(E)
    b[5] = -9.0
    for r, top in enumerate((600.0, 695.0, 700.5, 710.0, 722.0, 760.0, 1000.0, 3e38)):
        l[r::9, 5] = top
    b[E // 4:] -= 1.0                                    # the group of expert 5 is chosen
    _check(w, torch.from_numpy(l), k, b, "softmax", G, keep, renorm)


@pytest.mark.parametrize("T", [64, 5200])
@pytest.mark.parametrize("far", [600.0, 650.0, 690.0])
def test_gate_softmax_scores_that_a_double_holds_in_part(w, T, far):
    """Chosen by the bias: one score e^-far of the maximum's, others 45 under that, which a double
    holds with a few bits. The weights are those of the scores as doubles."""
    rng = np.random.default_rng(int(far))
    E, k = 64, 4
    l = rng.uniform(-1.0, 1.0, (T, E)).astype(np.float32)
    l[:, 5] = far + 45.0
    l[:, 9] = 45.0
    b = 0.1 * rng.standard_normal(E)
    b[5], b[9] = -9.0, 0.5
    _check(w, torch.from_numpy(l), k, b, "softmax")


def test_gate_past_32_bit_offsets(w):
    """The most tokens a call takes: 2^32 logits and more, the tokens on either side of 2^31 and 2^32
    logits and the last ones."""
    T, E, k = (1 << 26) - 4, 68, 2
    g = torch.Generator(device=DEV).manual_seed(1)
    l = torch.randn((T, E), generator=g, device=DEV, dtype=torch.bfloat16)
    ids, wts = w.moe_gate(l, k, scoring=w.GATE_SIGMOID)
    sync()
    at = np.r_[0:4, (1 << 31) // E - 2:(1 << 31) // E + 3, (1 << 32) // E - 2:(1 << 32) // E + 3, T - 5:T]
    rows = torch.from_numpy(at).to(DEV)
    want, ww = O.fp8b.gate(l[rows].double().cpu().numpy(), k, None, "sigmoid")
    assert np.array_equal(host(ids[rows]), want)
    assert np.abs(host(wts[rows]) - ww).max() <= 2.0 ** -23
