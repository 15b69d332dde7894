"""moe_select_experts against the 64-bit oracle: ids equal, weights within the
fp32 roundings of their formula; and the rules through a layer's handle."""
import math

import numpy as np
import pytest
import torch

from bit_quantized_mixture_b200 import moe, synth
from oracle import moe_oracle as O
from tests.gpu_util import bf16_tensor
from tests.test_oracle_block import TIES

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F32_MAX = float(np.finfo(np.float32).max)


def run(L, k, bias=None, **kw):
    rule = moe.Routing(bias=None if bias is None else torch.from_numpy(bias).to(DEV), **kw)
    ids, w = moe.select_experts(torch.from_numpy(L).to(DEV), k, rule)
    return ids.cpu().numpy(), w.cpu().numpy()


def check(L, k, bias=None, **kw):
    """As they are (a CTA per token), and repeated beyond 592 tokens (a warp per token)."""
    rid, rw = O.select_experts(L, k, bias=bias, **kw)
    for n in (1, -(-700 // len(L))):
        ids, w = run(np.tile(L, (n, 1)), k, bias, **kw)
        assert np.array_equal(ids, np.tile(rid, (n, 1)))
        assert_weights(L, w, np.tile(rw, (n, 1)), kw.get("scale", 1.0))


def assert_weights(L, w, rw, scale=1.0):
    # exp of a difference up to D: the difference's rounding D 2^-24, exp itself
    # 2 ulp = 2^-22 relative; sums of up to 1024 terms, 32 in a row and 5 folds
    # (37 x 2^-24), one division each for score and weight, the scale: twice
    # (numerator and sum) (D + 4) + 37 + 8 units of 2^-24; below 2^-126 nothing
    # is promised of a score
    fin = np.where(np.abs(L) < 1e30, L, 0.0)
    D = min(float(fin.max() - fin.min()), 104.0)
    tol = 2.0 ** -24 * (2 * (D + 4) + 45)
    assert np.all(np.abs(w - rw) <= tol * np.abs(rw) + 2.0 ** -125 * max(1.0, abs(scale)))


RULES = [
    dict(),
    dict(renorm=False, scale=2.5),
    dict(score="sigmoid"),
    dict(score="sigmoid", renorm=False, scale=0.5),
]


@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (31, 31), (32, 32), (33, 7), (40, 25), (256, 8), (512, 10), (600, 10), (1024, 32), (1000, 1)])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("rule", range(len(RULES)))
def test_scores_and_bias(E, k, biased, rule):
    rng = np.random.default_rng(E * 100 + k * 2 + biased)
    L = rng.standard_normal((13, E)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if biased else None
    check(L, k, bias, **RULES[rule])


@pytest.mark.parametrize("E,G,keep,k", [(64, 8, 4, 8), (256, 8, 4, 8), (512, 8, 3, 10), (512, 32, 5, 32), (600, 24, 5, 7), (1024, 4, 1, 32),
                                        (24, 24, 7, 5), (96, 3, 3, 32), (1000, 5, 2, 9), (32, 32, 1, 1), (34, 2, 1, 17)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(E, G, keep, k, group_score, score, biased):
    rng = np.random.default_rng(E + G + k)
    L = (1.5 * rng.standard_normal((11, E))).astype(np.float32)
    bias = (0.2 * rng.standard_normal(E)).astype(np.float32) if biased else None
    check(L, k, bias, score=score, num_groups=G, top_groups=keep, group_score=group_score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("renorm", [True, False])
def test_masks(score, G, renorm):
    """NaN, -inf and the lowest value in logits; +inf; rows with fewer eligible
    experts than k, one, none; groups without an eligible expert; biases that
    switch experts off."""
    E, k = 48, 6
    rng = np.random.default_rng(5)
    L = rng.standard_normal((16, E)).astype(np.float32)
    L[0] = -np.inf
    L[1] = np.nan
    L[2] = -F32_MAX
    L[3, 1:] = -np.inf
    L[4, :45] = -F32_MAX
    L[5, ::2] = np.nan
    L[6, :36] = -np.inf
    L[7, 5] = np.inf
    L[8, [3, 40]] = np.inf
    L[9] = np.inf
    L[10] = F32_MAX
    L[11] = -3e38
    L[12, 20:] = -np.inf
    L[13, ::3] = 0.0
    L[13, 1::3] = -0.0
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    bias[[2, 17, 33]] = [-np.inf, np.nan, -F32_MAX]
    bias[7] = np.inf
    for b in (None, bias):
        for gs in ("max", "top2"):
            check(L, k, b, score=score, num_groups=G, top_groups=max(1, G // 2), group_score=gs, renorm=renorm)


@pytest.mark.parametrize("score,shift,spread", [("sigmoid", 45.0, 3.0), ("sigmoid", 120.0, 30.0), ("sigmoid", -900.0, 60.0), ("softmax", 0.0, 400.0)])
@pytest.mark.parametrize("E,G,keep", [(40, 1, 1), (512, 1, 1), (512, 8, 3), (1000, 5, 2)])
@pytest.mark.parametrize("level", [0.0, 0.75])
def test_a_bias_of_one_value_changes_no_order(score, shift, spread, E, G, keep, level):
    """Saturated and vanished scores, whose keys are equal in 64 bits: their logits
    say which is larger, as without a bias (up to 1000 of them, more than a list
    holds, and a few among others)."""
    k = 8
    rng = np.random.default_rng(E + G)
    L = (shift + spread * rng.standard_normal((10, E))).astype(np.float32)
    if score == "sigmoid" and shift > 0:
        L[5:, 9:] -= shift + 30.0
    bias = np.full(E, level, dtype=np.float32)
    check(L, k, bias, score=score, num_groups=G, top_groups=keep)
    want, _ = run(L, k, score=score, num_groups=G, top_groups=keep)
    got, _ = run(L, k, bias, score=score, num_groups=G, top_groups=keep)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("score,la,lb,b1,b2", TIES)
@pytest.mark.parametrize("others", [0, 90])
def test_groups_of_the_same_scores_and_biases_tie(score, la, lb, b1, b2, others):
    """The lower group stays, with two more groups' worth of low experts and (more equal
    keys than a list holds) with groups of 92."""
    per = 2 + others
    low = lambda pair: pair + [-30.0] * others
    L = np.array([low([la, lb]) + low([lb, la]) + [-30.0] * per, low([lb, la]) + low([la, lb]) + [-30.0] * per], dtype=np.float32)
    bias = np.full(3 * per, -1.0, dtype=np.float32)
    bias[[0, per]], bias[[1, per + 1]] = b1, b2
    check(L, 2, bias, score=score, num_groups=3, top_groups=1, group_score="top2")
    ids, _ = run(L, 2, bias, score=score, num_groups=3, top_groups=1, group_score="top2")
    assert (np.sort(ids, axis=1) == [0, 1]).all()


@pytest.mark.parametrize("E,G,keep", [(48, 1, 1), (48, 4, 2), (600, 24, 5), (1024, 1, 1)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_a_bias_that_is_off_changes_no_score(E, G, keep, group_score):
    """Unnormalised softmax weights of the experts that are left are those of the
    whole row, also where the ones switched off hold nearly all of it, in rows
    decided in fp32 and (equal keys) in fp64, and in rows with more equal
    keys than a list holds."""
    k = 6
    rng = np.random.default_rng(E + G)
    L = rng.standard_normal((12, E)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    bias[::5] = -np.inf
    bias[1::7] = np.nan
    L[1, ::5] += 20.0
    L[2] = 0.5
    L[3, 1::7] = -np.inf
    check(L, k, bias, renorm=False, scale=2.5, num_groups=G, top_groups=keep, group_score=group_score)
    bias = np.where(np.arange(E) % 5 == 0, -np.inf, 0.25).astype(np.float32)
    L[4:8] = np.float32(0.25) * rng.integers(-1, 2, size=(4, E))
    check(L, k, bias, renorm=False, num_groups=G, top_groups=keep, group_score=group_score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(score):
    """Scores that underflow or saturate: the order stays the logits' and
    renormalised weights their exact ratios."""
    L = np.array([[-200, -201, -203, -220, -1000, -150.5], [100, 90, 99.5, -100, 40, 41], [-3e38, -2e38, -1e38, 3e38, 1, 2],
                  [-104, -103, -100, -87, -88, -89], [0, 0, 0, 0, 0, 0]], dtype=np.float32)
    for renorm in (True, False):
        check(L, 3, score=score, renorm=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift,spread", [(-30.0, 1.0), (-12.0, 0.01), (0.0, 12.0), (-90.0, 5.0), (20.0, 2.0)])
@pytest.mark.parametrize("bias", [None, 0.0, 1e-6])
def test_small_peaked_and_saturated_scores(score, shift, spread, bias):
    """Scores far below one, one expert that has nearly all, scores near one; biases
    of the scores' own size."""
    E, k = 256, 8
    rng = np.random.default_rng(21)
    L = (shift + spread * rng.standard_normal((12, E))).astype(np.float32)
    b = None if bias is None else (bias * rng.standard_normal(E)).astype(np.float32)
    for G, keep, gs in ((1, 1, "max"), (8, 3, "top2"), (8, 3, "max")):
        if shift == 20.0 and score == "sigmoid" and (b is not None or gs == "top2"):
            continue              # 1 - exp(-20): keys and sums differ below 64 bits' own rounding
        if shift == -90.0 and b is not None:
            continue              # scores vanish beside any bias
        check(L, k, b, score=score, num_groups=G, top_groups=keep, group_score=gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1, "max"), (8, 3, "top2"), (8, 3, "max")])
def test_keys_nearer_than_fp32_tells(score, groups):
    """Biases that bring every key to one value up to their own rounding
    (2^-25): the order is decided far below an fp32 key's error."""
    E, k = 256, 8
    rng = np.random.default_rng(9)
    L = rng.standard_normal((40, E)).astype(np.float32)
    x = L[:1].astype(np.float64)
    s = 1 / (1 + np.exp(-x)) if score == "sigmoid" else np.exp(x) / np.exp(x).sum()
    bias = (0.75 - s[0]).astype(np.float32)
    L[1] = L[0]
    L[2:] = L[0] + (np.float32(1e-7) * rng.standard_normal((38, E))).astype(np.float32)
    G, keep, gs = groups
    check(L, k, bias, score=score, num_groups=G, top_groups=keep, group_score=gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 2, 5])
@pytest.mark.parametrize("equal", [2, 3, 30])
def test_equal_keys_at_the_border_hide_no_larger_one(score, k, equal):
    """`equal` experts with one logit and bias, and behind them one whose key is larger by less than fp32
    tells (a saturated sigmoid, or a bias that absorbs the difference): it comes first."""
    E, T = 64, 4
    L = np.full((T, E), -40.0, dtype=np.float32)
    bias = np.zeros(E, dtype=np.float32)
    L[:, 3:3 + equal] = 21.5
    L[:, 50] = 30.0 if score == "sigmoid" else 21.501
    if score == "softmax":
        bias[:] = 1e5
    want, _ = O.select_experts(L, k, score=score, bias=bias)
    assert (want[:, 0] == 50).all()
    check(L, k, bias, score=score)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [(1, 1, "max"), (4, 2, "top2"), (8, 4, "max")])
def test_equal_keys_go_to_the_lowest(biased, groups):
    E, k = 512, 10
    rng = np.random.default_rng(1)
    L = rng.integers(-2, 3, size=(20, E)).astype(np.float32) * np.float32(0.5)
    L[0] = 0.25
    bias = (rng.integers(0, 2, size=E) * 0.5).astype(np.float32) if biased else None
    G, keep, gs = groups
    for score in ("softmax", "sigmoid"):
        check(L, k, bias, score=score, num_groups=G, top_groups=keep, group_score=gs)


@pytest.mark.parametrize("T", [250, 3000])
def test_many_tokens_and_row_distance(T):
    E, k = 128, 6
    rng = np.random.default_rng(2)
    L = rng.standard_normal((T, E)).astype(np.float32)
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    wide = torch.full((T, 200), 50.0, device=DEV)
    wide[:, 3:3 + E] = torch.from_numpy(L).to(DEV)
    ids, w = moe.select_experts(wide[:, 3:3 + E], k, moe.Routing("sigmoid", torch.from_numpy(bias).to(DEV)))
    ref_ids, ref_w = moe.select_experts(torch.from_numpy(L).to(DEV), k, moe.Routing("sigmoid", torch.from_numpy(bias).to(DEV)))
    assert torch.equal(ids, ref_ids) and torch.equal(w, ref_w)
    at = rng.choice(T, 200, replace=False)
    rid, rw = O.select_experts(L[at], k, score="sigmoid", bias=bias)
    assert np.array_equal(ids.cpu().numpy()[at], rid)
    assert_weights(L, w.cpu().numpy()[at], rw)


@pytest.mark.parametrize("T", [1, 77, 900])
def test_plain_rule_equals_the_built_in_route(T):
    E, k = 512, 10
    layer = moe.MoeLayer(128, 128, E, k, "int4", False, T, 0)
    L = torch.randn(T, E, device=DEV, generator=torch.Generator(DEV).manual_seed(4))
    ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    layer.route_from_logits(L, ids, w)
    i2, w2 = moe.select_experts(L, k, moe.Routing())
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    layer.close()


@pytest.mark.parametrize("T", [1, 5, 40])
def test_a_layers_routing_rule(T):
    """set_routing changes route, route_from_logits and route_forward; None
    restores them; the layer runs under the rule as under given ids."""
    from bit_quantized_mixture_b200.layer import build_layer
    wl = synth.custom("tiny-int4", T=T, H=256, I=128, E=64, k=6)
    layer, _ = build_layer(wl, 0, max_tokens=T)
    x = bf16_tensor(synth.activations_bf16(wl), DEV)
    bias = torch.linspace(-0.2, 0.2, wl.E, device=DEV)
    rule = moe.Routing("sigmoid", bias, num_groups=8, top_groups=3, group_score="top2", scale=2.5)
    new = lambda: (torch.empty(T, wl.k, dtype=torch.int32, device=DEV), torch.empty(T, wl.k, device=DEV))
    logits = torch.empty(T, wl.E, device=DEV)
    ids0, w0 = new()
    y0 = torch.empty(T, wl.H, dtype=torch.bfloat16, device=DEV)
    layer.route_forward(x, ids0, w0, y0)
    layer.set_routing(rule)
    ids, w = new()
    layer.route(x, ids, w, logits)
    rid, rw = O.select_experts(logits.cpu().numpy(), wl.k, score="sigmoid", bias=bias.cpu().numpy(), num_groups=8, top_groups=3,
                               group_score="top2", scale=2.5)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert_weights(logits.cpu().numpy(), w.cpu().numpy(), rw, 2.5)
    ids2, w2 = new()
    layer.route_from_logits(logits, ids2, w2)
    assert torch.equal(ids2, ids) and torch.equal(w2, w)
    y, y2 = torch.empty_like(y0), torch.empty_like(y0)
    ids3, w3 = new()
    layer.route_forward(x, ids3, w3, y)
    assert torch.equal(ids3, ids) and torch.equal(w3, w)
    layer.forward(x, ids, w, y2)
    layer.sync_status()
    assert torch.equal(y, y2)
    layer.set_routing(None)
    ids4, w4 = new()
    y4 = torch.empty_like(y0)
    layer.route_forward(x, ids4, w4, y4)
    layer.sync_status()
    assert torch.equal(ids4, ids0) and torch.equal(w4, w0) and torch.equal(y4, y0)
    with pytest.raises(moe.MoeError):
        layer.set_routing(moe.Routing(num_groups=7, top_groups=1))
    with pytest.raises(moe.MoeError):
        layer.set_routing(moe.Routing(bias=torch.zeros(8, device=DEV)))
    layer.close()


@pytest.mark.parametrize("T", [50, 800])
def test_streams_and_graphs(T):
    """On a stream of the caller's, and captured and replayed on new logits."""
    E, k = 512, 10
    rule = moe.Routing("sigmoid", torch.linspace(0, 0.3, E, device=DEV), num_groups=8, top_groups=4, group_score="top2")
    L = torch.randn(T, E, device=DEV)
    want = moe.select_experts(L, k, rule)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.select_experts(L, k, rule, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ids, w = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        moe.select_experts(L, k, rule, ids=ids, w=w)
    for seed in (1, 2):
        L.copy_(torch.randn(T, E, device=DEV, generator=torch.Generator(DEV).manual_seed(seed)))
        g.replay()
        want = moe.select_experts(L, k, rule)
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
