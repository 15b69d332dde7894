"""Pins of the oracle's expert selection, adapters and block norm against
hand-worked examples, and the refusals of their entry points (no GPU: every
refused call returns before device work)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from bit_quantized_mixture_b200 import moe
from oracle import moe_oracle as O

F32_MAX = float(np.finfo(np.float32).max)


# ------------------------------------------------------------- the oracle
def test_selection_without_a_rule_is_softmax_top_k():
    rng = np.random.default_rng(3)
    L = rng.standard_normal((9, 24)).astype(np.float32)
    ids, w = O.select_experts(L, 5)
    rid, rw = O.route_topk(L, 5)
    assert np.array_equal(ids, rid) and np.allclose(w, rw, rtol=1e-6, atol=0)


def test_selection_worked_example():
    # sigmoid scores 1/2, 1/(1+1/3) = 3/4, 1/4, 1/2 with logits 0, ln 3, -ln 3, 0
    L = np.array([[0.0, math.log(3), -math.log(3), 0.0]], dtype=np.float32)
    ids, w = O.select_experts(L, 2, score="sigmoid")
    assert ids.tolist() == [[1, 0]] and np.allclose(w, [[0.6, 0.4]], atol=1e-7)      # equal scores: the lower expert
    bias = np.array([0, 0, 0.6, 0], dtype=np.float32)                                # key of 2: 0.85, weight by 0.25
    ids, w = O.select_experts(L, 2, score="sigmoid", bias=bias, renorm=False, scale=2.0)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[0.5, 1.5]], atol=1e-7)
    # groups (0, 1) and (2, 3): largest key 0.75 against 0.5; two largest 1.25 against 0.75
    for kind in ("max", "top2"):
        ids, _ = O.select_experts(L, 2, score="sigmoid", num_groups=2, top_groups=1, group_score=kind)
        assert ids.tolist() == [[1, 0]]


def test_selection_masks():
    L = np.array([[np.nan, -np.inf, -F32_MAX, 1.0], [-np.inf] * 4, [np.inf, 0.0, np.inf, 0.0]], dtype=np.float32)
    ids, w = O.select_experts(L, 2)
    assert ids.tolist() == [[3, 0], [0, 1], [0, 2]]
    assert w.tolist() == [[1.0, 0.0], [0.0, 0.0], [0.5, 0.5]]


def test_keys_that_are_equal_in_64_bits_go_by_their_logits():
    """Scores that saturate, or vanish beside their biases: a bias of one value
    changes no order."""
    L = np.array([[40.0, 50.0, 45.0, 50.0], [-800.0, -900.0, -850.0, 0.0]], dtype=np.float32)
    for bias in (None, np.zeros(4, dtype=np.float32), np.full(4, 3.0, dtype=np.float32)):
        assert O.select_experts(L, 3, score="sigmoid", bias=bias)[0].tolist() == [[1, 3, 2], [3, 0, 2]]
        assert O.select_experts(L, 1, score="sigmoid", bias=bias, num_groups=2)[0].tolist() == [[1], [3]]
        assert O.select_experts(L[:1, [2, 0, 1, 0]], 1, score="sigmoid", bias=bias, num_groups=2)[0].tolist() == [[2]]
    for bias in (None, np.zeros(4, dtype=np.float32)):
        assert O.select_experts(L, 3, bias=bias)[0].tolist() == [[1, 3, 2], [3, 0, 2]]


TIES = [("softmax", 0.5, 1.0, 0.375, 0.0), ("softmax", 1.0, 0.5, 0.125, 0.25), ("softmax", -0.5, 0.25, 0.375, 0.0), ("sigmoid", 1.0, 0.5, 0.375, 0.125),
        ("sigmoid", 0.5, 3.0, -0.125, 0.125), ("sigmoid", 3.0, 0.5, 0.25, -0.125)]


@pytest.mark.parametrize("score,la,lb,b1,b2", TIES)
def test_groups_of_the_same_scores_and_biases_tie(score, la, lb, b1, b2):
    """(s_a + b_1) + (s_b + b_2) and (s_b + b_1) + (s_a + b_2) are one sum, which a
    rounding of each key would tell apart: the lower group stays."""
    bias = np.array([b1, b2, b1, b2, -1, -1], dtype=np.float32)
    for L in ([la, lb, lb, la, -3, -4], [lb, la, la, lb, -3, -4]):
        ids, _ = O.select_experts(np.array([L], dtype=np.float32), 2, score=score, bias=bias, num_groups=3, top_groups=1, group_score="top2")
        assert sorted(ids[0].tolist()) == [0, 1]


def test_a_bias_takes_no_part_in_the_scores():
    """Softmax scores 1/2, 1/4, 1/4; a bias that switches expert 0 off leaves the
    others theirs."""
    L = np.array([[math.log(2), 0.0, 0.0]], dtype=np.float32)
    for off in (-np.inf, np.nan, -F32_MAX):
        ids, w = O.select_experts(L, 2, bias=np.array([off, 0, 0.5], dtype=np.float32), renorm=False, scale=4.0)
        assert ids.tolist() == [[2, 1]] and np.allclose(w, [[1.0, 1.0]], atol=1e-7)


def test_adapters_worked_example():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    y = np.array([[10.0], [20.0], [30.0]])
    a = np.array([[[1.0, 0.0], [0.0, 1.0]], [[1.0, 1.0], [9.0, 9.0]]])
    b = np.array([[[2.0, 3.0]], [[5.0, 7.0]]])
    out = O.add_adapters(x, y, [0, -1, 1], a, b, [0.5, 2.0], ranks=[2, 1])
    assert out.tolist() == [[10 + 0.5 * (2 + 6)], [20], [30 + 2 * 5 * 11]]


def test_block_norm_worked_example():
    r, x = O.block_norm([[1.0, 1.0]], y=[[3.0, -1.0]], w_post=np.array([1.0, 1.0]), gate=np.array([[2.0]]), w_pre=np.array([1.0, 2.0]),
                        eps=1e-12, branch_scale=0.5, residual_scale=3.0)
    u = np.array([3.0, -1.0]) / math.sqrt(5.0)
    assert np.allclose(r, 3.0 + u)
    assert np.allclose(x, (3.0 + u) / math.sqrt(((3.0 + u) ** 2).mean()) * [1, 2])


# -------------------------------------------------------------- refusals
BUF = ctypes.create_string_buffer(1 << 16)
BASE = (ctypes.addressof(BUF) + 255) & ~255          # never dereferenced


def _err():
    return moe.lib().moe_last_error(None).decode()


def _rule(**kw):
    f = dict(score=0, num_groups=1, top_groups=1, group_score=0, renorm=1, scale=1.0, bias=None)
    f.update(kw)
    return moe.RoutingRule(**f)


@pytest.mark.parametrize("rule,args,status,text", [
    ({}, dict(E=1025), 2, "E <= 1024"),
    ({}, dict(E=0), 2, "E <= 1024"),
    ({}, dict(k=33), 2, "k <= min"),
    ({}, dict(E=4, k=5), 2, "k <= min"),
    ({}, dict(T=-1), 1, "negative T"),
    ({}, dict(ld=63), 1, "ld_logits"),
    ({}, dict(logits=None), 1, "null"),
    ({}, dict(ids=None), 1, "null"),
    ({"score": 2}, {}, 1, "unknown score"),
    ({"group_score": 7}, {}, 1, "unknown group score"),
    ({"num_groups": 33}, dict(E=66), 2, "32 groups"),
    ({"num_groups": 5}, {}, 1, "divide E"),
    ({"num_groups": 0}, {}, 1, "divide E"),
    ({"num_groups": 8, "top_groups": 9}, {}, 1, "top_groups"),
    ({"num_groups": 16, "top_groups": 2}, dict(k=9), 1, "fewer than k"),
    ({"scale": float("nan")}, {}, 1, "finite"),
    ({"renorm": 2}, {}, 1, "renorm"),
])
def test_select_refusals(rule, args, status, text):
    a = dict(logits=BASE, ld=64, T=4, E=64, k=8, ids=BASE, w=BASE)
    a.update(args)
    st = moe.lib().moe_select_experts(a["logits"], a["ld"], a["T"], a["E"], a["k"], _rule(**rule), a["ids"], a["w"], None)
    assert st == status and text in _err()


def test_no_tokens_is_a_no_op():
    L = moe.lib()
    assert L.moe_select_experts(BASE, 64, 0, 64, 8, _rule(), BASE, BASE, None) == 0
    assert L.moe_add_adapters(BASE, 64, BASE + 8192, 64, BASE + 8192, 64, 0, 0, BASE, _adapters(), None) == 0
    n = _norm(T=0)
    assert L.moe_block_norm(n, None) == 0


def _adapters(**kw):
    f = dict(a=BASE, b=BASE, scales=BASE, ranks=None, num_adapters=2, R=16, K=64, N=64)
    f.update(kw)
    return moe.AdapterSet(**f)


@pytest.mark.parametrize("ad,args,status,text", [
    ({"R": 12}, {}, 2, "multiples of 8"),
    ({"R": 136}, {}, 2, "multiples of 8"),
    ({"R": 0}, {}, 2, "multiples of 8"),
    ({"K": 60}, {}, 2, "multiples of 8"),
    ({"N": 4}, {}, 2, "multiples of 8"),
    ({"num_adapters": 0}, {}, 1, "num_adapters"),
    ({"a": None}, {}, 1, "null"),
    ({"a": BASE + 2}, {}, 1, "aligned"),
    ({}, dict(x=None), 1, "null"),
    ({}, dict(ids=None), 1, "null"),
    ({}, dict(T=-3), 1, "negative T"),
    ({}, dict(ldx=56), 1, "width apart"),
    ({}, dict(ldx=68), 1, "width apart"),
    ({}, dict(x=BASE + 8), 1, "width apart"),
    ({}, dict(ldy=60, y32=1), 1, "width apart"),
    ({}, dict(out=BASE), 1, "overlaps"),                       # out is x
    ({}, dict(out=BASE + 8192 + 128), 1, "overlaps"),          # out is y, one row on
    ({}, dict(ldo=128, out=BASE + 8192), 1, "overlaps"),       # in place with another distance
])
def test_adapter_refusals(ad, args, status, text):
    a = dict(x=BASE, ldx=64, y=BASE + 8192, ldy=64, out=BASE + 8192, ldo=64, y32=0, T=4, ids=BASE)
    a.update(args)
    st = moe.lib().moe_add_adapters(a["x"], a["ldx"], a["y"], a["ldy"], a["out"], a["ldo"], a["y32"], a["T"], a["ids"], _adapters(**ad), None)
    assert st == status and text in _err()


def _norm(**kw):
    f = dict(r=BASE, y=BASE + 4096, w_post=BASE, w_pre=BASE, r_out=BASE, x_out=BASE + 8192, ld_r=64, ld_y=64, ld_gate=64, ld_r_out=64,
             ld_x=64, T=4, H=64, eps=1e-6, branch_scale=1.0, residual_scale=1.0)
    f.update(kw)
    return moe.Norm(**f)


@pytest.mark.parametrize("kw,status,text", [
    (dict(H=60), 2, "multiple of 8"),
    (dict(H=16392), 2, "16384"),
    (dict(T=-1), 1, "negative T"),
    (dict(r=None), 1, "need r"),
    (dict(r_out=None, x_out=None, w_pre=None), 1, "need r"),
    (dict(w_pre=None), 1, "w_pre exactly"),
    (dict(x_out=None), 1, "w_pre exactly"),
    (dict(gate_kind=4, gate=BASE), 1, "gate kind"),
    (dict(gate_kind=1), 1, "go together"),
    (dict(gate=BASE), 1, "go together"),
    (dict(y=None), 1, "need y"),
    (dict(eps=0.0), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"),
    (dict(branch_scale=float("inf")), 1, "finite"),
    (dict(ld_y=56), 1, "apart"),
    (dict(ld_x=66), 1, "apart"),
    (dict(r=BASE + 4, r_out=BASE + 4), 1, "aligned"),
    (dict(gate_kind=1, gate=BASE + 2), 1, "aligned"),
    (dict(r_out=BASE + 4096), 1, "overlaps"),                  # r_out is y
    (dict(x_out=BASE), 1, "overlaps"),                         # x_out is r
    (dict(r_out=BASE + 128), 1, "overlaps"),                   # r, one row on
    (dict(gate_kind=3, gate=BASE + 8192), 1, "overlaps"),      # x_out is the gate
    (dict(r=BASE, ld_r=128, r_out=BASE + 16384, y=BASE + 64, ld_y=128, x_out=BASE + 64, ld_x=64), 1, "overlaps"),
])
def test_norm_refusals(kw, status, text):
    n = _norm(**kw)
    st = moe.lib().moe_block_norm(n, None)
    assert st == status and text in _err()


@pytest.mark.parametrize("ad,ids", [
    (dict(a=BASE + 8192 + 496), BASE), (dict(a=BASE + 8192 - 4096 + 16), BASE), (dict(b=BASE + 8192), BASE), (dict(scales=BASE + 8192 + 508), BASE),
    (dict(ranks=BASE + 8192 - 4), BASE), ({}, BASE + 8192 + 256), (dict(num_adapters=0x7fffffff, R=128, K=64), BASE)])
def test_adapters_refuse_outputs_over_their_inputs(ad, ids):
    """out, 512 bytes at BASE + 8192, over the adapters (the last: 2^45 bytes from BASE
    on), their scales and ranks, the ids."""
    st = moe.lib().moe_add_adapters(BASE, 64, BASE + 16384, 64, BASE + 8192, 64, 0, 4, ids, _adapters(**ad), None)
    assert st == 1 and "overlaps" in _err()


@pytest.mark.parametrize("kw", [
    dict(w_post=BASE + 128), dict(w_post=BASE + 8192 + 256), dict(w_pre=BASE + 384), dict(w_pre=BASE + 8192 - 16),
    dict(gate_kind=1, gate=BASE + 64), dict(gate_kind=1, gate=BASE + 8192), dict(gate_kind=2, gate=BASE + 508), dict(gate_kind=2, gate=BASE + 8192 - 12),
    dict(ld_x=128, w_pre=BASE + 8192 + 256 + 64), dict(ld_x=128, w_pre=BASE + 8192 + 128 + 16)])
def test_norm_refuses_outputs_over_what_every_row_reads(kw):
    """r_out is 512 bytes at BASE, x_out 512 at BASE + 8192 (896 with rows 256 apart)."""
    far = dict(w_post=BASE + 16384, w_pre=BASE + 16640)
    assert moe.lib().moe_block_norm(_norm(**{**far, **kw}), None) == 1 and "overlaps" in _err()


def test_addresses_and_sizes_out_of_range():
    """Row distances whose addresses would pass 64 bits, tokens past 2^30, misaligned 4-byte tensors, and
    selections written over what they read."""
    L = moe.lib()
    far = BASE + 32768

    def select(logits=BASE, ld=64, T=4, ids=far, w=far + 4096, bias=None):
        return L.moe_select_experts(logits, ld, T, 64, 8, _rule(bias=bias), ids, w, None)

    def adapters(T=4, ld=64, ids=BASE, **kw):
        return L.moe_add_adapters(BASE, ld, BASE + 8192, 64, BASE + 8192, 64, 0, T, ids, _adapters(**kw), None)

    def norm(**kw):
        return L.moe_block_norm(_norm(**kw), None)

    for st, status, text in (
            (lambda: select(ld=1 << 62), 1, "out of range"),
            (lambda: select(ld=1 << 55), 1, "out of range"),
            (lambda: select(T=(1 << 30) + 1), 2, "2^30"),
            (lambda: select(logits=BASE + 2), 1, "4-byte"),
            (lambda: select(ids=far + 1), 1, "4-byte"),
            (lambda: select(w=far + 4098), 1, "4-byte"),
            (lambda: select(bias=BASE + 3), 1, "4-byte"),
            (lambda: select(ids=BASE + 128), 1, "overlaps"),
            (lambda: select(w=far + 64), 1, "overlaps"),
            (lambda: select(w=BASE), 1, "overlaps"),
            (lambda: select(bias=far), 1, "overlaps"),
            (lambda: adapters(ld=1 << 60), 1, "width apart"),
            (lambda: adapters(T=(1 << 30) + 1), 2, "2^30"),
            (lambda: adapters(K=(1 << 30) + 8), 2, "2^30"),
            (lambda: adapters(N=(1 << 30) + 8), 2, "2^30"),
            (lambda: adapters(ids=BASE + 2), 1, "4-byte"),
            (lambda: adapters(scales=BASE + 2), 1, "4-byte"),
            (lambda: adapters(ranks=BASE + 1), 1, "4-byte"),
            (lambda: norm(ld_y=1 << 60), 1, "apart"),
            (lambda: norm(T=(1 << 30) + 1), 2, "2^30"),
            (lambda: norm(gate_kind=2, gate=BASE + 2), 1, "aligned")):
        assert st() == status and text in _err(), text


def test_a_rules_bias_is_fixed():
    rule = moe.Routing()
    assert rule.bias is None
    with pytest.raises(AttributeError):
        rule.bias = torch.zeros(4)


def test_handle_calls_refuse_null():
    L = moe.lib()
    assert L.moe_set_routing(None, _rule(), None) == 1
    assert L.moe_block_forward(None, moe.Block(), None) == 1
    assert L.moe_block_norm(None, None) == 1
    assert L.moe_select_experts(BASE, 64, 4, 64, 8, None, BASE, BASE, None) == 1
    assert L.moe_add_adapters(BASE, 64, BASE, 64, BASE, 64, 0, 4, BASE, None, None) == 1


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: moe.select_experts(torch.zeros(4, 8), 2, moe.Routing()),
                 lambda: moe.add_adapters(x, x, torch.zeros(4, dtype=torch.int32), x.view(1, 4, 64), x.view(1, 64, 4), torch.ones(1)),
                 lambda: moe.block_norm(x),
                 lambda: moe.Routing(score="linear"),
                 lambda: moe.Routing(bias=torch.zeros(4))):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == moe.MOE_ERR_INVALID_ARG
