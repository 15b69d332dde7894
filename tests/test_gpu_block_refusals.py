"""moe_block_forward: what it refuses before anything is enqueued, and the tensors
that may be the same."""
import ctypes

import pytest
import torch

from bit_quantized_mixture_b200 import moe
from tests.test_gpu_block_path import DEV, WL, layer, outputs, tensors  # noqa: F401 (layer: fixture)

pytestmark = pytest.mark.gpu
T = 12


def arguments(d, o):
    return dict(r=d["r"], x=o["x"], y=o["y"], ids=o["ids"], w=o["w"], w_in=d["w_in"], w_post=d["w_post"], w_next=d["w_next"], x_next=o["x_next"],
                logits=o["logits"], adapter_ids=d["adapter_ids"], router_adapters=d["router_adapters"], layer_adapters=d["layer_adapters"])


def test_results_over_one_another_and_over_what_is_given(layer):  # noqa: F811
    d, o = tensors(T, True, 3), outputs(T)
    kw = arguments(d, o)
    H, E = WL.H, WL.E
    f32 = lambda t, n: t.view(-1).view(torch.float32)[:n]
    i32 = lambda t, n: t.view(-1).view(torch.int32)[:n]
    a, b, s, _ = d["layer_adapters"]
    one = lambda t, shape: t.view(-1)[: shape[0] * shape[1] * shape[2]].view(shape)
    cases = [dict(w=o["ids"].view(torch.float32)), dict(logits=f32(o["x"], T * E).view(T, E)), dict(logits=f32(o["y"], T * E).view(T, E)),
             dict(ids=i32(o["y"], T * WL.k).view(T, WL.k)), dict(w=f32(o["x_next"], T * WL.k).view(T, WL.k)), dict(ids=i32(o["logits"], T * WL.k).view(T, WL.k)),
             dict(ids=i32(d["r"], T * WL.k).view(T, WL.k)), dict(w_in=o["y"][3]), dict(w_post=o["x"][0]), dict(w_post=o["y"][T - 1]), dict(w_next=o["y"][1]),
             dict(adapter_ids=i32(o["ids"], T)), dict(adapter_ids=i32(o["y"], T)),
             dict(layer_adapters=(one(o["x"], (1, 8, H)), b[:1].contiguous(), s[:1].contiguous(), None)),
             dict(layer_adapters=(a[:1].contiguous(), one(o["y"], (1, H, 8)), s[:1].contiguous(), None)),
             dict(layer_adapters=(a, b, f32(o["w"], 3), None)), dict(layer_adapters=(a, b, s, i32(o["logits"], 3))),
             dict(router_adapters=(a, one(o["x_next"], (3, E, 8)), s, None)),
             dict(w_in=d["r"].view(torch.bfloat16).view(-1)[:H]), dict(adapter_ids=i32(d["r"], T)), dict(layer_adapters=(a, b, f32(d["r"], 3), None))]
    r0 = d["r"].clone()
    for over in cases:
        with pytest.raises(moe.MoeError) as e:
            layer.block_forward(**{**kw, **over})
        assert e.value.status == moe.MOE_ERR_INVALID_ARG and "overlap" in str(e.value), over.keys()
    torch.cuda.synchronize()
    assert torch.equal(d["r"], r0) and torch.isnan(o["x"]).all()


@pytest.mark.parametrize("name", ["logits", "topk_ids", "topk_w", "adapter_ids"])
def test_misaligned_addresses(layer, name):  # noqa: F811
    d, o = tensors(T, True, 4), outputs(T)
    blk = moe.Block(r=d["r"].data_ptr(), x=o["x"].data_ptr(), y=o["y"].data_ptr(), topk_ids=o["ids"].data_ptr(), topk_w=o["w"].data_ptr(),
                    logits=o["logits"].data_ptr(), adapter_ids=d["adapter_ids"].data_ptr(), T=T, r_fp32=1, eps=1e-6, branch_scale=1.0, residual_scale=1.0)
    setattr(blk, name, getattr(blk, name) + 2)
    assert moe.lib().moe_block_forward(layer.h, ctypes.byref(blk), None) == moe.MOE_ERR_INVALID_ARG
    assert "4-byte" in moe.lib().moe_last_error(layer.h).decode()


def test_tensors_that_may_be_the_same(layer):  # noqa: F811
    """x_next over x or y, a gate that is one of the results."""
    layer.set_routing(None)
    for name in ("x", "y"):
        for gate in (None, "x", "y"):
            d, o, o2 = tensors(T, False, 5), outputs(T), outputs(T)
            r1, r2 = d["r"].clone(), d["r"].clone()
            layer.block_forward(**{**arguments(d, o), "r": r1, "gate": o[gate] if gate else None})
            layer.block_forward(**{**arguments(d, o2), "r": r2, "gate": o2[gate] if gate else None, "x_next": o2[name] if gate != name else o2["x_next"]})
            layer.sync_status()
            assert torch.equal(r1, r2) and torch.equal(o["x_next"], o2[name] if gate != name else o2["x_next"]) and torch.equal(o["logits"], o2["logits"])
