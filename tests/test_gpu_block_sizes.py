"""moe_block_forward where its parts take their kernels for many tokens: adapters on
tiles and on tcgen05 (bf16 beside the layer, fp32 beside the router), a warp per token
in the selection, four vectors per thread in the norm; in several weight formats."""
import numpy as np
import pytest
import torch

from bit_quantized_mixture_b200 import moe, synth
from bit_quantized_mixture_b200.layer import build_layer
from oracle import moe_oracle as O
from tests.test_gpu_adapters import DEV, assert_close, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quant,T,R", [("int4", 300, 32), ("int4", 1400, 128), ("int4", 7100, 16), ("int2", 700, 64), ("int2", 3300, 8), ("nvfp4", 1, 16),
                                       ("nvfp4", 200, 24), ("nvfp4", 5100, 64)])
def test_equals_its_calls(quant, T, R):
    n = 5
    wl = synth.custom("tiny-int4", quant=quant, T=T, H=256, I=128, E=32, k=4, shared=True)
    layer, _ = build_layer(wl, 0, max_tokens=T)
    if quant == "nvfp4":
        layer.set_act_global_scales(1e-3, 1e-3)    # one scale of a layer's activations, whatever they are
    g = torch.Generator(DEV).manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    H, E, k = wl.H, wl.E, wl.k
    ranks = torch.tensor([R, 1, 0, R - 1, 5], dtype=torch.int32, device=DEV)
    ad = lambda N: ((r(n, R, H) / 16).bfloat16(), (0.3 * r(n, N, R)).bfloat16(), 0.5 + torch.rand(n, generator=g, device=DEV), ranks)
    router, beside = ad(E), ad(H)
    wt = [(1 + 0.1 * r(H)).bfloat16() for _ in range(3)]
    ids_ad = (torch.arange(T, device=DEV) * (n + 1) // T - 1).to(torch.int32)
    rule = moe.Routing("sigmoid", 0.05 * r(E), num_groups=4, top_groups=2, group_score="top2", scale=2.5)
    layer.set_routing(rule)
    r0, gate = r(T, H), r(T)
    bf = lambda: torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    o = dict(x=bf(), y=bf(), x_next=bf(), ids=torch.empty(T, k, dtype=torch.int32, device=DEV), w=torch.empty(T, k, device=DEV), logits=torch.empty(T, E, device=DEV))
    res = r0.clone()
    layer.block_forward(res, w_in=wt[0], w_post=wt[1], w_next=wt[2], gate=gate, gate_sigmoid=True, adapter_ids=ids_ad, router_adapters=router,
                        layer_adapters=beside, branch_scale=0.7, **o)
    layer.sync_status()
    _, x = moe.block_norm(r0, pre_weight=wt[0])
    plain = torch.empty(T, E, device=DEV)
    layer.route(x, None, None, plain)
    logits = moe.add_adapters(x, plain, ids_ad, *router)
    ids, w = moe.select_experts(logits, k, rule)
    y0 = bf()
    layer.forward(x, ids, w, y0)
    y = moe.add_adapters(x, y0, ids_ad, *beside)
    r1, x1 = moe.block_norm(r0, y, wt[1], gate, True, wt[2], branch_scale=0.7)
    layer.sync_status()
    moe.adapters_status()
    for a, b in ((o["x"], x), (o["logits"], logits), (o["ids"], ids), (o["w"], w), (o["y"], y), (res, r1), (o["x_next"], x1)):
        assert torch.equal(a, b)
    # and the parts against their formulas
    assert_close(o["logits"], dict(x=x, y=plain, a=router[0], b=router[1], scales=router[2]), ids_ad, ranks)
    assert_close(o["y"], dict(x=x, y=y0, a=beside[0], b=beside[1], scales=beside[2]), ids_ad, ranks)
    at = np.linspace(0, T - 1, min(T, 200)).astype(int)
    want, _ = O.select_experts(f64(logits)[at], k, score="sigmoid", bias=f64(rule.bias), num_groups=4, top_groups=2, group_score="top2", scale=2.5)
    assert np.array_equal(o["ids"].cpu().numpy()[at], want)
    layer.close()
