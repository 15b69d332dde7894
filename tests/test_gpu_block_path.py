"""moe_block_forward: the norm, the layer under a routing rule with adapters
beside its router and beside itself, and the norm behind it, as one run."""
import numpy as np
import pytest
import torch

from bit_quantized_mixture_b200 import moe, synth
from bit_quantized_mixture_b200.layer import build_layer
from oracle import moe_oracle as O
from tests.gpu_util import OracleExperts

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
WL = synth.custom("tiny-int4", T=40, H=256, I=128, E=32, k=4, shared=True)
N_AD, RANK = 3, 8


@pytest.fixture(scope="module")
def layer():
    la = build_layer(WL, 0, max_tokens=WL.T)[0]
    yield la
    la.close()


def tensors(T, wide, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    H, E = WL.H, WL.E
    wt = lambda: (1 + 0.1 * r(H)).bfloat16()
    ad = lambda N: ((r(N_AD, RANK, H) / H ** 0.5).bfloat16(), (0.3 * r(N_AD, N, RANK)).bfloat16(), 0.5 + torch.rand(N_AD, generator=g, device=DEV), None)
    return dict(r=r(T, H).to(torch.float32 if wide else torch.bfloat16), w_in=wt(), w_post=wt(), w_next=wt(), gate=r(T),
                router_adapters=ad(E), layer_adapters=ad(H), adapter_ids=(torch.arange(T, device=DEV) % (N_AD + 1) - 1).to(torch.int32),
                rule=moe.Routing("sigmoid", 0.05 * r(E), num_groups=4, top_groups=2, group_score="top2", scale=2.5))


def outputs(T):
    H, E, k = WL.H, WL.E, WL.k
    bf = lambda: torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    return dict(x=bf(), y=bf(), ids=torch.empty(T, k, dtype=torch.int32, device=DEV), w=torch.empty(T, k, device=DEV), x_next=bf(),
                logits=torch.empty(T, E, device=DEV))


def run_block(layer, d, o, r):
    layer.set_routing(d["rule"])
    layer.block_forward(r, o["x"], o["y"], o["ids"], o["w"], w_in=d["w_in"], w_post=d["w_post"], w_next=d["w_next"], x_next=o["x_next"], gate=d["gate"],
                        gate_sigmoid=True, logits=o["logits"], adapter_ids=d["adapter_ids"], router_adapters=d["router_adapters"],
                        layer_adapters=d["layer_adapters"], branch_scale=0.7)


@pytest.mark.parametrize("T", [1, 6, 40])
@pytest.mark.parametrize("wide", [False, True])
def test_equals_its_calls(layer, T, wide):
    d, o = tensors(T, wide, T), outputs(T)
    r = d["r"].clone()
    run_block(layer, d, o, r)
    layer.sync_status()
    _, x = moe.block_norm(d["r"], pre_weight=d["w_in"])
    logits = torch.empty_like(o["logits"])
    layer.route(x, None, None, logits)
    moe.add_adapters(x, logits, d["adapter_ids"], *d["router_adapters"][:3], out=logits)
    ids, w = moe.select_experts(logits, WL.k, d["rule"])
    y = torch.empty_like(o["y"])
    layer.forward(x, ids, w, y)
    moe.add_adapters(x, y, d["adapter_ids"], *d["layer_adapters"][:3], out=y)
    r2, x2 = moe.block_norm(d["r"], y, d["w_post"], d["gate"], True, d["w_next"], branch_scale=0.7)
    layer.sync_status()
    for a, b in ((o["x"], x), (o["logits"], logits), (o["ids"], ids), (o["w"], w), (o["y"], y), (r, r2), (o["x_next"], x2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 40])
def test_against_the_oracle(layer, T):
    """The whole run from r in 64 bits, at the ids that the run chose: each
    bf16 rounding on the way is half a step, 2^-8 of its value, and the
    quantized layer's own bound is 1e-2 of its output."""
    d, o = tensors(T, True, 100 + T), outputs(T)
    r = d["r"].clone()
    run_block(layer, d, o, r)
    layer.sync_status()
    f = lambda t: t.double().cpu().numpy()
    _, x = O.block_norm(f(d["r"]), w_pre=f(d["w_in"]))
    assert np.abs(f(o["x"]) - x).max() <= 2.0 ** -8 * np.abs(x).max() * 1.01
    xq = f(o["x"])
    lw = O.bf16_bits_to_f64(synth.router_bf16(WL))
    ad = [f(t) for t in d["router_adapters"][:3]]
    logits = O.add_adapters(xq, xq @ lw.T, d["adapter_ids"].cpu().numpy(), *ad)
    assert np.abs(f(o["logits"]) - logits).max() <= 1e-4 * max(1.0, np.abs(logits).max())
    ids, w = O.select_experts(f(o["logits"]), WL.k, score="sigmoid", bias=f(d["rule"].bias), num_groups=4, top_groups=2, group_score="top2", scale=2.5)
    assert np.array_equal(ids, o["ids"].cpu().numpy()) and np.allclose(w, f(o["w"]), rtol=1e-5, atol=0)
    experts = OracleExperts(WL)
    bits = o["x"].view(torch.int16).cpu().numpy().view(np.uint16)
    y = O.moe_forward(bits, ids, f(o["w"]), WL.quant, experts, shared=experts.shared())
    y = O.add_adapters(xq, y, d["adapter_ids"].cpu().numpy(), *[f(t) for t in d["layer_adapters"][:3]])
    rel = np.linalg.norm(f(o["y"]) - y) / np.linalg.norm(y)
    assert rel <= 1e-2 + 2 * 2.0 ** -8
    r2, x2 = O.block_norm(f(d["r"]), y, f(d["w_post"]), f(d["gate"])[:, None], True, f(d["w_next"]), branch_scale=0.7)
    # y's relative error reaches r' through a norm (at most twice) and a gate below one
    assert np.linalg.norm(f(r) - r2) <= 2 * rel * 0.7 * np.linalg.norm(f(d["w_post"])) * np.sqrt(T) + 1e-6 * np.linalg.norm(r2)
    assert np.linalg.norm(f(o["x_next"]) - x2) <= (4 * rel + 2.0 ** -8) * np.linalg.norm(x2)


@pytest.mark.parametrize("T", [2, 30])
def test_captured_and_replayed(layer, T):
    d, o = tensors(T, False, 5), outputs(T)
    r = d["r"].clone()
    run_block(layer, d, o, r)
    layer.sync_status()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.block_forward(r, o["x"], o["y"], o["ids"], o["w"], w_in=d["w_in"], w_post=d["w_post"], w_next=d["w_next"], x_next=o["x_next"],
                            gate=d["gate"], gate_sigmoid=True, logits=o["logits"], adapter_ids=d["adapter_ids"],
                            router_adapters=d["router_adapters"], layer_adapters=d["layer_adapters"], branch_scale=0.7)
    layer.set_decode_path("kernels" if T <= 8 else "auto")       # the path that a capture takes
    for seed in (1, 2):
        fresh = tensors(T, False, seed)["r"]
        r.copy_(fresh)
        g.replay()
        layer.sync_status()
        got = {k: v.clone() for k, v in o.items()}
        r1, r2 = r.clone(), fresh.clone()
        run_block(layer, d, o, r2)
        layer.sync_status()
        assert torch.equal(r1, r2) and all(torch.equal(got[k], o[k]) for k in o)
    layer.set_decode_path("auto")


def test_plain_block_and_refusals(layer):
    """Without rule, adapters, gate or norms the block is route_forward and a
    residual add; bad calls are refused and leave everything as it was."""
    T = 6
    d, o = tensors(T, True, 1), outputs(T)
    layer.set_routing(None)
    o["x"].copy_(d["r"])
    r = d["r"].clone()
    layer.block_forward(r, o["x"], o["y"], o["ids"], o["w"])
    layer.sync_status()
    o2 = outputs(T)
    layer.route_forward(o["x"], o2["ids"], o2["w"], o2["y"])
    layer.sync_status()
    assert torch.equal(o["y"], o2["y"]) and torch.equal(r, d["r"] + o["y"].float())
    r0 = r.clone()
    base = dict(r=r, x=o["x"], y=o["y"], ids=o["ids"], w=o["w"])
    for kw in (dict(x_next=o["x_next"]), dict(w_next=d["w_next"]), dict(y=o["x"]), dict(router_adapters=d["router_adapters"]),
               dict(adapter_ids=d["adapter_ids"], router_adapters=d["layer_adapters"]), dict(eps=-1.0), dict(x=o["x"][:3]),
               dict(r=torch.empty(WL.T + 1, WL.H, device=DEV)), dict(x=o["x"].float())):
        with pytest.raises(moe.MoeError):
            layer.block_forward(**{**base, **kw})
    torch.cuda.synchronize()
    assert torch.equal(r, r0)
