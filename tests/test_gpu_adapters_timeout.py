"""The adapters' bounded device-side waits give up and report, without a fault: one
CTA of the tcgen05 kernel keeps back an arrival that its cluster waits for (the
library's test hook), the waits run out after a short limit, the kernel ends, every
stream that asks is told, and the next call is correct."""
import pytest
import torch

from bit_quantized_mixture_b200 import moe, synth
from bit_quantized_mixture_b200.layer import build_layer
from tests.test_gpu_adapters import DEV, make

pytestmark = pytest.mark.gpu
SHORT = 2_000_000          # SM cycles: about a millisecond


def call(d, ids, **kw):
    return moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"], **kw)


def fails(fn):
    with pytest.raises(moe.MoeError) as e:
        fn()
    assert e.value.status == moe.MOE_ERR_TIMEOUT and "bounded wait" in str(e.value)


@pytest.mark.parametrize("T,K,N,R,wide", [(3300, 136, 72, 16, False), (3300, 1032, 520, 16, False), (2800, 520, 264, 64, False), (1400, 1032, 520, 128, False),
                                          (7100, 264, 136, 32, True)])
@pytest.mark.parametrize("cta", [0, 5])
def test_withheld_arrival_is_reported_to_every_stream(T, K, N, R, wide, cta):
    d = make(T, K, N, R, 3, seed=1, y_dtype=torch.float32 if wide else torch.bfloat16)
    ids = (torch.arange(T, device=DEV) * 3 // T).to(torch.int32)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    want = call(d, ids)
    torch.cuda.synchronize()
    for stream in (None, s, t):                    # what was given up before this test
        try:
            moe.adapters_status(stream)
        except moe.MoeError:
            pass
    moe.debug_set_adapter_wait_test(cta, SHORT)
    with torch.cuda.stream(s):
        call(d, ids)
    torch.cuda.synchronize()
    fails(lambda: moe.adapters_status(t))          # another stream asks first
    fails(lambda: moe.adapters_status(s))
    fails(lambda: moe.adapters_status())
    for stream in (s, t, None):
        moe.adapters_status(stream)                # told once
    for _ in range(2):                             # the hook was one-shot
        assert torch.equal(call(d, ids), want)
    moe.adapters_status()


def test_a_handles_block_reports_to_its_handle():
    """2800 tokens: the layer's adapters run on the tcgen05 kernel with the handle's error word."""
    T, n, R = 2800, 3, 40
    wl = synth.custom("tiny-int4", T=T, H=256, I=128, E=32, k=4)
    layer, _ = build_layer(wl, 0, max_tokens=T)
    g = torch.Generator(DEV).manual_seed(1)
    r = lambda *shape: torch.randn(*shape, generator=g, device=DEV)
    ad = ((r(n, R, wl.H) / 16).bfloat16(), (0.1 * r(n, wl.H, R)).bfloat16(), torch.ones(n, device=DEV), None)
    x = r(T, wl.H).bfloat16()
    ids = (torch.arange(T, device=DEV) * n // T).to(torch.int32)

    def block():
        o = dict(r=torch.zeros(T, wl.H, device=DEV), x=x, y=torch.empty_like(x), ids=torch.empty(T, wl.k, dtype=torch.int32, device=DEV), w=torch.empty(T, wl.k, device=DEV))
        layer.block_forward(**o, adapter_ids=ids, layer_adapters=ad)
        return o

    want = block()
    layer.sync_status()
    moe.debug_set_adapter_wait_test(0, SHORT)
    block()
    fails(layer.sync_status)
    got = block()
    layer.sync_status()
    assert all(torch.equal(got[k], want[k]) for k in want)
    layer.close()


def test_the_hook_refuses_a_negative_limit():
    with pytest.raises(moe.MoeError) as e:
        moe.debug_set_adapter_wait_test(0, -1)
    assert e.value.status == moe.MOE_ERR_INVALID_ARG
    moe.debug_set_adapter_wait_test(-1)
