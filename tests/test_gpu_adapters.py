"""moe_add_adapters against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from bit_quantized_mixture_b200 import moe
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def make(T, K, N, R, n, seed=0, y_dtype=torch.bfloat16, device=DEV):
    g = torch.Generator(device).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=device)
    return dict(x=r(T, K).bfloat16(), y=r(T, N).to(y_dtype), a=(r(n, R, K) / K ** 0.5).bfloat16(), b=(r(n, N, R) / R ** 0.5).bfloat16(),
                scales=0.5 + torch.rand(n, generator=g, device=device))


def f64(t):
    return t.double().cpu().numpy()


def assert_close(out, d, ids, ranks=None):
    """|out - exact| within the roundings of either path: each z sums K
    products (in chains of at most K/16 + 16 fp32 steps, a step off by at most
    2^-23 of the running magnitude sum |a||x|); z is scaled (2^-24) and held in
    bf16 for bf16 outputs (half a step 2^-8), in three parts for fp32 ones
    (2^-24); the second product sums R terms and the add and the output round
    once more."""
    x, y, a, b, s = (f64(d[i]) for i in ("x", "y", "a", "b", "scales"))
    ids = ids.cpu().numpy()
    rk = None if ranks is None else ranks.cpu().numpy()
    want = O.add_adapters(x, y, ids, a, b, s, rk)
    n, R, K = a.shape
    wide = d["y"].dtype == torch.float32
    u_out, u_z = (2.0 ** -24, 2.0 ** -24) if wide else (2.0 ** -8, 2.0 ** -8)
    got = f64(out)
    for t, i in enumerate(ids):
        r = 0 if i < 0 or i >= n else (R if rk is None else max(0, min(int(rk[i]), R)))
        if r == 0:
            assert np.array_equal(got[t], y[t])
            continue
        ai, bi = a[i][:r], b[i][:, :r]
        zabs = np.abs(s[i]) * (np.abs(ai) @ np.abs(x[t]))
        z = np.abs(s[i] * (ai @ x[t]))
        ez = 2.0 ** -23 * (K / 16 + 16) * zabs + (u_z + 2.0 ** -23) * z
        tol = np.abs(bi) @ ez + 2.0 ** -23 * (r / 16 + 18) * (np.abs(bi) @ z) + 2.0 ** -23 * np.abs(y[t])
        tol = tol + u_out * (np.abs(want[t]) + tol)
        assert np.all(np.abs(got[t] - want[t]) <= tol), (t, np.max(np.abs(got[t] - want[t]) / tol))


SHAPES = [(1, 2048, 2048, 16, 3), (1, 8, 8, 8, 1), (2, 72, 40, 24, 2), (7, 256, 512, 128, 4), (16, 512, 264, 40, 5), (17, 520, 1000, 8, 3),
          (61, 1024, 512, 32, 40), (130, 264, 136, 64, 6), (200, 2048, 256, 16, 11), (333, 136, 72, 56, 2),
          (2113, 136, 72, 24, 7), (2305, 64, 96, 64, 30), (2200, 72, 40, 128, 3), (2049, 520, 264, 96, 4),
          (2801, 136, 72, 24, 7), (2817, 64, 96, 64, 30), (2900, 72, 40, 128, 3), (3000, 520, 264, 96, 4), (2800, 1032, 520, 16, 1), (4001, 128, 64, 8, 2),
          (8200, 72, 104, 40, 3), (2900, 8, 8, 8, 2), (20000, 64, 72, 16, 5), (100, 256, 264, 72, 3), (240, 64, 72, 32, 4), (60, 72, 1000, 128, 2)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("order", ["token", "request"])
def test_matches_the_oracle(shape, wide, order):
    T, K, N, R, n = shape
    d = make(T, K, N, R, n, seed=T + K, y_dtype=torch.float32 if wide else torch.bfloat16)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, n + 1, (T,), generator=g)           # -1 and n: no adapter
    if order == "request":
        ids = ids.sort().values
    ids = ids.to(torch.int32).to(DEV)
    out = moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"])
    assert_close(out, d, ids)


@pytest.mark.parametrize("T,R,wide", [(1499, 72, False), (1500, 72, False), (2299, 64, False), (2300, 40, False), (2799, 32, False), (2800, 8, False),
                                      (3600, 16, True), (3601, 16, True), (3700, 64, True), (3605, 128, True), (8192, 72, True)])
def test_both_sides_of_each_token_count_that_changes_the_kernel(T, R, wide):
    K, N, n = 136, 72, 5
    d = make(T, K, N, R, n, seed=T + R, y_dtype=torch.float32 if wide else torch.bfloat16)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, n, (T,), generator=g).sort().values.to(torch.int32).to(DEV)
    ranks = torch.randint(1, R + 1, (n,), generator=g).to(torch.int32).to(DEV)
    assert_close(moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"], ranks), d, ids, ranks)


@pytest.mark.parametrize("T", [1, 40, 200, 300, 2100, 2900, 8300])
@pytest.mark.parametrize("wide", [False, True])
def test_ranks_of_their_own(T, wide):
    """Unused rows and columns may hold anything, NaN included; a rank beyond R
    counts as R, a negative one as 0."""
    K, N, R, n = 192, 320, 32, 6
    d = make(T, K, N, R, n, seed=7, y_dtype=torch.float32 if wide else torch.bfloat16)
    ranks = torch.tensor([1, 32, 13, 0, 99, -5], dtype=torch.int32, device=DEV)
    for i, r in enumerate([1, 32, 13, 0, 32, 0]):
        d["a"][i, r:] = float("nan")
        d["b"][i, :, r:] = float("nan")
    ids = (torch.arange(T, device=DEV) * 5 % 7 - 1).to(torch.int32)
    out = moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"], ranks=ranks)
    assert_close(out, d, ids, ranks)


@pytest.mark.parametrize("T", [3, 150, 400, 2090, 2830, 8230])
@pytest.mark.parametrize("wide", [False, True])
def test_in_place_strides_and_untouched_rows(T, wide):
    K, N, R, n = 128, 96, 16, 4
    dt = torch.float32 if wide else torch.bfloat16
    d = make(T, K, N, R, n, seed=3, y_dtype=dt)
    ids = (torch.arange(T, device=DEV) % (n + 1) - 1).to(torch.int32)
    want = moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"])
    # x and out side by side in one matrix, rows behind the last token kept
    big = torch.full((T + 5, K + N + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    big[:T, 8:8 + K] = d["x"]
    yb = torch.full((T + 5, N + 24), 3.0, dtype=dt, device=DEV)
    yb[:T, 8:8 + N] = d["y"]
    y = yb[:T, 8:8 + N]
    got = moe.add_adapters(big[:T, 8:8 + K], y, ids, d["a"], d["b"], d["scales"], out=y)
    assert got.data_ptr() == y.data_ptr() and torch.equal(y, want)
    assert torch.all(yb[T:] == 3.0) and torch.all(yb[:, :8] == 3.0) and torch.all(yb[:, 8 + N:] == 3.0)
    if not wide:
        out = big[:T, 8 + K:8 + K + N]
        moe.add_adapters(big[:T, 8:8 + K], d["y"], ids, d["a"], d["b"], d["scales"], out=out)
        assert torch.equal(out, want) and torch.all(big[T:] == 7.0) and torch.all(big[:, 8 + K + N:] == 7.0)


@pytest.mark.parametrize("T", [20, 70, 300, 2070, 2870])
def test_special_values_stay_with_their_token(T):
    """A token's NaN or infinity reaches its own row only; tokens without an
    adapter keep every bit."""
    K, N, R, n = 64, 64, 8, 3
    d = make(T, K, N, R, n, seed=11)
    ids = (torch.arange(T, device=DEV) % 4 - 1).to(torch.int32)
    clean = moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"])
    d["x"][5] = float("nan")
    d["x"][6, 3] = float("inf")
    d["x"][8] = float("nan")                       # ids[8] = -1
    out = moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"])
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[5] = keep[6] = False
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[5].float()).all() and not torch.isfinite(out[6].float()).any()


@pytest.mark.parametrize("T", [30, 100, 280, 2080, 2880])
def test_special_weights_stay_with_their_adapter(T):
    """An adapter whose weights are not finite spoils its own tokens only."""
    K, N, R, n = 96, 64, 16, 4
    d = make(T, K, N, R, n, seed=12)
    ids = (torch.arange(T, device=DEV) * 3 % 5 - 1).to(torch.int32)
    clean = moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"])
    d["a"][1, 2, 5] = float("inf")
    d["b"][2, 7, 3] = float("nan")
    d["scales"][3] = float("nan")
    out = moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"])
    for i in (-1, 0):
        assert torch.equal(out[ids == i], clean[ids == i])
    bad = ~torch.isfinite(out.float())
    assert bad[ids == 1].any() and bad[ids == 2][:, 7].all() and not bad[ids == 2][:, :7].any() and bad[ids == 3].all()


@pytest.mark.parametrize("T", [150, 700, 4100])
def test_repeats_bit_for_bit_on_streams_and_graphs(T):
    K, N, R, n = 512, 512, 16, 5
    d = make(T, K, N, R, n, seed=2)
    ids = (torch.arange(T, device=DEV) * 5 // T - 1).to(torch.int32)
    want = moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"], out=out)
    d["x"].copy_(d["x"].flip(0))
    ids.copy_(ids.flip(0))
    g.replay()
    assert torch.equal(out, moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"]))


@pytest.mark.parametrize("T", [5, 300, 2900])
def test_no_adapter_at_all(T):
    d = make(T, 256, 192, 16, 2, seed=1)
    ids = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    assert torch.equal(moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"]), d["y"])


def test_many_runs_agree():
    """The same call many times, with other calls between: every run the same bits."""
    a = make(4096, 2048, 512, 16, 12, seed=5)
    b = make(8192, 640, 520, 64, 3, seed=6, y_dtype=torch.float32)
    ida = (torch.arange(4096, device=DEV) * 13 // 4096 - 1).to(torch.int32)
    idb = torch.randint(-1, 3, (8192,), generator=torch.Generator(DEV).manual_seed(1), device=DEV).to(torch.int32)
    run = lambda d, i: moe.add_adapters(d["x"], d["y"], i, d["a"], d["b"], d["scales"])
    wa, wb = run(a, ida), run(b, idb)
    for _ in range(40):
        ga, gb = run(a, ida), run(b, idb)
        assert torch.equal(ga, wa) and torch.equal(gb, wb)


@pytest.mark.parametrize("T", [200, 1000, 5000])
def test_two_streams_at_once(T):
    a, b = make(T, 512, 768, 16, 4, seed=1), make(T, 256, 1024, 64, 3, seed=2, y_dtype=torch.float32)
    ia, ib = ((torch.arange(T, device=DEV) * q // T - 1).to(torch.int32) for q in (5, 4))
    run = lambda d, i, **kw: moe.add_adapters(d["x"], d["y"], i, d["a"], d["b"], d["scales"], **kw)
    wa, wb = run(a, ia), run(b, ib)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(run(a, ia, stream=s), run(b, ib, stream=t)) for _ in range(10)]
    torch.cuda.synchronize()
    moe.adapters_status()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in got)


def test_no_tokens():
    d = make(1, 64, 64, 8, 2)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    out = moe.add_adapters(e, e.clone(), torch.empty(0, dtype=torch.int32, device=DEV), d["a"], d["b"], d["scales"])
    assert out.shape == (0, 64)


def test_refusals():
    d = make(4, 64, 64, 8, 2)
    ids = torch.zeros(4, dtype=torch.int32, device=DEV)
    call = lambda **kw: moe.add_adapters(**{**dict(x=d["x"], y=d["y"], adapter_ids=ids, a=d["a"], b=d["b"], scales=d["scales"]), **kw})
    for kw in (dict(x=d["x"].float()), dict(x=d["x"].t()), dict(y=d["y"].half()), dict(y=d["y"][:3]), dict(adapter_ids=ids.long()),
               dict(a=d["a"][:, :, :32].contiguous()), dict(b=d["b"].transpose(1, 2)), dict(scales=d["scales"][:1]), dict(out=d["x"]),
               dict(out=torch.empty(4, 64, device=DEV)), dict(ranks=torch.ones(3, dtype=torch.int32, device=DEV)), dict(y=d["y"].cpu()),
               dict(a=d["a"][:, :4].contiguous(), b=d["b"][:, :, :4].contiguous())):
        with pytest.raises(moe.MoeError):
            call(**kw)
