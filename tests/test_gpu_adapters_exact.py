"""moe_add_adapters, the same in each of its kernels: infinities, values at the
ends of fp32, and how exactly the second product's operand is held."""
import numpy as np
import pytest
import torch

from bit_quantized_mixture_b200 import moe
from oracle import moe_oracle as O
from tests.test_gpu_adapters import DEV, assert_close, f64, make

pytestmark = pytest.mark.gpu

# tokens and rank of each kernel: a cluster per token, tiles of 16, tiles of 64
# (fp32 outputs), tcgen05 with its ranks up to 64 and up to 128
SIZES = [(20, 8), (300, 16), (700, 128), (1600, 128), (2900, 16), (3700, 16), (3700, 72), (8300, 64)]


def oracle(d, ids, ranks=None):
    with np.errstate(all="ignore"):
        return O.add_adapters(*(f64(d[i]) for i in ("x", "y")), ids.cpu().numpy(), *(f64(d[i]) for i in ("a", "b", "scales")),
                              None if ranks is None else ranks.cpu().numpy())


def same_kind(out, want):
    """Finite where the exact value is, the same infinity, NaN where it is none."""
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isposinf(got), np.isposinf(want)) and \
        np.array_equal(np.isneginf(got), np.isneginf(want))


@pytest.mark.parametrize("T,R", SIZES)
@pytest.mark.parametrize("wide", [False, True])
def test_infinities_are_those_of_the_formula(T, R, wide):
    """An infinite z gives infinities with the signs of its weights, an infinite
    weight those of its z, whatever the other ranks hold."""
    K, N, n = 64, 72, 3
    d = make(T, K, N, R, n, seed=T, y_dtype=torch.float32 if wide else torch.bfloat16)
    ids = (torch.arange(T, device=DEV) % 4 - 1).to(torch.int32)
    d["x"][6, 3] = float("inf")                 # ids[6] = 1
    d["x"][13, 5] = -float("inf")               # ids[13] = 0
    d["x"][11] *= 2.0 ** -115                   # ids[11] = 2: a z far below one
    d["b"][2, 7, 0] = float("inf")
    d["b"][2, 70, R - 1] = -float("inf")
    one = torch.ones(n, dtype=torch.int32, device=DEV)      # one rank in use: z is that infinity alone
    for ranks in (one, None):
        same_kind(moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"], ranks), oracle(d, ids, ranks))


@pytest.mark.parametrize("T,R", SIZES)
@pytest.mark.parametrize("wide", [False, True])
def test_z_at_the_end_of_fp32(T, R, wide):
    """z between the largest finite bf16 and the largest finite fp32 stays finite."""
    K, N, n = 64, 72, 2
    d = make(T, K, N, R, n, seed=T + 1, y_dtype=torch.float32 if wide else torch.bfloat16)
    ids = torch.zeros(T, dtype=torch.int32, device=DEV)
    top = torch.finfo(torch.bfloat16).max
    d["a"].zero_()
    d["a"][:, 0, 0] = 1.0
    d["x"][:, 0] = top
    d["scales"][:] = 1.0 + 2.0 ** -9            # z = bf16's largest x (1 + 2^-9): below 2^128 (1 - 2^-24)
    d["b"][:, :, 0] = 0.5
    out = f64(moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"]))
    want = 0.5 * top * (1.0 + 2.0 ** -9)
    # z and its product with 0.5 are exact up to z's own rounding (2^-24); the output's half step
    assert np.all(np.abs(out - want) <= (2.0 ** -23 + (2.0 ** -24 if wide else 2.0 ** -8)) * want)


@pytest.mark.parametrize("T,R", SIZES + [(1600, 72), (2310, 64), (2000, 40)])
@pytest.mark.parametrize("wide", [False, True])
def test_z_is_held_in_fp32_for_either_output(T, R, wide):
    """Outputs that nearly cancel, y = -delta rounded, show every rounding before
    the last.  z sums K products (chains of at most K/16 + 16 fp32 steps, each off
    by at most 2^-23 of the running magnitude), is scaled (2^-24) and held in 24
    bits; the second product sums R terms in three parts (3 R/16 + 18 steps), y is
    added (2^-23) and the output rounded (half a step)."""
    K, N, n = 64, 72, 3
    d = make(T, K, N, R, n, seed=2 * T + R, y_dtype=torch.float32 if wide else torch.bfloat16)
    ids = (torch.arange(T, device=DEV) * n // T).to(torch.int32)
    x, a, b, s = (f64(d[i]) for i in ("x", "a", "b", "scales"))
    own = ids.cpu().numpy()
    z = s[own][:, None] * np.einsum("tk,trk->tr", x, a[own])
    delta = np.einsum("tr,tnr->tn", z, b[own])
    d["y"] = torch.from_numpy(-delta).to(DEV).to(d["y"].dtype)
    y = f64(d["y"])
    got = f64(moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"]))
    zabs = np.abs(s[own])[:, None] * np.einsum("tk,trk->tr", np.abs(x), np.abs(a[own]))
    ez = 2.0 ** -23 * (K / 16 + 16) * zabs + 2.0 ** -23 * np.abs(z)
    tol = np.einsum("tr,tnr->tn", ez + 2.0 ** -23 * (3 * R / 16 + 18) * np.abs(z), np.abs(b[own])) + 2.0 ** -23 * np.abs(y)
    tol += (2.0 ** -24 if wide else 2.0 ** -8) * (np.abs(y + delta) + tol)
    assert np.all(np.abs(got - (y + delta)) <= tol), np.max(np.abs(got - (y + delta)) / tol)


@pytest.mark.parametrize("T,R,wide", [(1399, 72, False), (1400, 128, False), (2699, 64, False), (2700, 40, False), (2799, 16, False), (2800, 8, False),
                                      (3499, 24, False), (3500, 32, False), (3999, 16, True), (4000, 32, True), (4999, 16, True), (5000, 8, True),
                                      (6999, 32, True), (7000, 24, True), (4999, 64, True), (5000, 40, True), (3599, 72, True), (3600, 128, True)])
def test_both_sides_of_each_token_count_that_changes_the_kernel(T, R, wide):
    K, N, n = 136, 72, 5
    d = make(T, K, N, R, n, seed=T + R, y_dtype=torch.float32 if wide else torch.bfloat16)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, n, (T,), generator=g).sort().values.to(torch.int32).to(DEV)
    ranks = torch.randint(1, R + 1, (n,), generator=g).to(torch.int32).to(DEV)
    assert_close(moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"], ranks), d, ids, ranks)


@pytest.mark.parametrize("T,K,N,R,n", [(1400, 1032, 1000, 128, 5), (1500, 520, 1000, 96, 40), (1900, 520, 520, 72, 30), (1920, 2048, 512, 128, 1)])
@pytest.mark.parametrize("order", ["token", "request"])
@pytest.mark.parametrize("mixed", [False, True])
def test_few_tiles_in_clusters_of_eight(T, K, N, R, n, order, mixed):
    """Up to 15 tiles of 128 tokens, each split over eight CTAs (K and N have eight
    chunks): 16 rows of a tile per CTA."""
    d = make(T, K, N, R, n, seed=T + R)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, n, (T,), generator=g)
    if order == "request":
        ids = ids.sort().values
    ids = ids.to(torch.int32).to(DEV)
    ranks = torch.randint(0, R + 1, (n,), generator=g).to(torch.int32).to(DEV) if mixed else None
    assert_close(moe.add_adapters(d["x"], d["y"], ids, d["a"], d["b"], d["scales"], ranks), d, ids, ranks)
