"""moe_block_norm against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from bit_quantized_mixture_b200 import moe
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(T, H, wide, post, gate, pre, seed=0):
    g = torch.Generator(DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    gates = {"none": lambda: None, "channel": lambda: r(H).bfloat16(), "token": lambda: r(T), "element": lambda: r(T, H).bfloat16()}
    return dict(r=(2 * r(T, H)).to(torch.float32 if wide else torch.bfloat16), y=(0.3 * r(T, H)).bfloat16(),
                post_weight=(1 + 0.1 * r(H)).bfloat16() if post else None, gate=gates[gate](),
                pre_weight=(1 + 0.1 * r(H)).bfloat16() if pre else None)


def oracle(d, sigmoid, offset, **kw):
    g = f64(d["gate"])
    if g is not None and g.ndim == 1 and d["gate"].dtype == torch.float32:
        g = g[:, None]
    return O.block_norm(f64(d["r"]), f64(d["y"]), f64(d["post_weight"]), g, sigmoid, f64(d["pre_weight"]), offset=float(offset), **kw)


def assert_close(got, d, sigmoid, offset, eps=1e-6, branch_scale=1.0, residual_scale=1.0):
    """r': the branch term is a product of five factors, the mean of squares
    (chains of at most 64 + 5 + 32 additions) under a square root, the gate's
    exp and division: (40 + 51) x 2^-24 of its magnitude; the residual term
    and the sum 4 x 2^-24 of theirs.  x: r''s error once in the value and once
    in the mean, the second norm's own 91 x 2^-24, one bf16 rounding."""
    r2, x = oracle(d, sigmoid, offset, eps=eps, branch_scale=branch_scale, residual_scale=residual_scale)
    u = 2.0 ** -24
    base = np.abs(residual_scale * f64(d["r"]))
    err = u * (4 * base + 91 * (np.abs(r2) + base) if d["y"] is not None else 2 * base)
    out_u = 2.0 ** -24 if d["r"].dtype == torch.float32 else 2.0 ** -8
    assert np.all(np.abs(f64(got[0]) - r2) <= err + out_u * (np.abs(r2) + err) + 1e-38)
    if x is None:
        assert got[1] is None
        return
    rms = np.sqrt((r2 * r2).mean(1, keepdims=True) + eps)
    rel = np.sqrt((err ** 2).mean(1, keepdims=True)) / rms
    w = np.abs(f64(d["pre_weight"]) + float(offset))
    ex = err / rms * w + np.abs(x) * (rel + 91 * u)
    assert np.all(np.abs(f64(got[1]) - x) <= ex + 2.0 ** -8 * (np.abs(x) + ex) + 1e-38)


@pytest.mark.parametrize("T,H", [(1, 8), (1, 2048), (3, 24), (7, 256), (5, 1368), (33, 2048), (2, 2056), (9, 4096), (3, 5128), (2, 8192), (4, 8200), (3, 16384),
                                 (700, 128), (1200, 512)])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("gate,sigmoid", [("none", False), ("channel", False), ("token", True), ("element", True)])
def test_matches_the_oracle(T, H, wide, gate, sigmoid):
    d = make(T, H, wide, True, gate, True, seed=T + H)
    offset = gate == "element"
    got = moe.block_norm(gate_sigmoid=sigmoid, unit_offset=offset, branch_scale=0.7, residual_scale=1.25, **d)
    assert_close(got, d, sigmoid, offset, branch_scale=0.7, residual_scale=1.25)


@pytest.mark.parametrize("T,H", [(1, 2048), (6, 640), (300, 1024)])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("post,pre", [(False, False), (False, True), (True, False)])
def test_parts(T, H, wide, gate, post, pre):
    d = make(T, H, wide, post, gate, pre, seed=T)
    got = moe.block_norm(**d)
    assert_close(got, d, False, False)


@pytest.mark.parametrize("T,H", [(1, 512), (50, 2048)])
@pytest.mark.parametrize("wide", [False, True])
def test_norm_alone(T, H, wide):
    """No branch: x = norm(residual_scale r), r' optional."""
    d = make(T, H, wide, False, "none", True, seed=4)
    d["y"] = None
    got = moe.block_norm(**d)
    assert torch.equal(got[0], d["r"])
    assert_close(got, d, False, False)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,H", [(1, 2048), (300, 520), (40, 8192)])
def test_in_place_and_strides(wide, T, H):
    d = make(T, H, wide, True, "element", True, seed=8)
    want = moe.block_norm(**d)
    dt = d["r"].dtype
    rb = torch.full((T + 3, H + 16), 5.0, dtype=dt, device=DEV)
    yb = torch.full((T + 3, H + 24), 6.0, dtype=torch.bfloat16, device=DEV)
    gb = torch.zeros(T, H + 8, dtype=torch.bfloat16, device=DEV)
    r, y, g = rb[:T, 8:8 + H], yb[:T, 16:16 + H], gb[:, 8:]
    r.copy_(d["r"]), y.copy_(d["y"]), g.copy_(d["gate"])
    got = moe.block_norm(r, y, d["post_weight"], g, False, d["pre_weight"], r_out=r, x_out=y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].data_ptr() == r.data_ptr()
    for buf, v, a in ((rb, 5.0, 8), (yb, 6.0, 16)):
        assert torch.all(buf[T:] == v) and torch.all(buf[:, :a] == v) and torch.all(buf[:, a + H:] == v)


def test_extreme_values():
    """Zero rows, tiny rows that eps dominates, large rows, NaN and infinity in
    their own row only, gates that saturate."""
    T, H = 6, 256
    d = make(T, H, True, True, "token", True, seed=1)
    d["y"][0] = 0
    d["r"][0] = 0
    d["y"][1] *= 1e-4
    d["r"][1] *= 1e-6
    d["r"][2] *= 1e15
    d["y"][2] *= 1e15
    d["gate"][:4] = torch.tensor([0.0, 200.0, -200.0, 88.0], device=DEV)
    got = moe.block_norm(gate_sigmoid=True, **d)
    assert_close(got, d, True, False)
    assert torch.all(got[0][0] == 0) and torch.all(got[1][0] == 0)
    d["y"][4, 7] = float("nan")
    d["r"][5, 7] = float("inf")
    bad = moe.block_norm(gate_sigmoid=True, **d)
    assert torch.equal(bad[0][:4], got[0][:4]) and torch.equal(bad[1][:4], got[1][:4])
    assert torch.isnan(bad[0][4]).all() and torch.isnan(bad[1][4].float()).all()
    assert torch.isinf(bad[0][5, 7]) and torch.equal(bad[0][5, :7], got[0][5, :7])


def test_streams_and_graphs():
    d = make(100, 2048, False, True, "token", True, seed=6)
    want = moe.block_norm(gate_sigmoid=True, **d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.block_norm(gate_sigmoid=True, stream=s, **d)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    r_out, x_out = torch.empty_like(want[0]), torch.empty_like(want[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.block_norm(gate_sigmoid=True, r_out=r_out, x_out=x_out, **d)
    d["y"].copy_(d["y"].flip(0))
    d["gate"].copy_(d["gate"].flip(0))
    g.replay()
    want = moe.block_norm(gate_sigmoid=True, **d)
    assert torch.equal(r_out, want[0]) and torch.equal(x_out, want[1])


def test_no_tokens_and_refusals():
    d = make(4, 64, False, True, "channel", True)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    r, x = moe.block_norm(e, e.clone(), pre_weight=d["pre_weight"])
    assert r.shape == x.shape == (0, 64)
    for kw in (dict(y=d["y"].float()), dict(y=d["y"][:3]), dict(r=d["r"].half()), dict(post_weight=d["post_weight"].float()), dict(gate=torch.ones(3, device=DEV)),
               dict(pre_weight=None, x_out=torch.empty_like(d["y"])), dict(r_out=d["y"]), dict(x_out=d["r"]), dict(eps=0.0), dict(r=d["r"].t()),
               dict(r_out=torch.empty(4, 64, device=DEV)), dict(y=None), dict(gate=d["gate"].cpu())):
        with pytest.raises(moe.MoeError):
            moe.block_norm(**{**d, **kw})


def test_vectors_between_an_outputs_rows():
    """A weight that lies between two rows of an output overlaps nothing."""
    T, H = 6, 512
    d = make(T, H, False, True, "channel", True, seed=4)
    want = moe.block_norm(**d)
    big = torch.zeros(T, 2 * H, dtype=torch.bfloat16, device=DEV)
    for row, name in ((0, "post_weight"), (3, "pre_weight"), (5, "gate")):
        big[row, H:] = d[name]
        d[name] = big[row, H:]
    got = moe.block_norm(**d, x_out=big[:, :H])
    assert torch.equal(got[0], want[0]) and torch.equal(big[:, :H], want[1]) and torch.equal(big[3, H:], d["pre_weight"])
    with pytest.raises(moe.MoeError):
        moe.block_norm(**{**d, "pre_weight": big[2, 8:8 + H]}, x_out=big[:, :H])


@pytest.mark.parametrize("T", [4095, 4096])
@pytest.mark.parametrize("H", [8, 520, 2048])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("gate,sigmoid", [("none", False), ("channel", True), ("token", True), ("element", False)])
def test_many_rows(T, H, wide, gate, sigmoid):
    """From 4096 rows on a thread holds four vectors, so that narrow rows are a warp's
    or two; in place as well."""
    d = make(T, H, wide, True, gate, True, seed=T + H)
    got = moe.block_norm(**d, gate_sigmoid=sigmoid)
    assert_close(got, d, sigmoid, False)
    r, y = d["r"].clone(), d["y"].clone()
    moe.block_norm(**{**d, "r": r, "y": y}, gate_sigmoid=sigmoid, r_out=r, x_out=y)
    assert torch.equal(r, got[0]) and torch.equal(y, got[1])
