"""Measured cases of the operators around the MoE layer.

  select_experts   logits to expert ids and weights under a routing rule
  add_adapters     low-rank adapters of many requests added beside a projection
  block_norm       norm on a block's output, gate, residual add and the next norm

`run` computes them in elementary torch operations, or with `own` set through
the package's entry points.
"""
import math

import numpy as np
import torch

own = False

LOWEST = torch.finfo(torch.float32).min


def listed():
    return [
        # one decode step of the 512-expert layer: sigmoid scores with a balance bias
        {"name": "select 1 token", "op": "select", "T": 1, "E": 512, "k": 10, "score": "sigmoid", "bias": True, "G": 1, "keep": 1,
         "group": "max", "renorm": True, "scale": 2.5, "draws": "router", "off": 0, "pad": 0},
        # an odd batch, an expert count that is no power of two, some experts switched off
        {"name": "select odd batch", "op": "select", "T": 333, "E": 600, "k": 7, "score": "softmax", "bias": True, "G": 24, "keep": 5,
         "group": "max", "renorm": False, "scale": 16.0, "draws": "router", "off": 37, "pad": 0},
        # a prefill chunk with group-limited routing: the two best experts of a group make its score
        {"name": "select prefill groups", "op": "select", "T": 8192, "E": 512, "k": 10, "score": "sigmoid", "bias": True, "G": 8, "keep": 4,
         "group": "top2", "renorm": True, "scale": 2.5, "draws": "router", "off": 0, "pad": 0},
        # several chunks at once with skewed experts and padded rows behind the last sequence (nothing eligible there)
        {"name": "select long padded", "op": "select", "T": 32768, "E": 1024, "k": 32, "score": "softmax", "bias": False, "G": 1, "keep": 1,
         "group": "max", "renorm": True, "scale": 1.0, "draws": "zipf", "off": 0, "pad": 1500},
        # one decode token with its adapter beside a [H, H] projection
        {"name": "adapters 1 token", "op": "adapters", "T": 1, "K": 2048, "N": 2048, "R": 16, "n": 8, "wide": False, "by": "token", "mixed": False},
        # a decode batch of many requests beside the router's fp32 logits, ranks of their own
        {"name": "adapters decode router", "op": "adapters", "T": 61, "K": 2048, "N": 512, "R": 32, "n": 40, "wide": True, "by": "token", "mixed": True},
        # a prefill chunk of a dozen requests
        {"name": "adapters prefill", "op": "adapters", "T": 4096, "K": 2048, "N": 2048, "R": 16, "n": 12, "wide": False, "by": "request", "mixed": False},
        # the largest chunk at a high rank
        {"name": "adapters prefill rank 64", "op": "adapters", "T": 8192, "K": 2048, "N": 2048, "R": 64, "n": 16, "wide": False, "by": "request", "mixed": False},
        # between two blocks of a decode step
        {"name": "norm 1 token", "op": "norm", "T": 1, "H": 2048, "wide": False, "post": True, "gate": "none", "sigmoid": False, "pre": True, "offset": False},
        # a small odd batch with an element gate and an fp32 residual stream
        {"name": "norm odd batch", "op": "norm", "T": 117, "H": 1368, "wide": True, "post": True, "gate": "element", "sigmoid": True, "pre": True, "offset": True},
        # the prefill chunk of the 2048-wide layer
        {"name": "norm prefill", "op": "norm", "T": 8192, "H": 2048, "wide": False, "post": True, "gate": "token", "sigmoid": True, "pre": True, "offset": False},
        # a wide model's chunk, fp32 residual stream, a learned scale per channel
        {"name": "norm wide", "op": "norm", "T": 4096, "H": 8192, "wide": True, "post": True, "gate": "channel", "sigmoid": False, "pre": True, "offset": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "adapters", "norm"])
    if op == "select":
        T, G = _log(rng, 1, 16384), rng.choice([1, 1, 2, 4, 5, 8, 16, 24])
        per = max(1 + (G == 1) * 7, _log(rng, 8, 1024) // G)
        E = per * G
        keep = rng.randint(1, G)
        k = rng.randint(1, min(32, per * keep))
        return {"op": op, "T": T, "E": E, "k": k, "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.6, "G": G, "keep": keep,
                "group": rng.choice(["max", "top2"]), "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5, 16.0]),
                "draws": rng.choice(["router", "zipf"]), "off": rng.choice([0, 0, E // 10]), "pad": rng.choice([0, 0, T // 5])}
    if op == "adapters":
        decode = rng.random() < 0.5
        return {"op": op, "T": _log(rng, 1, 256) if decode else _log(rng, 257, 8192), "K": 8 * _log(rng, 32, 256), "N": 8 * _log(rng, 16, 256),
                "R": 8 * _log(rng, 1, 8), "n": _log(rng, 1, 64) if decode else _log(rng, 1, 16), "wide": rng.random() < 0.4,
                "by": "token" if decode else "request", "mixed": rng.random() < 0.4}
    return {"op": op, "T": _log(rng, 1, 8192), "H": 8 * _log(rng, 16, 256) if rng.random() < 0.7 else 8 * _log(rng, 256, 512), "wide": rng.random() < 0.4,
            "post": rng.random() < 0.8, "gate": rng.choice(["none", "channel", "token", "element"]), "sigmoid": rng.random() < 0.5,
            "pre": rng.random() < 0.8, "offset": rng.random() < 0.3}


def work(case):
    T = case["T"]
    if case["op"] == "select":
        E = case["E"]
        return {"bytes": T * E * 4 + (E * 4 if case["bias"] else 0) + T * case["k"] * 8, "flops": 10 * T * E}
    if case["op"] == "adapters":
        K, N, R, n = (case[i] for i in "KNRn")
        size = 4 if case["wide"] else 2
        used = n * (1.0 - (1.0 - 1.0 / n) ** T) if case["by"] == "token" else min(n, T)
        return {"bytes": T * (2 * K + 2 * size * N + 4) + used * R * (K + N) * 2, "flops": 2 * T * R * (K + N)}
    H, size = case["H"], 4 if case["wide"] else 2
    row = H * (2 * size + 2 + (2 if case["pre"] else 0) + (2 if case["gate"] == "element" else 0)) + (4 if case["gate"] == "token" else 0)
    return {"bytes": T * row + H * 2 * (int(case["post"]) + int(case["pre"]) + int(case["gate"] == "channel")), "flops": 15 * T * H}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": case}
    T = case["T"]
    if case["op"] == "select":
        E = case["E"]
        if case["draws"] == "zipf":     # experts' popularity by rank^-1.1, Gumbel noise on top
            rank = torch.randperm(E, generator=g, device="cuda").float() + 1.0
            logits = -1.1 * torch.log(rank) - torch.log(-torch.log(uniform(T, E).clamp(1e-20, 1.0 - 1e-7)))
        else:                           # unit activations through a router of 0.02 x 2048 inputs
            logits = normal(T, E) * 0.905
        if case["off"]:
            logits[:, torch.randperm(E, generator=g, device="cuda")[: case["off"]]] = -math.inf
        if case["pad"]:
            logits[T - case["pad"]:] = -math.inf
        s["logits"] = logits
        s["bias"] = normal(E) * 0.05 if case["bias"] else None
        if own:                         # the routing rule is part of the model: made once
            from bit_quantized_mixture_b200 import moe
            s["rule"] = moe.Routing(score=case["score"], bias=s["bias"], num_groups=case["G"], top_groups=case["keep"],
                                    group_score=case["group"], renorm=case["renorm"], scale=case["scale"])
        s["ids"] = torch.empty(T, case["k"], dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, case["k"], dtype=torch.float32, device="cuda")
    elif case["op"] == "adapters":
        K, N, R, n = (case[i] for i in "KNRn")
        s["x"] = normal(T, K).bfloat16()
        y = normal(T, N)
        s["y"] = y if case["wide"] else y.bfloat16()
        s["a"] = (normal(n, R, K) / math.sqrt(K)).bfloat16()
        s["b"] = (normal(n, N, R) / math.sqrt(R)).bfloat16()
        s["scales"] = 0.25 + 1.5 * uniform(n)
        s["ranks"] = torch.randint(1, R + 1, (n,), generator=g, device="cuda", dtype=torch.int32) if case["mixed"] else None
        if case["by"] == "token":       # one token of each request, one in eight without an adapter
            ids = torch.randint(0, n, (T,), generator=g, device="cuda")
            ids = torch.where(uniform(T) < 0.125, -1, ids)
        else:                           # requests one after another, lengths of their own
            cuts = torch.sort(torch.randint(0, T + 1, (n - 1,), generator=g, device="cuda")).values
            ids = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
            ids = torch.randperm(n, generator=g, device="cuda")[ids]
        s["adapter_ids"] = ids.to(torch.int32)
        s["out"] = torch.empty_like(s["y"])
    else:
        H = case["H"]
        r = normal(T, H) * 2.0
        s["r"] = r if case["wide"] else r.bfloat16()
        s["y"] = (normal(T, H) * 0.3).bfloat16()
        base = 0.0 if case["offset"] else 1.0
        s["post_weight"] = (base + 0.1 * normal(H)).bfloat16() if case["post"] else None
        s["pre_weight"] = (base + 0.1 * normal(H)).bfloat16() if case["pre"] else None
        gates = {"none": None, "channel": lambda: normal(H).bfloat16(), "token": lambda: normal(T), "element": lambda: normal(T, H).bfloat16()}
        s["gate"] = gates[case["gate"]]() if case["gate"] != "none" else None
        s["r_out"] = torch.empty_like(s["r"])
        s["x_out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda") if case["pre"] else None
    return s


NORM = {"eps": 1e-6, "branch_scale": 0.7, "residual_scale": 1.0}


def run(s):
    case = s["case"]
    return {"select": _select, "adapters": _adapters, "norm": _norm}[case["op"]](s, case)


def _select(s, c):
    logits, bias = s["logits"], s["bias"]
    if own:
        from bit_quantized_mixture_b200 import moe
        moe.select_experts(logits, c["k"], s["rule"], ids=s["ids"], w=s["w"])
        return s["ids"], s["w"]
    # in 64 bits: which of two near keys is the larger one is not for rounding to say
    ok = logits > LOWEST
    if bias is not None:
        ok = ok & (bias > -math.inf)
    x = logits.double().clamp(max=-LOWEST)
    if c["score"] == "softmax":
        top = torch.where(ok, x, -math.inf).amax(1, keepdim=True)
        p = torch.where(ok, torch.exp(x - top), 0.0)
        total = p.sum(1, keepdim=True)
        score = torch.where(total > 0, p / total, 0.0)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    key = score + bias.double() if bias is not None else score
    by = key if bias is not None else x
    key, by = torch.where(ok, key, -math.inf), torch.where(ok, by, -math.inf)
    T, E = logits.shape
    G = c["G"]
    if G > 1:
        if c["group"] == "max" or E == G:
            of = by.view(T, G, E // G).amax(2)
        else:
            two = torch.topk(key.view(T, G, E // G), 2, dim=2).values
            of = two[..., 0] + torch.where(two[..., 1] > -math.inf, two[..., 1], 0.0)
        best = torch.sort(of, dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=logits.device).scatter_(1, best, True)
        by = torch.where(kept[:, :, None], by.view(T, G, E // G), -math.inf).view(T, E)
    value, ids = torch.sort(by, dim=1, descending=True, stable=True)
    value, ids = value[:, : c["k"]], ids[:, : c["k"]]
    w = torch.where(value > -math.inf, score.gather(1, ids), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _adapters(s, c):
    x, y, a, b, ids, scales, ranks = (s[i] for i in ("x", "y", "a", "b", "adapter_ids", "scales", "ranks"))
    if own:
        from bit_quantized_mixture_b200 import moe
        return moe.add_adapters(x, y, ids, a, b, scales, ranks=ranks, out=s["out"])
    n, R, K = a.shape
    z = (x.float() @ a.float().view(n * R, K).t()).view(-1, n, R)
    mine = torch.where(ids[:, None] == torch.arange(n, device=x.device), scales, 0.0)[:, :, None]
    if ranks is not None:
        mine = torch.where(torch.arange(R, device=x.device) < ranks[:, None], mine, 0.0)
    z = torch.where(mine != 0, z * mine, 0.0).view(-1, n * R)
    delta = z @ b.float().permute(0, 2, 1).reshape(n * R, -1)
    return (y.float() + delta).to(y.dtype)


def _norm(s, c):
    r, y, gate, post, pre = (s[i] for i in ("r", "y", "gate", "post_weight", "pre_weight"))
    if own:
        from bit_quantized_mixture_b200 import moe
        moe.block_norm(r, y, post_weight=post, gate=gate, gate_sigmoid=c["sigmoid"], pre_weight=pre, unit_offset=c["offset"],
                       r_out=s["r_out"], x_out=s["x_out"], **NORM)
        return s["r_out"], s["x_out"]
    off = 1.0 if c["offset"] else 0.0
    u = y.float()
    if post is not None:
        u = u * torch.rsqrt((u * u).mean(1, keepdim=True) + NORM["eps"]) * (post.float() + off)
    if gate is not None:
        g = gate.float()
        g = 1.0 / (1.0 + torch.exp(-g)) if c["sigmoid"] else g
        u = u * (g[:, None] if c["gate"] == "token" else g)
    r2 = NORM["residual_scale"] * r.float() + NORM["branch_scale"] * u
    x = (r2 * torch.rsqrt((r2 * r2).mean(1, keepdim=True) + NORM["eps"]) * (pre.float() + off)).bfloat16() if pre is not None else None
    return r2.to(r.dtype), x


def exact(case, seed):
    s = prepare(case, seed)
    host = {k: v.double().cpu().numpy() if isinstance(v, torch.Tensor) and v.is_floating_point() else v.cpu().numpy() if isinstance(v, torch.Tensor) else v
            for k, v in s.items() if k not in ("ids", "w", "rule", "out", "r_out", "x_out", "case")}
    if case["op"] == "select":
        return _exact_select(case, host["logits"], host["bias"])
    if case["op"] == "adapters":
        out = host["y"].copy()
        for i in range(case["n"]):
            rows = np.nonzero(host["adapter_ids"] == i)[0]
            r = int(host["ranks"][i]) if host["ranks"] is not None else case["R"]
            if rows.size:
                out[rows] += host["scales"][i] * ((host["x"][rows] @ host["a"][i, :r].T) @ host["b"][i, :, :r].T)
        return out
    branch = host["y"]
    if case["post"]:
        branch = branch / np.sqrt((branch ** 2).mean(1) + NORM["eps"])[:, None] * (host["post_weight"] + case["offset"])
    if case["gate"] != "none":
        g = host["gate"] if not case["sigmoid"] else 0.5 * (1.0 + np.tanh(0.5 * host["gate"]))
        branch = branch * (g.reshape(-1, 1) if case["gate"] == "token" else g)
    r = host["r"] * NORM["residual_scale"] + NORM["branch_scale"] * branch
    return r, (r / np.sqrt((r ** 2).mean(1) + NORM["eps"])[:, None] * (host["pre_weight"] + case["offset"]) if case["pre"] else None)


def _exact_select(case, logits, bias):
    T, E = logits.shape
    G, k, rows = case["G"], case["k"], np.arange(T)[:, None]
    live = np.isfinite(logits)
    with np.errstate(all="ignore"):
        if case["score"] == "softmax":
            e = np.exp(logits - np.max(logits, axis=1, keepdims=True), where=live, out=np.zeros_like(logits))
            score = np.divide(e, e.sum(1, keepdims=True), where=live, out=np.zeros_like(e))
        else:
            score = 0.5 * (1.0 + np.tanh(0.5 * logits))
        key = score if bias is None else score + bias
        rank_by = logits if bias is None else key
    key = np.where(live, key, -np.inf)
    rank_by = np.where(live, rank_by, -np.inf)
    if G > 1:
        per = E // G
        ordered = -np.sort(-key.reshape(T, G, per), axis=2)
        value = ordered[:, :, 0].copy()
        if case["group"] == "top2" and per > 1:
            value += np.where(np.isfinite(ordered[:, :, 1]), ordered[:, :, 1], 0.0)
        best = np.argsort(-value, axis=1, kind="stable")[:, : case["keep"]]
        keep = np.zeros((T, G), bool)
        keep[rows, best] = True
        rank_by = np.where(np.repeat(keep, per, axis=1), rank_by, -np.inf)
    ids = np.argsort(-rank_by, axis=1, kind="stable")[:, :k]
    w = np.where(np.isfinite(rank_by[rows, ids]), score[rows, ids], 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, where=total > 0, out=np.zeros_like(w))
    return ids.astype(np.int32), w * case["scale"]
