"""Measured cases of the operators around 8-bit products and expert routing.

A mixture-of-experts layer that serves with 8-bit weights runs them in this
order: moe_route picks each token's experts from the router's logits (and
moe_route_backward carries the gradient of their weights back when the router
is trained), moe_plan sorts the (token, expert) pairs by expert, i8_quant turns
activations into 8-bit codes with one scale per row, and i8_grouped_gemm
multiplies each expert's rows with that expert's weights.  i8_gemm is the same
product without experts (attention projections, dense layers, the output head).

``run`` computes an operator in plain torch operations (``own`` false) or
through the framework (``own`` true).
"""
import math

import numpy as np
import torch

own = False

MAX_EXPERTS = 256
MAX_K = 131056          # 8-bit products: 2^14 * K stays below 2^31
TINY = 2.0 ** -126      # the smallest sum of weights that is divided by as it is
QUANT_FLOOR = 2.0 ** -100   # the smallest row maximum that scales are made from

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_ES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # One step of a small decode batch: four tokens through a router with
        # balance biases and expert groups; nothing but latency.
        _route("route_decode", 4, 256, 8, "f32", "sigmoid", True, 8, 4, "top2", 0.0),
        # A packed prompt batch of an odd length with 1% padding tokens (all
        # logits masked), softmax scores in the model's 16-bit type.
        _route("route_prompt", 16381, 128, 8, "bf16", "softmax", False, 1, 1, "max", 0.01),
        # The router's gradient over one training micro-batch.
        {"name": "route_grad", "op": "route_grad", "T": 16384, "E": 256, "k": 8,
         "dtype": "f32", "score": "sigmoid", "renorm": True},
        # The plan of a decode batch: 256 pairs.
        {"name": "plan_decode", "op": "plan", "T": 32, "E": 128, "k": 8, "pad": 0.0},
        # The plan of a long prompt batch with padding tokens.
        {"name": "plan_prompt", "op": "plan", "T": 16384, "E": 256, "k": 8, "pad": 0.01},
        # Decode activations of an odd width.
        {"name": "quant_decode", "op": "quant", "R": 7, "K": 5003, "dtype": "f16"},
        # The activations of a prompt batch.
        {"name": "quant_prompt", "op": "quant", "R": 16384, "K": 8192, "dtype": "bf16"},
        # One token through a square projection: the weights are read once.
        {"name": "gemm_token", "op": "gemm", "M": 1, "N": 8192, "K": 8192, "d": "bf16"},
        # A few hundred tokens, every size ragged.
        {"name": "gemm_ragged", "op": "gemm", "M": 333, "N": 4104, "K": 4112, "d": "f16"},
        # The repository's headline size.
        {"name": "gemm_prompt", "op": "gemm", "M": 8192, "N": 8192, "K": 8192, "d": "bf16"},
        # Decode through 64 experts: about four rows each, bound by the weights.
        {"name": "grouped_decode", "op": "grouped", "T": 64, "E": 64, "k": 4, "N": 2048,
         "K": 2048, "d": "bf16"},
        # A prompt through 32 experts of uneven load.
        {"name": "grouped_prompt", "op": "grouped", "T": 8192, "E": 32, "k": 4, "N": 4096,
         "K": 2048, "d": "bf16"},
    ]


def _route(name, T, E, k, dtype, score, bias, groups, top_groups, group_score, pad):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "dtype": dtype,
            "score": score, "bias": bias, "groups": groups, "top_groups": top_groups,
            "group_score": group_score, "renorm": True, "scale": 1.0, "pad": pad}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "plan", "quant", "gemm", "grouped"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(1, _log(rng, 8, MAX_EXPERTS) // groups)
        top_groups = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(16, top_groups * (E // groups)))
        c = _route("", _log(rng, 1, 16384), E, k, rng.choice(["f32", "bf16", "f16"]),
                   rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups, top_groups,
                   rng.choice(["max", "top2"]), rng.choice([0.0, 0.02]))
        c["renorm"] = rng.random() < 0.7
        c["scale"] = rng.choice([1.0, 2.5])
        del c["name"]
        return c
    if op == "route_grad":
        E = _log(rng, 8, MAX_EXPERTS)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(16, E)),
                "dtype": rng.choice(["f32", "bf16", "f16"]),
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.7}
    if op == "plan":
        E = _log(rng, 8, MAX_EXPERTS)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E)),
                "pad": rng.choice([0.0, 0.02])}
    if op == "quant":
        R = _log(rng, 1, 16384)
        return {"op": op, "R": R, "K": _log(rng, 64, min(32768, (1 << 27) // R)),
                "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op == "gemm":
        M = _log(rng, 1, 8192)
        N = 8 * _log(rng, 16, 2048)
        K = 16 * _log(rng, 16, max(17, min(1024, (1 << 39) // (16 * M * N))))
        return {"op": op, "M": M, "N": N, "K": K, "d": rng.choice(["f32", "bf16", "f16"])}
    E = _log(rng, 8, 128)
    k = rng.randint(1, min(8, E))
    N = 8 * _log(rng, 32, 512)
    K = 16 * _log(rng, 32, 192)
    T = _log(rng, 1, max(2, min(8192, (1 << 38) // (k * N * K), (1 << 27) // (k * max(N, K)))))
    return {"op": op, "T": T, "E": E, "k": k, "N": N, "K": K,
            "d": rng.choice(["f32", "bf16", "f16"])}


# ------------------------------------------------------------------ the inputs

def _codes(gen, *shape):
    """8-bit codes as quantised normal values have them: the row maximum, at
    about four standard deviations, has the code 127."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    return x.mul_(32).round_().clamp_(-127, 127).to(torch.int8)


def _scales(gen, *shape):
    return 0.01 + 0.02 * torch.rand(shape, generator=gen, device="cuda")


def _logits(gen, T, E, pad):
    """Router logits: experts of uneven popularity, padding tokens masked."""
    x = torch.randn((T, E), generator=gen, device="cuda")
    x += 0.5 * torch.randn((1, E), generator=gen, device="cuda")
    if pad:
        x[torch.rand((T,), generator=gen, device="cuda") < pad] = -math.inf
    return x


def _ids(gen, T, E, k, pad):
    """Each token's k experts as a router gives them; -1 for padding tokens."""
    x = _logits(gen, T, E, pad)
    ids = x.topk(k, 1).indices.to(torch.int32)
    return torch.where(x[:, :1] == -math.inf, -1, ids).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "route":
        s["logits"] = _logits(gen, case["T"], case["E"], case["pad"]).to(_DT[case["dtype"]])
        s["b"] = (0.1 * torch.randn(case["E"], generator=gen, device="cuda")
                  if case["bias"] else None)
    elif op == "route_grad":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _logits(gen, T, E, 0.0).to(_DT[case["dtype"]])
        s["ids"] = s["logits"].float().topk(k, 1).indices.to(torch.int32)
        s["dweights"] = torch.randn((T, k), generator=gen, device="cuda")
    elif op == "plan":
        s["ids"] = _ids(gen, case["T"], case["E"], case["k"], case["pad"])
    elif op == "quant":
        x = torch.randn((case["R"], case["K"]), generator=gen, device="cuda")
        x *= torch.exp(torch.randn((case["R"], 1), generator=gen, device="cuda"))
        s["x"] = x.to(_DT[case["dtype"]])
        s["c127"] = torch.full((), 127.0, device="cuda")
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["sa"] = _codes(gen, M, K), _scales(gen, M)
        s["b"], s["sb"] = _codes(gen, N, K), _scales(gen, N)
    elif op == "grouped":
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        ids = _ids(gen, T, E, k, 0.0).reshape(-1).long()
        order = ids.sort(stable=True).indices
        counts = torch.bincount(ids, minlength=E)
        s["rows"] = torch.div(order, k, rounding_mode="floor").to(torch.int32)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["cap"] = int(counts.max())
        s["a"], s["sa"] = _codes(gen, T, K), _scales(gen, T)
        s["b"], s["sb"] = _codes(gen, E, N, K), _scales(gen, E, N)
    return s


# ------------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_route(s):
    import dense_gemm_swizzled_amd as sg
    return sg.moe_route(s["logits"], s["k"], score=s["score"], bias=s["b"],
                        n_groups=s["groups"], top_groups=s["top_groups"],
                        group_score=s["group_score"], renorm=s["renorm"], scale=s["scale"])


def _own_route_grad(s):
    import dense_gemm_swizzled_amd as sg
    return sg.moe_route_backward(s["dweights"], s["logits"], s["ids"], score=s["score"],
                                 renorm=s["renorm"])


def _own_plan(s):
    import dense_gemm_swizzled_amd as sg
    return sg.moe_plan(s["ids"], s["E"])


def _own_quant(s):
    import dense_gemm_swizzled_amd as sg
    return sg.i8_quant(s["x"])


def _own_gemm(s):
    import dense_gemm_swizzled_amd as sg
    return sg.i8_gemm(s["a"], s["sa"], s["b"], s["sb"], out_dtype=_DT[s["d"]])


def _own_grouped(s):
    import dense_gemm_swizzled_amd as sg
    return sg.i8_grouped_gemm(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], rows=s["rows"],
                              out_dtype=_DT[s["d"]])


_own = {"route": _own_route, "route_grad": _own_route_grad, "plan": _own_plan,
        "quant": _own_quant, "gemm": _own_gemm, "grouped": _own_grouped}


def _scores(x, score):
    """The experts' scores in x's type; masked logits (-inf, NaN) score zero."""
    live = x > -math.inf
    if score == "sigmoid":
        return torch.where(live, 1 / (1 + torch.exp(-x)), 0)
    top = torch.where(live, x, -math.inf).amax(1, keepdim=True)
    e = torch.where(live, torch.exp(x - top), 0)
    return e / e.sum(1, keepdim=True).clamp_min(TINY)


def _weights(s, ids, renorm, scale):
    """The chosen experts' weights from all scores s; zero where the id is -1."""
    w = torch.where(ids >= 0, s.gather(1, ids.clamp_min(0)), 0)
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp_min(TINY)
    return w * scale


def _plain_route(s):
    x = s["logits"]
    T, E = x.shape
    # Which experts: by logit, or, where a bias or sums of scores enter, by
    # score + bias in 64 bits (32 bits would order close scores by rounding).
    live = x > -math.inf
    if s["b"] is None and (s["groups"] == 1 or s["group_score"] == "max"):
        key = x.float()
    else:
        key = _scores(x.double(), s["score"])
        if s["b"] is not None:
            key = key + s["b"].double()
    key = torch.where(live & (key > -math.inf), key, -math.inf)
    if s["groups"] > 1:
        g = key.reshape(T, s["groups"], E // s["groups"])
        best = g.sort(dim=2, descending=True).values[:, :, :2]
        if s["group_score"] == "top2" and best.shape[2] > 1:
            gs = best[:, :, 0] + torch.where(best[:, :, 1] > -math.inf, best[:, :, 1], 0)
        else:
            gs = best[:, :, 0]
        top = gs.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, top, True)
        key = torch.where(keep[:, :, None], g, -math.inf).reshape(T, E)
    order = key.sort(dim=1, descending=True, stable=True)
    ids = torch.where(order.values > -math.inf, order.indices, -1)[:, :s["k"]]
    w = _weights(_scores(x.float(), s["score"]), ids, s["renorm"], s["scale"])
    return w, ids.to(torch.int32)


def _plain_route_grad(s):
    # w_j = s_j / S (S the sum of the chosen s), or s_j; then the scores' own
    # derivative: s (1 - s) for sigmoid, s_e (ds_e - sum s ds) for softmax.
    x, ids, g = s["logits"].float(), s["ids"].long(), s["dweights"]
    p = _scores(x, s["score"])
    w = p.gather(1, ids)
    if s["renorm"]:
        tot = w.sum(1, keepdim=True).clamp_min(TINY)
        d = (g - (g * w).sum(1, keepdim=True) / tot) / tot
    else:
        d = g
    full = torch.zeros_like(x).scatter_add_(1, ids, d)
    if s["score"] == "sigmoid":
        dx = full * p * (1 - p)
    else:
        dx = p * (full - (full * p).sum(1, keepdim=True))
    return dx.to(s["logits"].dtype)


def _plain_plan(s):
    ids, E, k = s["ids"], s["E"], s["k"]
    flat = ids.reshape(-1)
    live = (flat >= 0) & (flat < E)
    key = torch.where(live, flat, E)
    srt = key.sort(stable=True)
    edges = torch.arange(E + 1, device=key.device, dtype=key.dtype)
    offsets = torch.searchsorted(srt.values, edges).to(torch.int32)
    rows = torch.where(srt.values < E, torch.div(srt.indices, k, rounding_mode="floor"), -1)
    place = torch.empty_like(srt.indices)
    place[srt.indices] = torch.arange(flat.numel(), device=key.device)
    slots = torch.where(live, place, -1).reshape(ids.shape)
    return offsets, rows.to(torch.int32), slots.to(torch.int32)


def _plain_quant(s):
    # The codes are defined by these 32-bit steps, each rounded to nearest
    # even, so they are whole numbers that two implementations share exactly.
    # (A tensor divisor: a number would be multiplied by its reciprocal.)
    x = s["x"].float()
    a = x.abs().amax(1, keepdim=True)
    a = torch.where(a < math.inf, a.clamp_min(QUANT_FLOOR), math.nan)
    q = torch.nan_to_num((x * torch.div(s["c127"], a)).round(), nan=0.0).to(torch.int8)
    K = x.shape[1]
    q = torch.nn.functional.pad(q, (0, -K % 16))
    return q, torch.div(a, s["c127"]).reshape(-1)


def _plain_gemm(s):
    acc = s["a"].float() @ s["b"].float().t()
    return (acc * s["sa"][:, None] * s["sb"][None, :]).to(_DT[s["d"]])


def _plain_grouped(s):
    # Each expert's rows padded to the largest load, one batched product.
    R, E = s["rows"].numel(), s["E"]
    at = torch.arange(R, device="cuda", dtype=torch.int32)
    e = torch.searchsorted(s["offsets"][1:], at, right=True)
    pos = at - s["offsets"][e]
    rows = s["rows"].long()
    a = torch.zeros((E, s["cap"], s["K"]), device="cuda")
    a[e, pos] = s["a"][rows].float()
    acc = torch.bmm(a, s["b"].float().transpose(1, 2).contiguous())[e, pos]
    return (acc * s["sa"][rows][:, None] * s["sb"][e]).to(_DT[s["d"]])


_plain = {"route": _plain_route, "route_grad": _plain_route_grad, "plan": _plain_plan,
          "quant": _plain_quant, "gemm": _plain_gemm, "grouped": _plain_grouped}


# ------------------------------------------------------------------- the floor

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * _ES[case["dtype"]] + 8 * T * k + 4 * E * case["bias"],
                "flops": 8 * T * E}
    if op == "route_grad":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 2 * T * E * _ES[case["dtype"]] + 8 * T * k, "flops": 8 * T * E}
    if op == "plan":
        P = case["T"] * case["k"]
        return {"bytes": 12 * P + 4 * (case["E"] + 1), "flops": 0}
    if op == "quant":
        R, K = case["R"], case["K"]
        return {"bytes": R * K * _ES[case["dtype"]] + R * (K + -K % 16) + 4 * R,
                "flops": 3 * R * K}
    es = _ES[case["d"]]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K + 4) + M * N * es, "flops": 2 * M * N * K}
    # The experts that some token has chosen: their weights are read once.
    P, E, N, K = case["T"] * case["k"], case["E"], case["N"], case["K"]
    return {"bytes": case["T"] * (K + 4) + min(P, E) * N * (K + 4) + P * (N * es + 4),
            "flops": 2 * P * N * K}


# ----------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "route_grad":
        return _exact_route_grad(s)
    if op == "quant":
        x = s["x"].double().cpu().numpy()
        return None, np.maximum(np.abs(x).max(1), QUANT_FLOOR) / 127
    if op == "gemm":
        acc = torch.einsum("mk,nk->mn", s["a"].double(), s["b"].double())
        return torch.outer(s["sa"].double(), s["sb"].double()) * acc
    if op == "grouped":
        out = []
        off = s["offsets"].tolist()
        for e in range(s["E"]):
            r = s["rows"][off[e]:off[e + 1]].long()
            out.append((s["sa"][r].double()[:, None] * s["a"][r].double())
                       @ (s["sb"][e].double()[:, None] * s["b"][e].double()).t())
        return torch.cat(out)
    return None     # a plan holds whole numbers only


def _exact_route(s):
    """Token by token over numpy arrays: the scores, then the experts that
    the pass returns, in the definition's order."""
    x = s["logits"].double().cpu().numpy()
    T, E = x.shape
    k, G = s["k"], s["groups"]
    with np.errstate(over="ignore", invalid="ignore"):
        if s["score"] == "sigmoid":
            p = np.where(x > -np.inf, 1 / (1 + np.exp(-x)), 0.0)
        else:
            m = x.max(1, keepdims=True)
            e = np.exp(np.where(m > -np.inf, x - m, -np.inf))
            p = e / np.maximum(e.sum(1, keepdims=True), TINY)
    b = np.zeros(E) if s["b"] is None else s["b"].double().cpu().numpy()
    by_logit = s["b"] is None and (G == 1 or s["group_score"] == "max")
    w = np.zeros((T, k))
    for t in range(T):
        key = x[t].copy() if by_logit else np.where(x[t] > -np.inf, p[t] + b, -np.inf)
        if G > 1:
            parts = key.reshape(G, E // G)
            best = -np.sort(-parts, 1)
            gs = best[:, 0].copy()
            if s["group_score"] == "top2" and E // G > 1:
                gs += np.where(best[:, 1] > -np.inf, best[:, 1], 0)
            drop = np.lexsort((np.arange(G), -gs))[s["top_groups"]:]
            parts[drop] = -np.inf
        chosen = np.argsort(-key, kind="stable")[:k]
        v = np.where(key[chosen] > -np.inf, p[t, chosen], 0.0)
        if s["renorm"]:
            v = v / max(v.sum(), TINY)
        w[t] = v * s["scale"]
    return w, None


def _exact_route_grad(s):
    """By automatic differentiation in 64 bits."""
    x = s["logits"].double().cpu().requires_grad_()
    p = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.softmax(x, 1)
    w = p.gather(1, s["ids"].long().cpu())
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    (w * s["dweights"].double().cpu()).sum().backward()
    return x.grad
