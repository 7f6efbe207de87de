"""Measured cases of the losses of a language model with routed experts.

A training step ends in them: gemm_xent multiplies the last hidden states with
the output head and takes the softmax cross entropy over the vocabulary without
keeping the logits, gemm_xent_backward returns the gradients of the hidden
states and of the head; moe_balance measures how evenly a router spreads its
tokens over the experts, moe_balance_backward returns the gradient of its
logits.  Scoring a few tokens (perplexity, log probabilities of a prompt) runs
gemm_xent alone.

``run`` computes an operator in plain torch operations (``own`` false) or
through the framework (``own`` true).
"""
import math

import torch

own = False

TINY = 2.0 ** -126      # the smallest sum of scores that is divided by as it is
IGNORE = -100           # a target outside the vocabulary: the token has no loss

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_ES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # Four tokens scored against a vocabulary: the head is read once.
        _xent("xent_score", 4, 32768, 2048, "bf16", 1.0),
        # An evaluation batch, every size ragged, scaled logits.
        _xent("xent_eval", 333, 50003, 1032, "f16", 0.5),
        # A training micro-batch at a large vocabulary.
        _xent("xent_train", 8192, 131072, 4096, "bf16", 1.0),
        # The gradients of a small fine-tuning batch.
        _xent_grad("xent_grad_tune", 64, 8192, 1024, "bf16", 1.0, False),
        # Ragged sizes, a penalty on the logarithm of the softmax's divisor.
        _xent_grad("xent_grad_ragged", 1021, 32003, 2056, "f16", 1.0, True),
        # The gradients of a training micro-batch.
        _xent_grad("xent_grad_train", 8192, 65536, 4096, "bf16", 1.0, False),
        # A router over a handful of tokens: nothing but latency.
        _balance("balance", "balance_few", 37, 64, 4, "f32", "softmax", 0.0),
        # A training micro-batch through a router with sigmoid scores.
        _balance("balance", "balance_train", 16384, 256, 8, "f32", "sigmoid", 0.0),
        # Long sequences in the model's 16-bit type, 1% padding tokens.
        _balance("balance", "balance_long", 65521, 128, 8, "bf16", "softmax", 0.01),
        # The gradients of the same three.
        _balance("balance_grad", "balance_grad_few", 37, 64, 4, "f32", "softmax", 0.0),
        _balance("balance_grad", "balance_grad_train", 16384, 256, 8, "f32", "sigmoid", 0.0),
        _balance("balance_grad", "balance_grad_long", 65521, 128, 8, "bf16", "softmax", 0.01),
    ]


def _xent(name, M, N, K, dtype, alpha):
    return {"name": name, "op": "xent", "M": M, "N": N, "K": K, "dtype": dtype, "alpha": alpha}


def _xent_grad(name, M, N, K, dtype, alpha, dlse):
    return {"name": name, "op": "xent_grad", "M": M, "N": N, "K": K, "dtype": dtype,
            "alpha": alpha, "dlse": dlse}


def _balance(op, name, T, E, k, dtype, score, pad):
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "dtype": dtype, "score": score,
            "pad": pad}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["xent", "xent", "xent_grad", "xent_grad", "balance", "balance_grad"])
    if op in ("xent", "xent_grad"):
        cap = 1 << (42 if op == "xent" else 41)     # M * N * K of the largest listed case
        M = _log(rng, 1, 8192)
        K = 8 * _log(rng, 16, 1024)
        N = _log(rng, 64, max(65, min(131072, (1 << 29) // K, cap // (M * K))))
        c = _xent("", M, N, K, rng.choice(["bf16", "bf16", "f16"]), rng.choice([1.0, 0.5]))
        if op == "xent_grad":
            c = _xent_grad("", M, N, K, c["dtype"], c["alpha"], rng.random() < 0.4)
    else:
        E = _log(rng, 8, 256)
        c = _balance(op, "", _log(rng, 1, 65521), E, rng.randint(1, min(8, E)),
                     rng.choice(["f32", "bf16", "f16"]), rng.choice(["softmax", "sigmoid"]),
                     rng.choice([0.0, 0.02]))
        if c["T"] * E * _ES[c["dtype"]] > 1 << 24:
            c["T"] = (1 << 24) // (E * _ES[c["dtype"]]) - 3
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs

def _scores(x, score):
    """The experts' scores in x's type; masked logits (-inf, NaN) score zero."""
    live = x > -math.inf
    if score == "sigmoid":
        return torch.where(live, 1 / (1 + torch.exp(-x)), 0)
    top = torch.where(live, x, -math.inf).amax(1, keepdim=True)
    e = torch.where(live, torch.exp(x - top), 0)
    return e / e.sum(1, keepdim=True).clamp_min(TINY)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    if case["op"] in ("xent", "xent_grad"):
        # Logits of a standard deviation of 1.5; the targets' are up to 12
        # larger, so that some tokens are nearly certain and some are not.
        # One token in twenty has no target.
        M, N, K = case["M"], case["N"], case["K"]
        b = randn(N, K).mul_(1.5 / (math.sqrt(K) * case["alpha"]))
        t = torch.randint(0, N, (M,), generator=gen, device="cuda")
        w = b[t]
        known = 12 * rand(M, 1) * (rand(M, 1) < 0.7) / case["alpha"]
        a = randn(M, K) + known * w / (w * w).sum(1, keepdim=True)
        s["a"], s["b"] = a.to(_DT[case["dtype"]]), b.to(_DT[case["dtype"]])
        s["t"] = torch.where(rand(M) < 0.05, IGNORE, t)
        if case["op"] == "xent_grad":
            z = s["a"].float() @ s["b"].float().t()
            s["lse"] = z.mul_(case["alpha"]).logsumexp(1)
            # The mean over the tokens; 16-bit floats of a narrow range are
            # trained with a scaled loss.
            scale = 1024.0 if case["dtype"] == "f16" else 1.0
            s["dloss"] = torch.full((M,), scale / M, device="cuda")
            s["dlse"] = 2e-3 * s["lse"] * s["dloss"] if case["dlse"] else None
        return s
    T, E, k = case["T"], case["E"], case["k"]
    x = randn(T, E) + 0.5 * randn(1, E)     # experts of uneven popularity
    if case["pad"]:
        x[rand(T) < case["pad"]] = -math.inf
    s["logits"] = x.to(_DT[case["dtype"]])
    ids = x.topk(k, 1).indices.to(torch.int32)
    s["ids"] = torch.where(x[:, :1] == -math.inf, -1, ids).contiguous()
    if case["op"] == "balance_grad":
        flat = s["ids"].reshape(-1).long()
        s["counts"] = torch.bincount(flat[flat >= 0], minlength=E).to(torch.int32)
        s["tokens"] = (x > -math.inf).any(1).sum().to(torch.int32)
        scale = float(T * E) if case["dtype"] == "f16" else 1.0
        s["dloss"] = torch.full((), 0.01 * scale, device="cuda")
    return s


# ------------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_xent(s):
    import dense_gemm_swizzled_amd as sg
    return sg.gemm_xent(s["a"], s["b"], s["t"], alpha=s["alpha"])


def _own_xent_grad(s):
    import dense_gemm_swizzled_amd as sg
    return sg.gemm_xent_backward(s["dloss"], s["a"], s["b"], s["t"], s["lse"], alpha=s["alpha"],
                                 dlse=s["dlse"])


def _own_balance(s):
    import dense_gemm_swizzled_amd as sg
    return sg.moe_balance(s["logits"], s["ids"], score=s["score"])


def _own_balance_grad(s):
    import dense_gemm_swizzled_amd as sg
    return sg.moe_balance_backward(s["dloss"], s["logits"], s["counts"], s["tokens"],
                                   score=s["score"])


_own = {"xent": _own_xent, "xent_grad": _own_xent_grad, "balance": _own_balance,
        "balance_grad": _own_balance_grad}


def _targets(s):
    """Which tokens have a target, and an index for each."""
    t, N = s["t"], s["b"].shape[0]
    valid = (t >= 0) & (t < N)
    return valid, torch.where(valid, t, 0)[:, None]


def _plain_xent(s):
    z = (s["a"].float() @ s["b"].float().t()) * s["alpha"]
    valid, at = _targets(s)
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    return torch.where(valid, lse - z.gather(1, at)[:, 0], 0), lse


def _plain_xent_grad(s):
    a, b = s["a"].float(), s["b"].float()
    valid, at = _targets(s)
    dl = torch.where(valid, s["dloss"], 0)
    whole = dl if s["dlse"] is None else dl + s["dlse"]
    z = (a @ b.t()) * s["alpha"]
    g = torch.exp(z - s["lse"][:, None]) * whole[:, None]
    g.scatter_add_(1, at, -dl[:, None])
    g *= s["alpha"]
    return (g @ b).to(s["a"].dtype), (g.t() @ a).to(s["b"].dtype)


def _shares(s):
    """Which tokens count, their scores, the scores' sums and the shares of
    the sums, in 32 bits."""
    x = s["logits"].float()
    p = _scores(x, s["score"])
    total = p.sum(1, keepdim=True).clamp_min(TINY)
    return (x > -math.inf).any(1), p, total, p / total


def _plain_balance(s):
    live, _, _, share = _shares(s)
    E = s["E"]
    ids = s["ids"].reshape(-1)
    ok = (ids >= 0) & (ids < E)
    counts = torch.zeros(E, device="cuda").scatter_add_(0, torch.where(ok, ids, 0).long(),
                                                        ok.float())
    tokens = live.sum()
    load = E * counts / counts.sum().clamp_min(1)
    loss = (load * (share.sum(0) / tokens.clamp_min(1))).sum()
    return loss, counts.to(torch.int32), tokens.to(torch.int32)


def _plain_balance_grad(s):
    _, p, total, share = _shares(s)
    counts = s["counts"].float()
    d = s["dloss"] * s["E"] * counts / counts.sum().clamp_min(1) / s["tokens"].clamp_min(1)
    d = d - (share * d).sum(1, keepdim=True)
    if s["score"] == "sigmoid":
        dx = p * (1 - p) / total * d
    else:
        dx = p * d
    return dx.to(s["logits"].dtype)


_plain = {"xent": _plain_xent, "xent_grad": _plain_xent_grad, "balance": _plain_balance,
          "balance_grad": _plain_balance_grad}


# ------------------------------------------------------------------- the floor

def work(case):
    op = case["op"]
    if op in ("xent", "xent_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        both = (M + N) * K * 2
        if op == "xent":
            return {"bytes": both + 16 * M, "flops": 2 * M * N * K}
        # The logits once more, then one product for each gradient.
        return {"bytes": 2 * both + (20 if case["dlse"] else 16) * M, "flops": 6 * M * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "balance":
        return {"bytes": T * E * _ES[case["dtype"]] + 4 * T * k + 4 * E + 8, "flops": 8 * T * E}
    return {"bytes": 2 * T * E * _ES[case["dtype"]] + 4 * E + 8, "flops": 10 * T * E}


# ----------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("xent", "xent_grad"):
        return _exact_xent(s)
    # On the host, by automatic differentiation.
    x = s["logits"].double().cpu().requires_grad_(case["op"] == "balance_grad")
    live = x[:, 0] > -math.inf      # padding tokens are masked as a whole
    if case["op"] == "balance":
        counts = torch.bincount(s["ids"].cpu().reshape(-1)[s["ids"].cpu().reshape(-1) >= 0],
                                minlength=case["E"]).double()
    else:
        counts = s["counts"].cpu().double()
    y = x[live]
    p = torch.softmax(y, 1) if case["score"] == "softmax" else torch.sigmoid(y)
    p = p / p.sum(1, keepdim=True)
    load = case["E"] * counts / max(float(counts.sum()), 1.0)
    loss = torch.dot(load, p.sum(0) / max(p.shape[0], 1))
    if case["op"] == "balance":
        return loss, None, None
    (loss * s["dloss"].double().cpu()).backward()
    return x.grad


def _exact_xent(s):
    """The tokens in runs, so that the logits in 64 bits stay small."""
    a, b, N = s["a"].double(), s["b"].double(), s["b"].shape[0]
    step = max(1, (1 << 29) // N)
    loss, lse, da = [], [], []
    db = torch.zeros_like(b) if s["op"] == "xent_grad" else None
    for i in range(0, a.shape[0], step):
        ai, ti = a[i:i + step], s["t"][i:i + step]
        logp = torch.log_softmax(s["alpha"] * torch.mm(ai, b.t()), 1)
        has = (ti >= 0) & (ti < N)
        rows, cols = torch.nonzero(has)[:, 0], ti[has]
        if db is None:
            nll = torch.zeros(ai.shape[0], dtype=torch.float64, device="cuda")
            nll[rows] = -logp[rows, cols]
            loss.append(nll)
            z0 = s["alpha"] * torch.mv(ai, b[0])
            lse.append(z0 - logp[:, 0])
            continue
        dl = s["dloss"][i:i + step].double() * has
        g = logp.exp_()
        g *= (dl if s["dlse"] is None else dl + s["dlse"][i:i + step].double())[:, None]
        g[rows, cols] -= dl[rows]
        g *= s["alpha"]
        da.append(torch.mm(g, b))
        db += torch.mm(g.t(), ai)
    return (torch.cat(da), db) if db is not None else (torch.cat(loss), torch.cat(lse))
