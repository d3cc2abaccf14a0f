"""Measured cases of the router and dense-projection operators.

Four operators stand around the routed experts of a mixture-of-experts block:

* ``linear``       y = act(x W^T + b) + residual: the router's logits, the dense
                   projections beside the experts and the residual add.
* ``linear_grad``  its gradients: dx, dW and db from dy.
* ``route``        logits -> top-k experts, their weights, per-expert counts, the
                   mean probability of each expert, the balance and z losses.
* ``route_grad``   the gradient of the weights and of both losses with respect
                   to the logits.

``run`` computes a case in plain 32-bit torch operations, or, where ``own`` is
set, through the package's entry points.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
_INF = float("inf")


# ---- the cases --------------------------------------------------------------


def _lin(name, T, K, N, **kw):
    c = {"name": name, "op": "linear", "T": T, "K": K, "N": N, "dtype": "bf16", "out": "same",
         "act": "none", "bias": True, "residual": False, "pre": False, "pad": 0}
    return {**c, **kw}


def _lin_grad(name, T, K, N, **kw):
    c = {"name": name, "op": "linear_grad", "T": T, "K": K, "N": N, "dtype": "bf16",
         "dy": "same", "act": "none", "dw": "same", "pad": 0}
    return {**c, **kw}


def _route(name, T, E, k, **kw):
    c = {"name": name, "op": "route", "T": T, "E": E, "k": k, "dtype": "f32", "score": "softmax",
         "norm": True, "scale": 1.0, "bias": False, "masked": 0.0, "closed": 0.0, "stats": True}
    return {**c, **kw}


def listed():
    return [
        # router logits of a single decoded token: weights of 512 experts are read, latency counts
        _lin("logits, one token", 1, 2560, 512, out="f32"),
        # router logits of one prefill chunk
        _lin("logits, chunk of 2048", 2048, 2560, 512, out="f32"),
        # dense down projection with the residual add for a batch of 16 decoded tokens
        _lin("down + residual, 16 tokens", 16, 10240, 2560, residual=True),
        # odd everything: rows of a wider tensor, half precision, an output width of 1001
        _lin("ragged half precision", 777, 1032, 1001, dtype="f16", act="silu", residual=True,
             pad=24),
        # dense up projection with GELU of a long-prompt chunk, keeping what its backward needs
        _lin("up + GELU, chunk of 4096", 4096, 2816, 11264, act="gelu_tanh", pre=True),
        # the router's weight and input gradients from the gradient of its logits
        _lin_grad("router gradients", 2048, 2560, 512, dy="f32"),
        # the gradients of the dense up projection
        _lin_grad("up + GELU gradients", 4096, 2816, 11264, act="gelu_tanh"),
        # routing of a single decoded token
        _route("route one token", 1, 512, 10, stats=False),
        # training or prefill chunk: routing, counts and losses
        _route("route, chunk of 2048", 2048, 512, 10),
        # long prompt, sigmoid scores with a selection bias, padded tokens, some experts closed
        _route("route, sigmoid, 32768 tokens", 32768, 128, 8, score="sigmoid", scale=2.5,
               bias=True, masked=0.1, closed=0.05),
        # gradient of a chunk's routing
        _route("route gradient, 2048", 2048, 512, 10, op="route_grad"),
        # gradient of a long prompt's routing, 16-bit logits, weights not renormalised
        _route("route gradient, 32768", 32768, 256, 8, op="route_grad", dtype="bf16", norm=False,
               masked=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_grad", "route", "route", "route_grad"))
    if op.startswith("linear"):
        T = _log_int(rng, 1, 4096)
        K = 8 * _log_int(rng, 8, 1408)  # rows of K 16-bit values are multiples of 16 bytes
        N = _log_int(rng, 3, 11264)
        dtype = rng.choice(("bf16", "bf16", "f16"))
        act, pad = rng.choice(_ACTS), rng.choice((0, 0, 8, 40))
        if op == "linear":
            c = _lin("", T, K, N, dtype=dtype, act=act, pad=pad, out=rng.choice(("same", "f32")),
                     bias=rng.random() < 0.7, residual=rng.random() < 0.5, pre=rng.random() < 0.3)
        else:
            c = _lin_grad("", T, K, N, dtype=dtype, act=act, pad=pad, dy=rng.choice(("same", "f32")))
            if act == "none" and c["dy"] == "same" and rng.random() < 0.5:
                c["dw"] = "f32"
    else:
        E = _log_int(rng, 8, 512)
        k = min(E, _log_int(rng, 1, 16))
        c = _route("", _log_int(rng, 1, 32768), E, k, op=op, dtype=rng.choice(("f32", "f32", "bf16")),
                   score=rng.choice(("softmax", "sigmoid")), norm=rng.random() < 0.6,
                   scale=rng.choice((1.0, 2.5)), bias=rng.random() < 0.4,
                   masked=rng.choice((0.0, 0.1, 0.5)), closed=rng.choice((0.0, 0.0, 0.2)),
                   stats=rng.random() < 0.8)
    del c["name"]
    return c


# ---- inputs -----------------------------------------------------------------


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(g, T, K, pad, dtype):
    """[T, K] rows, with pad > 0 the first K columns of a wider tensor."""
    return _randn(g, T, K + pad).to(dtype)[:, :K]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"].startswith("linear"):
        T, K, N, dt = case["T"], case["K"], case["N"], _DT[case["dtype"]]
        s["x"] = _rows(g, T, K, case["pad"], dt)
        s["W"] = (0.02 * _randn(g, N, K)).to(dt)
        if case["op"] == "linear":
            ydt = dt if case["out"] == "same" else torch.float32
            s["ydt"] = ydt
            s["b"] = 0.1 * _randn(g, N) if case["bias"] else None
            s["r"] = _rows(g, T, N, case["pad"], ydt) if case["residual"] else None
        else:
            # gradients the size a mean loss over the chunk gives them (fp16: with its loss scale)
            amp = 1e-2 if dt == torch.float16 else 1e-4
            s["dy"] = (amp * _randn(g, T, N)).to(dt if case["dy"] == "same" else torch.float32)
            s["p"] = _randn(g, T, N).to(dt) if case["act"] != "none" else None
            s["dwdt"] = dt if case["dw"] == "same" else torch.float32
        return s
    T, E, k = case["T"], case["E"], case["k"]
    l = (_randn(g, T, E) + _randn(g, E)).to(_DT[case["dtype"]])
    if case["closed"]:  # experts that a token may not use
        l[torch.rand(T, E, generator=g, device="cuda") < case["closed"]] = -_INF
    s["bias"] = 0.1 * _randn(g, E) if case["bias"] else None
    if case["bias"]:
        # Ids have to be the same whatever the rounding of a score, so tokens whose first keys
        # lie within 4e-6 of one another are given another token's logits.
        q = l.double()
        q = (torch.sigmoid(q) if case["score"] == "sigmoid" else
             torch.softmax(q, 1).nan_to_num(0.0)) + s["bias"].double()
        top = torch.where(l > -_INF, q, -_INF).topk(min(E, k + 1), dim=1).values
        near = ((top[:, :-1] - top[:, 1:]) < 4e-6).any(1)
        good = int(torch.argmin(near.to(torch.int32)))
        l[near] = l[good].clone()
    s["mask"] = None
    if case["masked"]:  # padding: these rows hold anything
        s["mask"] = torch.rand(T, generator=g, device="cuda") >= case["masked"]
        l[~s["mask"]] = float("nan")
    s["l"] = l
    if case["op"] == "route_grad":
        r = _route_plain(s)
        s["ids"], s["counts"] = r["ids"], r["counts"]
        s["dw"] = 1e-3 * _randn(g, T, k)
        s["dloss"] = torch.tensor([1e-2, 1e-3], device="cuda")
    return s


# ---- plain forms ------------------------------------------------------------


def _act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    if name == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _linear_plain(s):
    z = s["x"].float() @ s["W"].float().t()
    if s["b"] is not None:
        z = z + s["b"]
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"y": y.to(s["ydt"])}
    if s["pre"]:
        out["pre"] = z.to(s["x"].dtype)
    return out


def _linear_grad_plain(s):
    dp = s["dy"].float()
    if s["act"] != "none":
        dp = dp * _act_grad(s["p"].float(), s["act"])
    return {"dx": (dp @ s["W"].float()).to(s["x"].dtype),
            "dW": (dp.t() @ s["x"].float()).to(s["dwdt"]), "db": dp.sum(0)}


def _open_rows(s):
    """32-bit logits (0 where closed), which of them may be used, and the tokens that take part."""
    l = s["l"].float()
    ok = l > -_INF
    if s["mask"] is not None:
        ok = ok & s["mask"][:, None]
    return torch.where(ok, l, 0.0), ok, ok.any(1)


def _log_score(l, score):
    return l if score == "softmax" else l.clamp(max=0) - torch.log1p(torch.exp(-l.abs()))


def _softmax(a, ok):
    """Softmax over the entries in ok (rows without any: 0) and its log-sum-exp (0 there)."""
    m = torch.where(ok, a, -_INF).amax(1, keepdim=True).clamp(min=-3e38)
    e = torch.where(ok, torch.exp(torch.where(ok, a - m, 0.0)), 0.0)
    t = e.sum(1, keepdim=True)
    some = t > 0
    return (torch.where(some, e / torch.where(some, t, 1.0), 0.0),
            torch.where(some, m + torch.log(torch.where(some, t, 1.0)), 0.0)[:, 0])


def _route_plain(s):
    T, E = s["l"].shape
    l, ok, live = _open_rows(s)
    a = _log_score(l, s["score"])
    p, lse = _softmax(a, ok)
    key = l
    if s["bias"] is not None:
        key = (p if s["score"] == "softmax" else 1 / (1 + torch.exp(-l))) + s["bias"]
    key = torch.where(ok, key, -_INF)
    at = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :s["k"]]
    used = ok.gather(1, at)
    sel = a.gather(1, at)
    if s["norm"]:
        w = _softmax(sel, used)[0]
    else:
        w = torch.where(used, p.gather(1, at) if s["score"] == "softmax" else torch.exp(sel), 0.0)
    out = {"ids": torch.where(used, at, -1).to(torch.int32), "w": w * s["scale"]}
    if s["stats"] or s["op"] == "route_grad":
        n = live.sum()
        counts = torch.zeros(E + 1, dtype=torch.int32, device=l.device)
        counts.scatter_add_(0, torch.where(used, at, E).reshape(-1),
                            torch.ones(at.numel(), dtype=torch.int32, device=l.device))
        counts[E] = n
        n1 = n.clamp(min=1).float()
        prob = p.sum(0) / n1
        z = _softmax(l, ok)[1] if s["score"] == "sigmoid" else lse
        balance = E * (counts[:E].float() / (n1 * s["k"]) * prob).sum()
        out.update(counts=counts, prob=prob, loss=torch.stack((balance, (z * z).sum() / n1)))
    return out


def _route_grad_plain(s):
    E = s["l"].shape[1]
    l, ok, live = _open_rows(s)
    a = _log_score(l, s["score"])
    p, lse = _softmax(a, ok)
    n1 = s["counts"][E].clamp(min=1).float()
    f = s["counts"][:E].float() * (s["dloss"][0] * E / (n1 * n1 * s["k"]))
    used = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long()
    dw = torch.where(used, s["dw"], 0.0) * s["scale"]
    da = p * (f - (p * f).sum(1, keepdim=True))
    if s["norm"]:
        q = _softmax(a.gather(1, at), used)[0]
        dsel = q * (dw - (q * dw).sum(1, keepdim=True))
    elif s["score"] == "softmax":
        ps = torch.where(used, p.gather(1, at), 0.0)
        dsel = ps * dw
        da = da - p * dsel.sum(1, keepdim=True)
    else:
        dsel = torch.where(used, torch.exp(a.gather(1, at)), 0.0) * dw
    da.scatter_add_(1, at, dsel)
    if s["score"] == "sigmoid":
        da = da / (1 + torch.exp(l))
        p, lse = _softmax(l, ok)
    da = da + p * (lse * (2 * s["dloss"][1] / n1))[:, None]
    return {"dlogits": torch.where(ok, da, 0.0).to(s["l"].dtype)}


# ---- one pass ---------------------------------------------------------------


def _run_own(s):
    from moe_prefill_routing_gb300 import binding as B

    op = s["op"]
    if op == "linear":
        pre = None
        if s["pre"]:
            pre = torch.empty((s["T"], s["N"]), dtype=s["x"].dtype, device=s["x"].device)
        y = B.linear(s["x"], s["W"], bias=s["b"], residual=s["r"], act=s["act"],
                     out_dtype=s["ydt"], pre=pre)
        return {"y": y} if pre is None else {"y": y, "pre": pre}
    if op == "linear_grad":
        dx, dW, db = B.linear_grad(s["x"], s["W"], s["dy"], pre=s["p"], act=s["act"],
                                   dw_dtype=s["dwdt"])
        return {"dx": dx, "dW": dW, "db": db}
    if op == "route":
        r = B.route(s["l"], s["k"], bias=s["bias"], mask=s["mask"], score=s["score"],
                    norm=s["norm"], scale=s["scale"], stats=s["stats"])
        names = ("ids", "w", "counts", "prob", "loss") if s["stats"] else ("ids", "w")
        return {n: r[n] for n in names}
    return {"dlogits": B.route_grad(s["l"], s["ids"], s["counts"], dw=s["dw"], dloss=s["dloss"],
                                    mask=s["mask"], score=s["score"], norm=s["norm"],
                                    scale=s["scale"])}


_PLAIN = {"linear": _linear_plain, "linear_grad": _linear_grad_plain, "route": _route_plain,
          "route_grad": _route_grad_plain}


def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    c = case
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if c["op"].startswith("linear"):
        T, K, N, b = c["T"], c["K"], c["N"], size[c["dtype"]]
        if c["op"] == "linear":
            o = b if c["out"] == "same" else 4
            n = T * K * b + N * K * b + T * N * o * (2 if c["residual"] else 1)
            n += 4 * N * bool(c["bias"]) + T * N * b * bool(c["pre"])
            return {"bytes": n, "flops": 2.0 * T * K * N}
        n = 2 * T * K * b + N * K * (b + (b if c["dw"] == "same" else 4)) + 4 * N
        n += T * N * ((b if c["dy"] == "same" else 4) + (b if c["act"] != "none" else 0))
        return {"bytes": n, "flops": 4.0 * T * K * N}
    T, E, k, b = c["T"], c["E"], c["k"], size[c["dtype"]]
    n = T * E * b + T * k * 8 + (T if c["masked"] else 0)
    if c["op"] == "route":
        n += (8 * E + 12 if c["stats"] else 0) + (4 * E if c["bias"] else 0)
        return {"bytes": n, "flops": 6.0 * T * E}
    return {"bytes": n + T * E * b + 4 * E + 12, "flops": 10.0 * T * E}


# ---- the definitions in 64 bits ---------------------------------------------


def _act64(z, name):
    f = torch.nn.functional
    if name == "none":
        return z
    if name == "gelu_tanh":
        return f.gelu(z, approximate="tanh")
    return {"relu": f.relu, "silu": f.silu, "gelu": f.gelu}[name](z)


def _scores64(s, l, ok):
    """Probabilities for the balance loss, scores, and log-sum-exp of the open experts' logits."""
    z = l.masked_fill(~ok, -_INF)
    if s["score"] == "softmax":
        p = torch.softmax(z, 1)
        return p, p, torch.logsumexp(z, 1)
    q = torch.sigmoid(l) * ok
    return q / q.sum(1, keepdim=True), q, torch.logsumexp(z, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        z = torch.einsum("tk,nk->tn", s["x"].double(), s["W"].double())
        z = z if s["b"] is None else z + s["b"].double()
        y = _act64(z, s["act"])
        out = {"y": y if s["r"] is None else y + s["r"].double()}
        return {**out, "pre": z} if s["pre"] else out
    if case["op"] == "linear_grad":
        dp = s["dy"].double()
        if s["act"] != "none":
            z = s["p"].double().requires_grad_(True)
            # at 0 the derivative of relu is taken as 0
            dp, = torch.autograd.grad(_act64(z, s["act"]), z, dp)
        return {"dx": torch.einsum("tn,nk->tk", dp, s["W"].double()),
                "dW": torch.einsum("tn,tk->nk", dp, s["x"].double()), "db": dp.sum(0)}
    # tokens that take part, and the rest of the definition on those alone
    E, k, sig = case["E"], case["k"], case["score"] == "sigmoid"
    open_all = (s["l"] > -_INF) & (True if s["mask"] is None else s["mask"][:, None])
    live = open_all.any(1)
    ok = open_all[live]
    n = max(1, int(live.sum()))
    l = s["l"][live].double().masked_fill(~ok, 0.0).requires_grad_(True)
    p, q, lse = _scores64(s, l, ok)
    if case["op"] == "route":
        key = l.detach() if s["bias"] is None else q.detach() + s["bias"].double()
        key = key.masked_fill(~ok, -_INF)
        at = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    else:
        at = s["ids"][live].long().clamp(min=0)
    used = ok.gather(1, at) if case["op"] == "route" else s["ids"][live] >= 0
    w = q.gather(1, at) * used
    if s["norm"]:
        # a ratio of scores; from their logarithms, as all of them may be tiny
        la = torch.nn.functional.logsigmoid(l) if sig else l
        some = used.any(1, keepdim=True)
        w = torch.softmax(la.gather(1, at).masked_fill(~used & some, -_INF), 1) * used
    w = w * case["scale"]
    if case["op"] == "route":
        full = torch.zeros(case["T"], k, dtype=torch.float64, device=l.device)
        full[live] = w.detach()
        out = {"ids": None, "w": full}
        if case["stats"]:
            hits = torch.bincount(at[used], minlength=E).double()
            prob = p.detach().sum(0) / n
            out.update(counts=None, prob=prob,
                       loss=torch.stack((E * (hits / (n * k)) @ prob, lse.detach().square().sum() / n)))
        return out
    share = s["counts"][:E].double() / (n * k)
    total = ((w * s["dw"][live].double()).sum()
             + s["dloss"][0].double() * E * (share * p.sum(0) / n).sum()
             + s["dloss"][1].double() * lse.square().sum() / n)
    dl, = torch.autograd.grad(total, l)
    full = torch.zeros(case["T"], E, dtype=torch.float64, device=l.device)
    full[live] = dl * ok
    return {"dlogits": full}
