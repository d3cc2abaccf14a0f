"""The router and the dense projections in numpy, 64 bits: the definitions
that include/moe_prefill.h gives for moe_linear, moe_linear_grad, moe_route
and moe_route_grad, in the plainest form (no care for speed or range beyond
what 64 bits give).  Test infrastructure only."""
import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def _sigmoid(z):
    z = np.asarray(z, dtype=np.float64)
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "silu":
        return z * _sigmoid(z)
    if name == "gelu":
        return z * (1.0 + _erf(z / math.sqrt(2.0))) / 2.0
    return z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))) / 2.0


def act_grad(z, name):
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = _sigmoid(z)
        return s + z * s * (1.0 - s)
    if name == "gelu":
        return (1.0 + _erf(z / math.sqrt(2.0))) / 2.0 + z * np.exp(-z * z / 2.0) / math.sqrt(
            2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = np.tanh(c * (z + 0.044715 * z ** 3))
    return (1.0 + t) / 2.0 + z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z) / 2.0


def linear(x, W, bias=None, residual=None, act_name="none"):
    """(y, pre)."""
    z = x @ W.T
    if bias is not None:
        z = z + bias
    y = act(z, act_name)
    return (y if residual is None else y + residual), z


def linear_grad(x, W, dy, pre=None, act_name="none"):
    """(dx, dW, db)."""
    dp = dy if act_name == "none" else dy * act_grad(pre, act_name)
    return dp @ W, dp.T @ x, dp.sum(0)


def _open(logits, mask):
    with np.errstate(invalid="ignore"):
        ok = (logits > -np.inf) & (logits < np.inf)
    if mask is not None:
        ok &= np.asarray(mask, dtype=bool)[:, None]
    return ok


def route(logits, k, bias=None, mask=None, score="softmax", norm=True, scale=1.0):
    """ids, w, counts, prob, loss, and keys (the row's choice keys, closed experts -inf)."""
    T, E = logits.shape
    ok = _open(logits, mask)
    ids = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    keys = np.full((T, E), -np.inf)
    counts = np.zeros(E + 1, dtype=np.int32)
    prob, z = np.zeros(E), 0.0
    for t in range(T):
        at = np.flatnonzero(ok[t])
        if at.size == 0:
            continue
        l = logits[t, at].astype(np.float64)
        e = np.exp(l - l.max())
        s = e / e.sum() if score == "softmax" else _sigmoid(l)
        a = l if score == "softmax" else -np.logaddexp(0.0, -l)  # log of the score, up to a constant
        keys[t, at] = l if bias is None else s + bias[at]
        order = sorted(range(at.size), key=lambda i: (-keys[t, at[i]], at[i]))[:k]
        ids[t, :len(order)] = at[order]
        sel = np.exp(a[order] - a[order].max())
        w[t, :len(order)] = scale * (sel / sel.sum() if norm else s[order])
        counts[at[order]] += 1
        counts[E] += 1
        p = np.exp(a - a.max())
        prob[at] += p / p.sum()
        z += (l.max() + math.log(e.sum())) ** 2
    n = max(1, int(counts[E]))
    prob /= n
    loss = np.array([E * float(np.dot(counts[:E] / (n * k), prob)), z / n])
    return dict(ids=ids, w=w, counts=counts, prob=prob, loss=loss, keys=keys)


def route_value(logits, ids, counts, dw, dloss, mask=None, score="softmax", norm=True, scale=1.0):
    """sum(dw * w) + dloss . loss with the choice and the counts held fixed:
    the function that moe_route_grad differentiates."""
    T, E = logits.shape
    k = ids.shape[1]
    ok = _open(logits, mask)
    n = max(1, int(counts[E]))
    f = counts[:E] / (n * k)
    total = 0.0
    for t in range(T):
        at = np.flatnonzero(ok[t])
        if at.size == 0:
            continue
        l = np.full(E, -np.inf)
        l[at] = logits[t, at]
        a = l.copy() if score == "softmax" else np.where(l > -np.inf, -np.logaddexp(
            0.0, -np.where(l > -np.inf, l, 0.0)), -np.inf)
        p = np.exp(a - a.max())
        p /= p.sum()
        lse = l.max() + math.log(np.exp(l - l.max()).sum())
        total += dloss[0] * E * float(np.dot(f, p)) / n + dloss[1] * lse * lse / n
        js = [j for j in range(k) if 0 <= ids[t, j] < E and ok[t, ids[t, j]]]
        if js:
            sel = a[ids[t, js]]
            if norm:
                q = np.exp(sel - sel.max())
                q /= q.sum()
            else:
                q = p[ids[t, js]] if score == "softmax" else np.exp(sel)
            total += scale * float(np.dot(dw[t, js], q))
    return total


def route_grad(logits, ids, counts, dw, dloss, mask=None, score="softmax", norm=True, scale=1.0):
    """dlogits, by the chain rule through log-scores a."""
    T, E = logits.shape
    k = ids.shape[1]
    ok = _open(logits, mask)
    n = max(1, int(counts[E]))
    c = dloss[0] * E * counts[:E] / (n * k) / n
    out = np.zeros((T, E))
    for t in range(T):
        at = np.flatnonzero(ok[t])
        if at.size == 0:
            continue
        l = logits[t, at].astype(np.float64)
        where = {int(e): i for i, e in enumerate(at)}
        a = l if score == "softmax" else -np.logaddexp(0.0, -l)
        p = np.exp(a - a.max())
        p /= p.sum()
        da = p * (c[at] - np.dot(p, c[at]))
        js = [j for j in range(k) if int(ids[t, j]) in where]
        if js:
            i = np.array([where[int(ids[t, j])] for j in js])
            d = scale * dw[t, js]
            if norm:
                q = np.exp(a[i] - a[i].max())
                q /= q.sum()
                da[i] += q * (d - np.dot(q, d))
            elif score == "softmax":
                da[i] += p[i] * d
                da -= p * np.dot(p[i], d)
            else:
                da[i] += np.exp(a[i]) * d
        e = np.exp(l - l.max())
        lse = l.max() + math.log(e.sum())
        dl = da if score == "softmax" else da * _sigmoid(-l)
        out[t, at] = dl + 2.0 * dloss[1] * lse / n * e / e.sum()
    return out
