"""The block norm, MXFP4 rows and the MXFP4 product in numpy, 64 bits: the
definitions that include/moe_prefill.h gives for moe_block_norm,
moe_block_norm_grad, moe_quantize_rows_mxfp4 and moe_linear_mxfp4, in the
plainest form.  Test infrastructure only."""
import numpy as np

from . import router

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _norm(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def _gate(gate, act, T):
    if gate is None:
        return np.ones((T, 1))
    g = gate[:, None]
    return 1.0 / (1.0 + np.exp(-g)) if act == "sigmoid" else g


def stream(x, o, post=None, gate=None, mask=None, post_norm=True, gate_act="none", alpha=1.0,
           eps=1e-6):
    """xn, not rounded."""
    live = np.ones(len(x), bool) if mask is None else mask.astype(bool)
    x, o = np.where(live[:, None], x, 0.0), np.where(live[:, None], o, 0.0)
    n = o * _norm(o, eps) if post_norm else o
    n = n if post is None else n * post
    return np.where(live[:, None], alpha * x + _gate(gate, gate_act, len(x)) * n, 0.0)


def normed(xn, pre, mask=None, eps=1e-6):
    """h of the stream as it is stored, not rounded."""
    if mask is not None:
        xn = np.where(mask.astype(bool)[:, None], xn, 0.0)
    return xn * _norm(xn, eps) * pre


def grads(xn, o=None, dxn=None, dh=None, pre=None, post=None, gate=None, mask=None,
          post_norm=True, gate_act="none", alpha=1.0, eps=1e-6):
    """dx, do, dgate, dpre, dpost (those there are), and as "size" the magnitudes
    that each is made of: what a relative error of every step is relative to."""
    live = np.ones((len(xn), 1), bool) if mask is None else mask.astype(bool)[:, None]
    z = lambda v: np.where(live, v, 0.0)  # noqa: E731
    d = xn.shape[1]
    ds, size = np.zeros(xn.shape), np.zeros(xn.shape)
    out, mag = {}, {}
    if dxn is not None:
        ds = z(dxn)
        size = np.abs(ds)
    if dh is not None:
        x, h = z(xn), z(dh)
        r = _norm(x, eps)
        a = h * pre
        ds = ds + r * a - r ** 3 * np.mean(a * x, axis=1, keepdims=True) * x
        size = size + np.abs(r * a) + r ** 3 * np.mean(np.abs(a * x), axis=1,
                                                       keepdims=True) * np.abs(x)
        out["dpre"] = np.sum(h * x * r, axis=0)
        mag["dpre"] = np.sum(np.abs(h * x * r), axis=0)
    if o is None:
        out["dx"], mag["dx"] = ds, size
        return out, mag
    out["dx"], mag["dx"] = alpha * ds, abs(alpha) * size
    o = z(o)
    r1 = _norm(o, eps) if post_norm else np.ones((len(o), 1))
    p = np.ones(d) if post is None else post
    g = _gate(gate, gate_act, len(o)) * live
    q = np.sum(ds * p * o, axis=1, keepdims=True)
    q_size = np.sum(size * np.abs(p * o), axis=1, keepdims=True)
    if gate is not None:
        slope = g * (1 - g) if gate_act == "sigmoid" else 1.0
        out["dgate"] = (live * r1 * q * slope)[:, 0]
        mag["dgate"] = (live * r1 * q_size * np.abs(slope))[:, 0]
    if post is not None:
        out["dpost"] = np.sum(g * r1 * ds * o, axis=0)
        mag["dpost"] = np.sum(np.abs(g * r1 * o) * size, axis=0)
    do = g * r1 * ds * p
    m = np.abs(g * r1 * p) * size
    if post_norm:
        do = do - r1 ** 3 * g * q / d * o
        m = m + np.abs(r1 ** 3 * g * q_size / d * o)
    out["do"], mag["do"] = z(do), m
    return out, mag


# ---- MXFP4 rows -------------------------------------------------------------------


def mx_encode(v):
    """Codes [R, K] (one a value) and scale bytes [R, K/32]."""
    R, K = v.shape
    b = np.asarray(v, dtype=np.float64).reshape(R, K // 32, 32)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], 0.0, b)
    top = np.abs(b).max(axis=2)
    exp = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127).clip(-127, 127)
    a = np.ldexp(np.abs(b), -exp[:, :, None])
    # the nearest magnitude; of two equally near ones that with the even code
    dist = np.abs(a[..., None] - VALUES)
    order = dist + np.where(np.arange(8) % 2, 1e-9, 0.0)
    code = np.argmin(order, axis=3)
    code = np.where(a >= 6.0, 7, code) + 8 * np.signbit(b)
    return (code.reshape(R, K).astype(np.uint8),
            np.where(bad, 255, exp + 127).astype(np.uint8))


def mx_values(code, scale):
    v = VALUES[code & 7] * np.where(code >= 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int32) - 127))
    return v * np.repeat(s, 32, axis=1)


def mx_pack(code, scale):
    """Codes [R, K/2] two a byte, and the scale tiles [ceil(R/128), ceil(K/128), 512]."""
    R, KB = scale.shape
    tiles = np.zeros(((R + 127) // 128, (KB + 3) // 4, 512), np.uint8)
    for r in range(R):
        for k in range(KB):
            tiles[r // 128, k // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + k % 4] = scale[r, k]
    return code[:, 0::2] | code[:, 1::2] << 4, tiles


def mx_unpack(codes, tiles):
    R, K = codes.shape[0], 2 * codes.shape[1]
    code = np.empty((R, K), np.uint8)
    code[:, 0::2], code[:, 1::2] = codes & 15, codes >> 4
    r, k = np.arange(R)[:, None], np.arange(K // 32)[None, :]
    return code, tiles[r // 128, k // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + k % 4]


def linear_mx(x, W, bias=None, residual=None, act="none"):
    """From the operands' values; y and the sums before the activation."""
    return router.linear(x, W, bias, residual, act)
