"""Measured cases of the block norm and the MXFP4 row operators.

Operators around a block (routed experts, a dense expert beside them) of a residual stream:

* ``norm``       the norm after a block, its gate, the scaled residual add and the norm before the
                 next block: xn = alpha x + gate (norm(o) . post), h = norm(xn) . pre; h also as
                 MXFP4 rows.
* ``norm_grad``  its gradients: dx, do, dgate, dpre, dpost from dxn and dh.
* ``quant``      rows to MXFP4 (OCP Microscaling: 4-bit E2M1 elements, a power of two for each 32 of
                 them) and back.
* ``linear``     act(x W^T + b) + residual with both operands in MXFP4, x quantised by the call or
                 in MXFP4 already.

``run`` computes a case in plain 32-bit torch operations, or, where ``own`` is set, through the
package's entry points.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
_EPS = 1e-6


# ---- the cases --------------------------------------------------------------


def _norm(name, T, d, **kw):
    c = {"name": name, "op": "norm", "T": T, "d": d, "stream": "bf16", "block": "bf16", "o": True,
         "pre": True, "post_norm": True, "post": True, "gate": "none", "alpha": 1.0, "masked": 0.0,
         "pad": 0, "mx": False}
    return {**c, **kw}


def _quant(name, T, K, **kw):
    return {"name": name, "op": "quant", "T": T, "K": K, "dtype": "bf16", "pad": 0, **kw}


def _lin(name, T, K, N, **kw):
    c = {"name": name, "op": "linear", "T": T, "K": K, "N": N, "dtype": "bf16", "given": "rows",
         "out": "bf16", "act": "none", "bias": False, "residual": False, "pad": 0}
    return {**c, **kw}


def listed():
    return [
        # one decoded token between two blocks: latency counts
        _norm("norm, one token", 1, 2560),
        # a prefill chunk with a gate for each token, h also in 4 bits for the dense expert
        _norm("norm + MXFP4, chunk of 2048", 2048, 2560, gate="sigmoid", alpha=0.5, mx=True),
        # a long prompt, residual stream kept in 32 bits, padded tokens
        _norm("norm, f32 stream, 32768", 32768, 2816, stream="f32", masked=0.1),
        # odd everything: half precision rows of a wider tensor, no norm of the block's output
        _norm("norm, ragged half", 777, 1001, stream="f16", block="f16", post_norm=False,
              gate="plain", alpha=0.7, pad=24),
        # a training chunk, every gradient
        _norm("norm gradients, 2048", 2048, 2560, op="norm_grad", gate="sigmoid", alpha=0.5),
        # a long training batch
        _norm("norm gradients, 32768", 32768, 2816, op="norm_grad", masked=0.1),
        # the hidden rows of a dense expert, quantised and read back
        _quant("quantise + read, 4096", 4096, 11264),
        # up projection of one decoded token: the weights are read once, latency counts
        _lin("up + GELU, one token", 1, 2560, 10240, act="gelu_tanh"),
        # down projection with the residual add for a batch of 16 decoded tokens
        _lin("down + residual, 16 tokens", 16, 10240, 2560, residual=True),
        # odd everything: half precision, rows of a wider tensor, K that ends inside a tile
        _lin("ragged half precision", 777, 1056, 1001, dtype="f16", out="f16", act="silu",
             bias=True, residual=True, pad=24),
        # up projection of a long-prompt chunk, quantised by the call
        _lin("up + GELU, chunk of 4096", 4096, 2816, 11264, act="gelu_tanh"),
        # down projection of rows that are in 4 bits already, into a 32-bit residual stream
        _lin("down, MXFP4 rows, 4096", 4096, 11264, 2816, given="mx", out="f32", residual=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_grad", "norm_grad", "quant", "linear", "linear", "linear"))
    if op.startswith("norm"):
        d = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:  # most models' widths
            d = max(64, d // 64 * 64)
        T = min(_log_int(rng, 1, 32768), 32768 * 2816 // d)
        stream, block = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("f16", "f16"),
                                    ("f32", "bf16"), ("f32", "f16"), ("f32", "f32")))
        o = op == "norm_grad" or rng.random() < 0.8
        c = _norm("", T, d, op=op, stream=stream, block=block, o=o, pre=not o or rng.random() < 0.8,
                  post_norm=rng.random() < 0.6, post=rng.random() < 0.7,
                  gate=rng.choice(("none", "plain", "sigmoid")), alpha=rng.choice((1.0, 0.5)),
                  masked=rng.choice((0.0, 0.0, 0.1, 0.5)), pad=rng.choice((0, 0, 8, 24)))
        c["mx"] = op == "norm" and c["pre"] and d % 32 == 0 and rng.random() < 0.5
    elif op == "quant":
        K = 32 * _log_int(rng, 2, 352)
        c = _quant("", min(_log_int(rng, 1, 16384), 4096 * 11264 // K), K,
                   dtype=rng.choice(("bf16", "bf16", "f16", "f32")), pad=rng.choice((0, 0, 8, 24)))
    else:
        K, N = 32 * _log_int(rng, 2, 352), _log_int(rng, 3, 11264)
        T = min(_log_int(rng, 1, 4096), 4096 * 2816 * 11264 // (K * N))
        dt = rng.choice(("bf16", "bf16", "f16"))
        c = _lin("", T, K, N, dtype=dt, given=rng.choice(("rows", "rows", "mx")),
                 out=rng.choice((dt, dt, "f32")), act=rng.choice(_ACTS), bias=rng.random() < 0.5,
                 residual=rng.random() < 0.5, pad=rng.choice((0, 0, 8, 40)))
    del c["name"]
    return c


# ---- MXFP4 rows -------------------------------------------------------------
#
# Codes [R, K/2]: element 2i in the low half of byte i.  Scales: bytes 2^(S - 127) of blocks of 32
# along K, in tiles of 128 rows x 4 blocks, [ceil(R/128), ceil(K/128), 512]: row 32 q + l, block b
# of a tile at byte 16 l + 4 q + b.  What is past the last row and block is 0.


def _pow2(x):
    """2^x in 32 bits, exactly (pow and ldexp need not be), x = -127 ... 127."""
    x = x.to(torch.int32)
    normal = ((x.clamp(min=-126) + 127) << 23).view(torch.float32)
    return torch.where(x < -126, 2.0 ** -127, normal)


def _mx_encode(v):
    """E2M1 codes [R, K] and scale bytes [R, K/32] of 32-bit rows."""
    R, K = v.shape
    b = v.reshape(R, K // 32, 32)
    bad = ~torch.isfinite(b).all(2)
    b = torch.where(bad[:, :, None], 0.0, b)
    top = torch.frexp(b.abs().amax(2))
    x = torch.where(top.mantissa == 0, -127, top.exponent - 3).clamp(-127, 127)
    a = b.abs() * _pow2(-x)[:, :, None]
    # the points between neighbouring magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6; a tie goes to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = code + 8 * torch.signbit(b).to(torch.uint8)
    return code.reshape(R, K), torch.where(bad, 255, x + 127).to(torch.uint8)


def _mx_values(code, scale, dtype=torch.float32):
    """What codes [R, K] and scale bytes [R, K/32] stand for."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=dtype, device=code.device)
    v = lut[(code & 7).long()]
    v = torch.where(code >= 8, -v, v)
    s = torch.where(scale == 255, float("nan"), _pow2(scale.int().clamp(max=254) - 127)).to(dtype)
    return v * s.repeat_interleave(32, 1)


def _mx_pack(code, scale):
    R, KB = scale.shape
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    RT, KT = -(-R // 128), -(-KB // 4)
    full = torch.zeros(RT * 128, KT * 4, dtype=torch.uint8, device=code.device)
    full[:R, :KB] = scale
    tiles = full.reshape(RT, 4, 32, KT, 4).permute(0, 3, 2, 1, 4).reshape(RT, KT, 512)
    return codes.contiguous(), tiles.contiguous()


def _mx_unpack(codes, tiles):
    R, K = codes.shape[0], 2 * codes.shape[1]
    RT, KT = tiles.shape[:2]
    code = torch.stack((codes & 15, codes >> 4), 2).reshape(R, K)
    scale = tiles.reshape(RT, KT, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(RT * 128, KT * 4)
    return code, scale[:R, :K // 32]


# ---- inputs -----------------------------------------------------------------


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(g, T, K, pad, dtype, amp=1.0):
    """[T, K] rows, with pad > 0 the first K columns of a wider tensor."""
    return (amp * _randn(g, T, K + pad)).to(dtype)[:, :K]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    T, pad = case["T"], case["pad"]
    if case["op"].startswith("norm"):
        d, S, B = case["d"], _DT[case["stream"]], _DT[case["block"]]
        # a residual stream has a few wide channels
        wide = 1 + 20 * (torch.rand(d, generator=g, device="cuda") < 0.004)
        s["x"] = _rows(g, T, d, pad, S, 2 * torch.cat((wide, wide.new_ones(pad))))
        s["o"] = _rows(g, T, d, pad, B, 0.5) if case["o"] else None
        s["w_pre"] = 1 + 0.2 * _randn(g, d) if case["pre"] else None
        s["w_post"] = 0.5 + 0.1 * _randn(g, d) if case["post"] and case["o"] else None
        s["gate_t"] = _randn(g, T) if case["gate"] != "none" and case["o"] else None
        s["mask"] = None
        if case["masked"]:  # padding: these rows hold anything
            s["mask"] = torch.rand(T, generator=g, device="cuda") >= case["masked"]
            s["x"][~s["mask"]] = float("nan")
            if s["o"] is not None:
                s["o"][~s["mask"]] = float("inf")
        if case["op"] == "norm_grad":
            # gradients as large as a mean loss's (fp16: with its loss scale)
            amp = 1e-2 if "f16" in (case["stream"], case["block"]) else 1e-4
            s["dxn"] = _rows(g, T, d, pad, S, amp)
            s["dh"] = _rows(g, T, d, pad, B, amp) if case["pre"] else None
            s["xn"] = _norm_plain({**s, "mx": False, "pre": False})["xn"]
            if s["mask"] is not None:
                s["dxn"][~s["mask"]] = float("nan")
            del s["x"]
        return s
    dt = _DT[case["dtype"]]
    K = case["K"]
    s["x"] = _rows(g, T, K, pad, dt)
    s["x"][:, ::97] *= 12  # channels far wider than the others of their blocks
    s["x"][::5, 32:64] = 0.0  # and blocks of zeros
    if case["op"] == "quant":
        return s
    if case["given"] == "mx":
        s["x_codes"], s["x_scales"] = _mx_pack(*_mx_encode(s["x"].float()))
        del s["x"]
    N, out = case["N"], _DT[case["out"]]
    # the weights in MXFP4, laid out once
    s["w_codes"], s["w_scales"] = _mx_pack(*_mx_encode(0.02 * _randn(g, N, K)))
    s["b"] = 0.1 * _randn(g, N) if case["bias"] else None
    s["r"] = _rows(g, T, N, pad, out) if case["residual"] else None
    return s


# ---- plain forms ------------------------------------------------------------


def _live(s, v):
    """32-bit rows, 0 where the mask is."""
    v = v.float()
    return v if s["mask"] is None else torch.where(s["mask"][:, None], v, 0.0)


def _rms(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + _EPS)


def _gate(s):
    g = s["gate_t"][:, None]
    return 1 / (1 + torch.exp(-g)) if s["gate"] == "sigmoid" else g


def _norm_plain(s):
    xn = _live(s, s["x"])
    out = {}
    if s["o"] is not None:
        n = _live(s, s["o"])
        if s["post_norm"]:
            n = n * _rms(n)
        if s["w_post"] is not None:
            n = n * s["w_post"]
        if s["gate_t"] is not None:
            n = n * _gate(s)
        out["xn"] = (s["alpha"] * xn + n).to(s["x"].dtype)
        xn = out["xn"].float()
    if s["pre"]:
        out["h"] = (xn * _rms(xn) * s["w_pre"]).to(_DT[s["block"]])
    if s["mx"]:
        out["mx"] = _mx_values(*_mx_encode(out["h"].float())).to(torch.bfloat16)
    return out


def _norm_grad_plain(s):
    xn, o, ds = _live(s, s["xn"]), _live(s, s["o"]), _live(s, s["dxn"])
    out = {}
    if s["pre"]:
        dh, r2 = _live(s, s["dh"]), _rms(xn)
        a = dh * s["w_pre"]
        ds = ds + r2 * a - r2 ** 3 * (a * xn).mean(1, keepdim=True) * xn
        out["dpre"] = (dh * xn * r2).sum(0)
    out["dx"] = (s["alpha"] * ds).to(s["xn"].dtype)
    r1 = _rms(o) if s["post_norm"] else 1.0
    n = o * r1
    dn = ds
    if s["gate_t"] is not None:
        g = _gate(s)
        u = n if s["w_post"] is None else n * s["w_post"]
        dg = (ds * u).sum(1)
        out["dgate"] = dg * (g * (1 - g))[:, 0] if s["gate"] == "sigmoid" else dg
        dn = ds * g
    if s["w_post"] is not None:
        out["dpost"] = (dn * n).sum(0)
        dn = dn * s["w_post"]
    if s["post_norm"]:
        dn = r1 * dn - r1 ** 3 * (dn * o).mean(1, keepdim=True) * o
    out["do"] = dn.to(s["o"].dtype)
    return out


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


def _quant_plain(s):
    return {"values": _mx_values(*_mx_encode(s["x"].float())).to(torch.bfloat16)}


def _linear_plain(s):
    if s["given"] == "mx":
        x = _mx_values(*_mx_unpack(s["x_codes"], s["x_scales"]))
    else:
        x = _mx_values(*_mx_encode(s["x"].float()))
    z = x @ _mx_values(*_mx_unpack(s["w_codes"], s["w_scales"])).t()
    if s["b"] is not None:
        z = z + s["b"]
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(_DT[s["out"]])}


# ---- one pass ---------------------------------------------------------------


def _run_own(s):
    from moe_prefill_routing_gb300 import binding as B

    op = s["op"]
    if op == "norm":
        r = B.block_norm(s["x"], s["o"], pre=s["w_pre"], post=s["w_post"], gate=s["gate_t"],
                         mask=s["mask"], post_norm=s["post_norm"],
                         gate_act="sigmoid" if s["gate"] == "sigmoid" else "none",
                         alpha=s["alpha"], eps=_EPS, h_dtype=_DT[s["block"]], mxfp4=s["mx"])
        out = {n: r[n] for n in ("xn", "h") if n in r and (n == "h" or s["o"] is not None)}
        if s["mx"]:
            out["mx"] = B.dequantize_rows_mxfp4(r["mx"])
        return out
    if op == "norm_grad":
        r = B.block_norm_grad(s["xn"], s["o"], dxn=s["dxn"], dh=s["dh"], pre=s["w_pre"],
                              post=s["w_post"], gate=s["gate_t"], mask=s["mask"],
                              post_norm=s["post_norm"],
                              gate_act="sigmoid" if s["gate"] == "sigmoid" else "none",
                              alpha=s["alpha"], eps=_EPS)
        return {n: r[n] for n in ("dx", "do", "dgate", "dpre", "dpost") if n in r}
    if op == "quant":
        return {"values": B.dequantize_rows_mxfp4(B.quantize_rows_mxfp4(s["x"]))}
    x = s["x"] if s["given"] == "rows" else B.Mxfp4Rows(s["x_codes"], s["x_scales"])
    return {"y": B.linear_mxfp4(x, B.Mxfp4Rows(s["w_codes"], s["w_scales"]), bias=s["b"],
                                residual=s["r"], act=s["act"], out_dtype=_DT[s["out"]])}


_PLAIN = {"norm": _norm_plain, "norm_grad": _norm_grad_plain, "quant": _quant_plain,
          "linear": _linear_plain}


def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    c = case
    size = {"bf16": 2, "f16": 2, "f32": 4}
    T = c["T"]
    if c["op"].startswith("norm"):
        b, k = size[c["stream"]], size[c["block"]]
        weights = 4 * c["d"] * (c["pre"] + (c["post"] and c["o"]))
        rows = T * (4 if c["gate"] != "none" and c["o"] else 0) + T * (1 if c["masked"] else 0)
        if c["op"] == "norm":
            n = b + (b + k if c["o"] else 0) + (k if c["pre"] else 0) + (2 if c["mx"] else 0)
            return {"bytes": T * c["d"] * n + weights + rows, "flops": 12.0 * T * c["d"]}
        n = 3 * b + 2 * k + (k if c["pre"] else 0)
        return {"bytes": T * c["d"] * n + 2 * weights + 2 * rows, "flops": 30.0 * T * c["d"]}
    K, b = c["K"], size[c["dtype"]]
    if c["op"] == "quant":
        return {"bytes": T * K * (b + 2), "flops": 10.0 * T * K}
    N, o = c["N"], size[c["out"]]
    n = T * K * (17 / 32 if c["given"] == "mx" else b) + N * K * 17 / 32 + 4 * N * bool(c["bias"])
    return {"bytes": n + T * N * o * (2 if c["residual"] else 1), "flops": 2.0 * T * K * N}


# ---- the definitions in 64 bits ---------------------------------------------


def _quantised64(v):
    """Rows to MXFP4 and back, in 64 bits: the nearest of the sixteen values of each block, of two
    equally near ones that with the even code."""
    b = v.double().reshape(v.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    x = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
    step = ((x.long() + 1023) << 52).view(torch.float64)  # 2^x
    a = b.abs() / step
    # spacing of the magnitudes: 0.5 below 2, 1 below 4, then 2; round() takes ties to even
    gap = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / gap) * gap).clamp(max=6.0)
    return (torch.copysign(q, b) * step).reshape(v.shape)


def _kept64(s, v):
    v = v.double()
    return v if s["mask"] is None else v.masked_fill(~s["mask"][:, None], 0.0)


def _norm64(s, x, o, w_pre, w_post, gate, alpha):
    """s (not rounded) and a function of the stream that gives h."""
    def unit(v):
        return v / (v.square().mean(1, keepdim=True) + _EPS).sqrt()

    if o is not None:
        n = unit(o) if s["post_norm"] else o
        if w_post is not None:
            n = n * w_post
        if gate is not None:
            n = n * (torch.sigmoid(gate) if s["gate"] == "sigmoid" else gate)[:, None]
        x = alpha * x + n
    return x, (lambda xn: unit(xn) * w_pre)


def _d(v):
    return None if v is None else v.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        o = None if s["o"] is None else _kept64(s, s["o"])
        x, norm = _norm64(s, _kept64(s, s["x"]), o, _d(s["w_pre"]), _d(s["w_post"]),
                          _d(s["gate_t"]), s["alpha"])
        out = {}
        if o is not None:
            out["xn"] = x
            x = x.to(s["x"].dtype).double()  # h is of the stream as it is stored
        if s["pre"]:
            out["h"] = norm(x)
        if s["mx"]:
            out["mx"] = _quantised64(out["h"].to(_DT[s["block"]]))
        return out
    if case["op"] == "norm_grad":
        live = slice(None) if s["mask"] is None else s["mask"]
        full = lambda v, like: torch.zeros(like.shape, dtype=torch.float64,  # noqa: E731
                                           device="cuda").index_put_((torch.arange(
                                               like.shape[0], device="cuda")[live],), v)
        # of a sum of both halves: x = 0 stands for the stream below, which dS does not depend on
        o = s["o"].double()[live].requires_grad_(True)
        xn = s["xn"].double()[live].requires_grad_(True)
        wp, wq = _d(s["w_pre"]), _d(s["w_post"])
        gate = None if s["gate_t"] is None else s["gate_t"].double()[live].requires_grad_(True)
        wq = None if wq is None else wq.requires_grad_(True)
        ds, out = s["dxn"].double()[live], {}
        if s["pre"]:
            wp.requires_grad_(True)
            h = _norm64(s, xn, None, wp, None, None, 1.0)[1](xn)
            more, out["dpre"] = torch.autograd.grad(h, (xn, wp), s["dh"].double()[live])
            ds = ds + more
        out["dx"] = full(s["alpha"] * ds, s["xn"])
        z, _ = _norm64(s, torch.zeros_like(o), o, None, wq, gate, s["alpha"])
        of = [v for v in (o, wq, gate) if v is not None]
        got = list(torch.autograd.grad(z, of, ds))
        out["do"] = full(got.pop(0), s["xn"])
        if wq is not None:
            out["dpost"] = got.pop(0)
        if gate is not None:
            out["dgate"] = full(got.pop(0), s["gate_t"])
        return out
    if case["op"] == "quant":
        return {"values": _quantised64(s["x"])}
    if case["given"] == "mx":
        x = _mx_values(*_mx_unpack(s["x_codes"], s["x_scales"]), dtype=torch.float64)
    else:
        x = _quantised64(s["x"])
    w = _mx_values(*_mx_unpack(s["w_codes"], s["w_scales"]), dtype=torch.float64)
    z = torch.einsum("tk,nk->tn", x, w)
    z = z if s["b"] is None else z + s["b"].double()
    f = torch.nn.functional
    z = {"none": lambda v: v, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
         "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[case["act"]](z)
    return {"y": z if s["r"] is None else z + s["r"].double()}
