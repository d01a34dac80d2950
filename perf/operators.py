"""Measured cases of the operators around the MoE layer of a pre-norm block: the residual
addition with its RMS norm (bf16 or MXFP8 out), the router's balance and z losses with the
per-expert counts, and the dense product with bias, activation and residual (the router's
logits, and a shared expert beside the routed ones); each forward and backward.

``run`` computes a case in its plain form (elementary torch operations in fp32, rounded
once at the end) or, where ``own`` is true, through the framework's entry points.  ``exact``
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "f32": F32}
EPS = 1e-6
BALANCE_COEF, Z_COEF = 1e-2, 1e-3


# ------------------------------------------------------------------ cases --

def _norm(name, rows, d, x="bf16", s="bf16", mx=False, pad=0):
    return {"name": name, "op": "norm_fwd", "rows": rows, "d": d, "x": x, "s": s, "mx": mx,
            "pad": pad}


def _norm_bwd(name, rows, d, dy="bf16", s="bf16", skip=True):
    return {"name": name, "op": "norm_bwd", "rows": rows, "d": d, "dy": dy, "s": s, "skip": skip}


def _balance(name, op, T, E, k, masked=0.0, dead=0):
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "masked": masked, "dead": dead}


def _linear(name, M, N, K, act="none", bias=True, residual=False, out="bf16", keep_z=False,
            pad=0):
    return {"name": name, "op": "linear_fwd", "M": M, "N": N, "K": K, "act": act, "bias": bias,
            "residual": residual, "out": out, "keep_z": keep_z, "pad": pad}


def _linear_bwd(name, M, N, K, act="none", dy="bf16", dx="bf16", bias=True):
    return {"name": name, "op": "linear_bwd", "M": M, "N": N, "K": K, "act": act, "dy": dy,
            "dx": dx, "bias": bias}


def listed():
    return [
        # one token of a serving step through the widest layer: latency
        _norm("norm_token", 1, 7168),
        # a training batch of the widest layer: the layer's fp32 output joins the bf16 stream,
        # the next layer reads the norm as MXFP8
        _norm("norm_mx_8192x7168", 8192, 7168, x="f32", mx=True),
        # the layer's fp32 dx through the norm of an fp32 stream
        _norm_bwd("norm_bwd_16384x4096_f32", 16384, 4096, dy="f32", s="f32"),
        # a width that is no multiple of the tiles, an odd number of rows
        _norm_bwd("norm_bwd_4099x2880", 4099, 2880),
        # the smallest router: launches are all there is
        _balance("balance_tiny", "balance_fwd", 256, 8, 2),
        # the batch of the imbalanced workload, padding tokens masked
        _balance("balance_16384x128", "balance_fwd", 16384, 128, 8, masked=0.06),
        # the large workload's router
        _balance("balance_bwd_8192x384", "balance_bwd", 8192, 384, 8),
        # one token through the up product of a shared expert
        _linear("linear_token", 1, 2048, 7168, act="silu"),
        # the router's logits of the fine workload, fp32
        _linear("router_logits_4096x64", 4096, 64, 2048, out="f32"),
        # the down product of a shared expert, adding to the routed output
        _linear("linear_8192x7168x2048", 8192, 7168, 2048, residual=True),
        # the up product's training step
        _linear_bwd("linear_bwd_4096x1024x2048", 4096, 1024, 2048, act="silu"),
        # the losses' logit gradient back through the router of the imbalanced workload
        _linear_bwd("router_bwd_16384x128x4096", 16384, 128, 4096, dy="f32", dx="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        if 3072 not in c.values():  # a size that nothing here has
            return c


def _draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "balance_fwd", "balance_bwd", "linear_fwd",
                     "linear_bwd"])
    kinds = ("bf16", "f32")
    if op == "norm_fwd":
        mx = rng.random() < 0.5
        d = 32 * _log(rng, 4, 256) if mx else _log(rng, 128, 8192)
        rows = _log(rng, 1, max(2, min(16384, 8192 * 7168 // d)))
        c = _norm("", rows, d, x=rng.choice(kinds), s=rng.choice(kinds), mx=mx,
                  pad=rng.choice((0, 0, 8, 1)))
    elif op == "norm_bwd":
        d = _log(rng, 128, 8192)
        rows = _log(rng, 1, max(2, min(16384, 16384 * 4096 // d)))
        c = _norm_bwd("", rows, d, dy=rng.choice(kinds), s=rng.choice(kinds),
                      skip=rng.random() < 0.7)
    elif op.startswith("balance"):
        E = _log(rng, 2, 512)
        c = _balance("", op, _log(rng, 1, 16384), E, rng.randint(1, min(8, E)),
                     masked=rng.choice((0.0, 0.1, 0.5)), dead=rng.choice((0, 0, 1)) if E > 8 else 0)
    else:
        while True:
            M, N, K = _log(rng, 1, 16384), _log(rng, 8, 7168), 8 * _log(rng, 8, 896)
            most = 8192 * 7168 * 2048
            if M * N * K <= (most if op == "linear_fwd" else most // 2):
                break
        act = rng.choice(("none", "relu", "silu", "gelu"))
        if op == "linear_fwd":
            c = _linear("", M, N, K, act=act, bias=rng.random() < 0.7,
                        residual=rng.random() < 0.5, out=rng.choice(kinds),
                        keep_z=act != "none" and rng.random() < 0.5, pad=rng.choice((0, 0, 8)))
        else:
            c = _linear_bwd("", M, N, K, act=act, dy=rng.choice(kinds), dx=rng.choice(kinds),
                            bias=rng.random() < 0.7)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs --

def _randn(g, *shape, dtype=BF16, scale=1.0, pad=0):
    """Normal values; with `pad`, the leading columns of rows that are `pad` elements longer."""
    t = torch.empty(*shape[:-1], shape[-1] + pad, device="cuda", dtype=F32)
    t.normal_(generator=g)
    if scale != 1.0:
        t *= scale
    t = t.to(dtype)
    return t[..., :shape[-1]] if pad else t


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    if c["op"] == "norm_fwd":
        return {"case": c,
                "x": _randn(g, c["rows"], c["d"], dtype=DTYPES[c["x"]], pad=c["pad"]),
                "residual": _randn(g, c["rows"], c["d"], dtype=DTYPES[c["s"]], scale=3.0),
                "weight": 1.0 + _randn(g, c["d"], dtype=F32, scale=0.1)}
    if c["op"] == "norm_bwd":
        s = DTYPES[c["s"]]
        return {"case": c,
                "dy": _randn(g, c["rows"], c["d"], dtype=DTYPES[c["dy"]]),
                "s": _randn(g, c["rows"], c["d"], dtype=s, scale=3.0),
                "ds": _randn(g, c["rows"], c["d"], dtype=s) if c["skip"] else None,
                "weight": 1.0 + _randn(g, c["d"], dtype=F32, scale=0.1)}
    if c["op"].startswith("balance"):
        T, E, k = c["T"], c["E"], c["k"]
        # uneven experts, and `dead` of them taken out of the routing
        logits = _randn(g, T, E, dtype=F32) + _randn(g, E, dtype=F32, scale=0.5)
        if c["dead"] and E - c["dead"] >= k:
            logits[:, E - c["dead"]:] = -math.inf
        idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        mask = None
        if c["masked"]:
            mask = (torch.rand(T, generator=g, device="cuda") >= c["masked"]).to(torch.uint8)
        st = {"case": c, "logits": logits, "topk_idx": idx, "mask": mask}
        if c["op"] == "balance_bwd":
            # what the forward leaves for the backward
            m = torch.ones(T, dtype=F64, device="cuda") if mask is None else mask.to(F64)
            st["lse"] = torch.logsumexp(logits.to(F64), 1).to(F32)
            st["counts"] = torch.zeros(E, dtype=F64, device="cuda").index_add_(
                0, idx.reshape(-1).long(), m.repeat_interleave(k)).to(torch.int32)
            st["n_valid"] = m.sum().to(torch.int32).reshape(1)
            st["dloss"] = 1.0 + _randn(g, 2, dtype=F32, scale=0.1)
        return st
    M, N, K = c["M"], c["N"], c["K"]
    w = _randn(g, N, K, scale=1.0 / math.sqrt(K))
    if c["op"] == "linear_fwd":
        return {"case": c, "x": _randn(g, M, K, pad=c["pad"]), "w": w,
                "bias": _randn(g, N, dtype=F32, scale=0.1) if c["bias"] else None,
                "residual": _randn(g, M, N, dtype=DTYPES[c["out"]]) if c["residual"] else None}
    dy = DTYPES[c["dy"]]
    return {"case": c, "x": _randn(g, M, K), "w": w, "dy": _randn(g, M, N, dtype=dy),
            "z": _randn(g, M, N, dtype=dy) if c["act"] != "none" else None}


# -------------------------------------------------------------------- run --

def run(state):
    c = state["case"]
    return (_run_own if own else _run_plain)(c, state)


def _run_own(c, st):
    from routing_dispatch_grouped_router_gb300 import api
    op = c["op"]
    if op == "norm_fwd":
        if c["mx"]:
            values = torch.empty(c["rows"], c["d"], dtype=BF16, device="cuda")
            s, _, _ = api.add_rmsnorm_mx(st["x"], st["weight"], st["residual"], eps=EPS,
                                         values=values)
            return [s, values]
        return list(api.add_rmsnorm(st["x"], st["weight"], st["residual"], eps=EPS))
    if op == "norm_bwd":
        return list(api.add_rmsnorm_backward(st["dy"], st["s"], st["weight"], st["ds"], eps=EPS))
    if op == "balance_fwd":
        return list(api.router_balance(st["logits"], st["topk_idx"], st["mask"],
                                       balance_coef=BALANCE_COEF, z_coef=Z_COEF))
    if op == "balance_bwd":
        return api.router_balance_backward(st["dloss"], st["logits"], st["lse"], st["counts"],
                                           st["n_valid"], c["k"], st["mask"],
                                           balance_coef=BALANCE_COEF, z_coef=Z_COEF)
    if op == "linear_fwd":
        out = api.linear(st["x"], st["w"], st["bias"], act=c["act"], residual=st["residual"],
                         out_dtype=DTYPES[c["out"]], keep_z=c["keep_z"])
        return list(out) if c["keep_z"] else out
    dx, dw, db = api.linear_backward(st["dy"], st["x"], st["w"], st["z"], act=c["act"],
                                     bias=c["bias"], dx_dtype=DTYPES[c["dx"]])
    return [dx, dw, db] if c["bias"] else [dx, dw]


def _mx_values(v):
    """MXFP8 of fp32 rows: E4M3 values times a power of two per 32 columns."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(dim=2, keepdim=True)
    shared = ((amax.view(torch.int32) >> 23) - 127 - 8).clamp(-127, 127)
    shared = torch.where(amax > 0, shared, torch.full_like(shared, -127))
    down, up = ((127 - shared) << 23).view(F32), ((127 + shared) << 23).view(F32)
    q = (b * down).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).to(F32)
    return (q * up).reshape(v.shape)


def _act(z, act):
    """(act(z), act'(z)) in fp32."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0.0), (z > 0).to(z.dtype)
    if act == "silu":
        a, da = z, 1.0
    else:  # gelu in its tanh form: z sigmoid(2 sqrt(2/pi) (z + 0.044715 z^3))
        r = 2.0 * math.sqrt(2.0 / math.pi)
        a, da = r * (z + 0.044715 * z * z * z), r * (1.0 + 3.0 * 0.044715 * z * z)
    sig = 1.0 / (1.0 + torch.exp(-a))
    return z * sig, sig + z * sig * (1.0 - sig) * da


def _run_plain(c, st):
    op = c["op"]
    if op == "norm_fwd":
        s = (st["x"].to(F32) + st["residual"].to(F32)).to(DTYPES[c["s"]])
        v = s.to(F32)  # the norm of the stream as it is stored
        n = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS) * st["weight"]
        return [s, (_mx_values(n) if c["mx"] else n).to(BF16)]
    if op == "norm_bwd":
        v, dy = st["s"].to(F32), st["dy"].to(F32)
        rstd = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
        n = v * rstd
        gr = dy * st["weight"]
        dx = rstd * (gr - n * (gr * n).mean(dim=1, keepdim=True))
        if st["ds"] is not None:
            dx = dx + st["ds"].to(F32)
        return [dx.to(DTYPES[c["s"]]), (dy * n).sum(dim=0)]
    if op == "balance_fwd":
        l, E, k = st["logits"], c["E"], c["k"]
        m = torch.ones(c["T"], device=l.device) if st["mask"] is None else st["mask"].to(F32)
        top = l.amax(dim=1, keepdim=True)
        e = torch.exp(l - top)
        z = e.sum(dim=1, keepdim=True)
        lse = (top + torch.log(z)).squeeze(1)
        n_valid = m.sum()
        n = n_valid.clamp(min=1.0)
        prob = ((e / z) * m[:, None]).sum(dim=0) / n
        counts = torch.zeros(E, dtype=torch.int32, device=l.device)
        counts.index_add_(0, st["topk_idx"].reshape(-1).long(),
                          m.to(torch.int32).repeat_interleave(k))
        f = counts.to(F32) / (n * k)
        loss = torch.stack([BALANCE_COEF * E * (f * prob).sum(),
                            Z_COEF * (m * lse * lse).sum() / n])
        return [loss, counts, prob, lse, n_valid.to(torch.int32).reshape(1)]
    if op == "balance_bwd":
        l, E, k = st["logits"], c["E"], c["k"]
        n = st["n_valid"].to(F32).clamp(min=1.0)
        prob = torch.exp(l - st["lse"][:, None])
        a = st["dloss"][0] * BALANCE_COEF * E * (st["counts"].to(F32) / (n * k)) / n
        zc = st["dloss"][1] * 2.0 * Z_COEF * st["lse"] / n
        dl = prob * (a - (prob * a).sum(dim=1, keepdim=True) + zc[:, None])
        return dl if st["mask"] is None else dl * st["mask"].to(F32)[:, None]
    if op == "linear_fwd":
        z = st["x"].to(F32) @ st["w"].to(F32).t()
        if st["bias"] is not None:
            z = z + st["bias"]
        y = _act(z, c["act"])[0]
        if st["residual"] is not None:
            y = y + st["residual"].to(F32)
        out = DTYPES[c["out"]]
        return [y.to(out), z.to(out)] if c["keep_z"] else y.to(out)
    dz = st["dy"].to(F32)
    if st["z"] is not None:
        dz = dz * _act(st["z"].to(F32), c["act"])[1]
    dx = (dz @ st["w"].to(F32)).to(DTYPES[c["dx"]])
    dw = dz.t() @ st["x"].to(F32)
    return [dx, dw, dz.sum(dim=0)] if c["bias"] else [dx, dw]


# ------------------------------------------------------------------- work --

def _size(kind):
    return 4 if kind == "f32" else 2


def work(case):
    c = case
    op = c["op"]
    if op == "norm_fwd":
        n = c["rows"] * c["d"]
        # x and the stream in, the stream and the norm out (MXFP8: values, codes and scales)
        b = n * (_size(c["x"]) + 2 * _size(c["s"]) + 2) + 4 * c["d"]
        return {"bytes": b + (n + n // 32 if c["mx"] else 0), "flops": 6 * n}
    if op == "norm_bwd":
        n = c["rows"] * c["d"]
        b = n * (_size(c["dy"]) + _size(c["s"]) * (3 if c["skip"] else 2)) + 8 * c["d"]
        return {"bytes": b, "flops": 12 * n}
    if op == "balance_fwd":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 4 * T * (E + k + 1) + (T if c["masked"] else 0) + 8 * E, "flops": 5 * T * E}
    if op == "balance_bwd":
        T, E = c["T"], c["E"]
        return {"bytes": 4 * T * (2 * E + 1) + (T if c["masked"] else 0) + 4 * E, "flops": 6 * T * E}
    M, N, K = c["M"], c["N"], c["K"]
    if op == "linear_fwd":
        o = _size(c["out"])
        outs = o * M * N * (1 + int(c["residual"]) + int(c["keep_z"]))
        return {"bytes": 2 * (M * K + N * K) + outs + (4 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    dy = _size(c["dy"]) * M * N * (2 if c["act"] != "none" else 1)
    return {"bytes": dy + 2 * (M * K + N * K) + _size(c["dx"]) * M * K + 4 * N * K
            + (4 * N if c["bias"] else 0), "flops": 4 * M * N * K}


# ------------------------------------------------------------------ exact --

def _e4m3(v):
    """The nearest E4M3 value (ties to even, 448 at most) of 64-bit values."""
    _, e = torch.frexp(v.abs())
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    op = c["op"]
    if op == "norm_fwd":
        s = (st["x"].to(F64) + st["residual"].to(F64)).to(DTYPES[c["s"]])
        v = s.to(F64)
        n = st["weight"].to(F64) * v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / c["d"] + EPS)
        if c["mx"]:
            b = n.unflatten(1, (c["d"] // 32, 32))
            _, e = torch.frexp(b.abs().amax(2, keepdim=True))
            sc = torch.ldexp(torch.ones_like(b[..., :1]), (e - 9).clamp(-127, 127))
            n = (_e4m3(b / sc) * sc).flatten(1)
        return [s.to(F64), n]
    if op == "norm_bwd":
        v, dy, w = st["s"].to(F64), st["dy"].to(F64), st["weight"].to(F64)
        ms = v.pow(2).sum(1, keepdim=True) / c["d"] + EPS
        dot = (dy * w * v).sum(1, keepdim=True)
        dx = dy * w / ms.sqrt() - v * dot / (c["d"] * ms * ms.sqrt())
        if st["ds"] is not None:
            dx += st["ds"].to(F64)
        return [dx, (dy * v / ms.sqrt()).sum(0)]
    if op.startswith("balance"):
        l, E, k = st["logits"].to(F64), c["E"], c["k"]
        m = torch.ones(c["T"], dtype=F64, device=l.device) if st["mask"] is None \
            else st["mask"].to(F64)
        n = max(float(m.sum()), 1.0)
        p = torch.softmax(l, dim=1)
        if op == "balance_fwd":
            lse = torch.logsumexp(l, dim=1)
            counts = torch.bincount(st["topk_idx"][m > 0].reshape(-1).long(), minlength=E)
            prob = m @ p / n
            loss = torch.stack([BALANCE_COEF * E / (n * k) * (counts.to(F64) @ prob),
                                Z_COEF * (m @ lse.pow(2)) / n])
            return [loss, counts.to(torch.int32), prob, lse, m.sum().to(torch.int32).reshape(1)]
        # the derivative of the two losses, with the counts held constant
        f = st["counts"].to(F64) / (n * k)
        up = st["dloss"].to(F64)
        lse = st["lse"].to(F64)[:, None]
        balance = up[0] * BALANCE_COEF * E / n * p * (f - (p @ f)[:, None])
        return (balance + up[1] * 2 * Z_COEF / n * lse * p) * m[:, None]
    x, w = st["x"].to(F64), st["w"].to(F64)

    def act(z):  # value and derivative
        t = {"none": lambda: torch.full_like(z, math.inf), "relu": lambda: z * math.inf,
             "silu": lambda: z,
             "gelu": lambda: math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)}[c["act"]]()
        h = torch.sigmoid(torch.nan_to_num(t, nan=-math.inf, posinf=math.inf, neginf=-math.inf))
        slope = {"silu": lambda: 1.0,
                 "gelu": lambda: math.sqrt(8 / math.pi) * (1 + 0.134145 * z ** 2)}
        if c["act"] in slope:
            return z * h, h + z * h * (1 - h) * slope[c["act"]]()
        return z * h, h

    if op == "linear_fwd":
        z = x @ w.T
        if st["bias"] is not None:
            z += st["bias"].to(F64)
        y = act(z)[0]
        if st["residual"] is not None:
            y = y + st["residual"].to(F64)
        return [y, z] if c["keep_z"] else y
    dz = st["dy"].to(F64)
    if st["z"] is not None:
        dz = dz * act(st["z"].to(F64))[1]
    return [dz @ w, dz.T @ x, dz.sum(0)] if c["bias"] else [dz @ w, dz.T @ x]
