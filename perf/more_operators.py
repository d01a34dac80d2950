"""Measured cases of what a model does between the router and the next block, beside the fused
layer: products grouped by expert over ragged rows, dropout on a branch, and the norms after and
before a block with its gate and residual scale; each forward and backward.

``run`` computes a case in its plain form (elementary torch operations in fp32, rounded once at
the end) or, where ``own`` is true, through the framework's entry points.  ``exact`` gives the
same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "f32": F32}
EPS = 1e-6
SITE = 5  # the dropout's place in the model


# ------------------------------------------------------------------ cases --

def _drop(name, op, rows, d, p, x="bf16", y="bf16", residual=False, pad=0):
    return {"name": name, "op": op, "rows": rows, "d": d, "p": p, "x": x, "y": y,
            "residual": residual, "pad": pad}


def _norms(name, rows, d, x="bf16", s="bf16", gate="none", alpha=1.0, pad=0):
    return {"name": name, "op": "norms_fwd", "rows": rows, "d": d, "x": x, "s": s, "gate": gate,
            "alpha": alpha, "pad": pad}


def _norms_bwd(name, rows, d, x="bf16", s="bf16", dy="bf16", gate="none", alpha=1.0, skip=True):
    return {"name": name, "op": "norms_bwd", "rows": rows, "d": d, "x": x, "s": s, "dy": dy,
            "gate": gate, "alpha": alpha, "skip": skip}


def _grouped(name, op, rows, E, N, K, out="bf16", split="even"):
    return {"name": name, "op": op, "rows": rows, "E": E, "N": N, "K": K, "out": out,
            "split": split}


def listed():
    return [
        # a small batch's branch: launches are all there is
        _drop("drop_64x2048", "drop_fwd", 64, 2048, 0.1),
        # a training batch of the widest layer: its fp32 output, dropped, joins the bf16 stream
        _drop("drop_8192x7168", "drop_fwd", 8192, 7168, 0.1, x="f32", residual=True),
        # the gradient of a branch whose rows have an odd length
        _drop("drop_bwd_4099x2881", "drop_bwd", 4099, 2881, 0.25),
        # one token of a serving step through the widest layer: latency
        _norms("norms_token", 1, 7168, gate="channel"),
        # a training batch of the widest layer: fp32 branch, bf16 stream, a gate per token
        _norms("norms_8192x7168", 8192, 7168, x="f32", gate="token", alpha=0.9),
        # the training step between two blocks of an fp32 stream
        _norms_bwd("norms_bwd_16384x4096_f32", 16384, 4096, x="f32", s="f32"),
        # a width that is no multiple of the tiles, an odd number of rows, a gate per channel
        _norms_bwd("norms_bwd_4099x2880", 4099, 2880, gate="channel", alpha=0.5),
        # one token at eight experts: the weights' bytes are all there is
        _grouped("grouped_token", "grouped_fwd", 8, 128, 4096, 1536, split="one"),
        # a serving batch of 40 tokens at eight of 64 experts
        _grouped("grouped_decode_320", "grouped_fwd", 320, 64, 2048, 2048),
        # the down product of a training batch whose experts are very unevenly loaded
        _grouped("grouped_131072_zipf", "grouped_fwd", 131072, 128, 4096, 1536, split="zipf"),
        # the training step of the up product, evenly loaded
        _grouped("grouped_bwd_32768", "grouped_bwd", 32768, 64, 2048, 2048),
        # odd widths, groups that end inside every tile, some of them empty, fp32 dx
        _grouped("grouped_bwd_5003", "grouped_bwd", 5003, 24, 1400, 2888, out="f32",
                 split="zipf"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST = 131072 * 4096 * 1536  # products of the largest listed case
MOST_WEIGHTS = 128 * 4096 * 1536


def draw(rng):
    op = rng.choice(["drop_fwd", "drop_bwd", "norms_fwd", "norms_bwd", "grouped_fwd",
                     "grouped_bwd"])
    kinds = ("bf16", "f32")
    if op.startswith("drop"):
        d = _log(rng, 1, 8192)
        rows = _log(rng, 1, max(2, min(16384, 8192 * 7168 // d)))
        c = _drop("", op, rows, d, rng.choice((0.05, 0.1, 0.3, 0.5)), x=rng.choice(kinds),
                  y=rng.choice(kinds), residual=op == "drop_fwd" and rng.random() < 0.6,
                  pad=rng.choice((0, 0, 8, 1)))
    elif op == "norms_fwd":
        d = _log(rng, 128, 8192)
        rows = _log(rng, 1, max(2, min(16384, 8192 * 7168 // d)))
        c = _norms("", rows, d, x=rng.choice(kinds), s=rng.choice(kinds),
                   gate=rng.choice(("none", "channel", "token")), alpha=rng.choice((1.0, 0.7)),
                   pad=rng.choice((0, 0, 8, 1)))
    elif op == "norms_bwd":
        d = _log(rng, 128, 8192)
        rows = _log(rng, 1, max(2, min(16384, 16384 * 4096 // d)))
        c = _norms_bwd("", rows, d, x=rng.choice(kinds), s=rng.choice(kinds),
                       dy=rng.choice(kinds), gate=rng.choice(("none", "channel", "token")),
                       alpha=rng.choice((1.0, 0.7)), skip=rng.random() < 0.7)
    else:
        most, weights = MOST, MOST_WEIGHTS
        if op == "grouped_bwd":  # two products, and fp32 weight gradients
            most, weights = most // 2, weights // 2
        while True:
            E, N, K = _log(rng, 1, 384), 8 * _log(rng, 8, 896), 8 * _log(rng, 8, 896)
            rows = _log(rng, 1, 131072)
            if rows * N * K <= most and E * N * K <= weights and rows * max(N, K) <= 1 << 29:
                break
        c = _grouped("", op, rows, E, N, K, out=rng.choice(kinds),
                     split=rng.choice(("even", "zipf")))
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


def _shares(c):
    """Each expert's share of the rows, before the seed orders them."""
    E = c["E"]
    w = [1.0 / (i + 1) for i in range(E)] if c["split"] == "zipf" else [1.0] * E
    t = sum(w)
    return [v / t for v in w]


def _sizes(c, seed):
    """Rows of each expert."""
    r = random.Random(seed)
    E, rows = c["E"], c["rows"]
    n = [0] * E
    if c["split"] == "one":  # one token: its experts are distinct
        for e in r.sample(range(E), rows):
            n[e] = 1
        return n
    shares = _shares(c)
    r.shuffle(shares)
    for e in r.choices(range(E), weights=shares, k=rows):
        n[e] += 1
    return n


def _gate(c, g):
    """(gate, its shape: per channel, or one per token)."""
    if c["gate"] == "none":
        return None
    shape = (c["d"],) if c["gate"] == "channel" else (c["rows"], 1)
    return 0.5 + _randn(g, *shape, dtype=F32, scale=0.2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    op = c["op"]
    if op.startswith("drop"):
        return {"case": c, "x": _randn(g, c["rows"], c["d"], dtype=DTYPES[c["x"]], pad=c["pad"]),
                "residual": _randn(g, c["rows"], c["d"], dtype=DTYPES[c["y"]], scale=3.0)
                if c["residual"] else None,
                # what a training program keeps: the seed and the step's number
                "rng": torch.tensor([(seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 63), 17 + seed],
                                    dtype=torch.int64, device="cuda")}
    if op.startswith("norms"):
        rows, d, s = c["rows"], c["d"], DTYPES[c["s"]]
        st = {"case": c, "x": _randn(g, rows, d, dtype=DTYPES[c["x"]], pad=c.get("pad", 0)),
              "post": 1.0 + _randn(g, d, dtype=F32, scale=0.1),
              "pre": 1.0 + _randn(g, d, dtype=F32, scale=0.1), "gate": _gate(c, g)}
        if op == "norms_fwd":
            st["residual"] = _randn(g, rows, d, dtype=s, scale=3.0)
        else:
            st["s"] = _randn(g, rows, d, dtype=s, scale=3.0)
            st["dy"] = _randn(g, rows, d, dtype=DTYPES[c["dy"]])
            st["ds"] = _randn(g, rows, d, dtype=s) if c["skip"] else None
        return st
    n = _sizes(c, seed)
    off = [0]
    for v in n:
        off.append(off[-1] + v)
    w = torch.empty(c["E"], c["N"], c["K"], device="cuda", dtype=BF16)
    w.normal_(std=1.0 / math.sqrt(c["K"]), generator=g)
    st = {"case": c, "x": _randn(g, c["rows"], c["K"]), "w": w, "bounds": off,
          "offsets": torch.tensor(off, dtype=torch.int32, device="cuda")}
    if op == "grouped_bwd":
        st["dy"] = _randn(g, c["rows"], c["N"])
    return st


# -------------------------------------------------------------------- run --

def run(state):
    c = state["case"]
    return (_run_own if own else _run_plain)(c, state)


def _run_own(c, st):
    from routing_dispatch_grouped_router_gb300 import api
    op = c["op"]
    if op == "drop_fwd":
        return api.dropout(st["x"], c["p"], st["rng"], SITE, residual=st["residual"],
                           out_dtype=DTYPES[c["y"]])
    if op == "drop_bwd":
        return api.dropout_backward(st["x"], c["p"], st["rng"], SITE, dx_dtype=DTYPES[c["y"]])
    if op == "norms_fwd":
        return list(api.post_pre_rmsnorm(st["x"], st["residual"], st["post"], st["pre"],
                                         st["gate"], residual_scale=c["alpha"], eps=EPS))
    if op == "norms_bwd":
        out = api.post_pre_rmsnorm_backward(st["dy"], st["x"], st["s"], st["post"], st["pre"],
                                            st["gate"], st["ds"], residual_scale=c["alpha"],
                                            eps=EPS)
        return list(out if st["gate"] is not None else out[:4])
    if op == "grouped_fwd":
        return api.grouped_linear(st["x"], st["w"], st["offsets"], out_dtype=DTYPES[c["out"]])
    return list(api.grouped_linear_backward(st["dy"], st["x"], st["w"], st["offsets"],
                                            dx_dtype=DTYPES[c["out"]]))


def _philox(rng, blocks, device):
    """Philox4x32-10 (Salmon et al. 2011) of blocks 0 .. blocks - 1: int64 [blocks, 4]."""
    low = 0xFFFFFFFF
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    i = torch.arange(blocks, dtype=torch.int64, device=device)
    c0, c1 = i & low, i >> 32
    c2, c3 = (rng[1] & low).expand(blocks), torch.full_like(i, SITE)
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # (64 bits that wrap)
        c0, c1, c2, c3 = (((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1,
                          a & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([c0, c1, c2, c3], dim=1)


def _rstd(v):
    return torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)


def _run_plain(c, st):
    op = c["op"]
    if op.startswith("drop"):
        rows, d = c["rows"], c["d"]
        bits = _philox(st["rng"], (rows * d + 3) // 4, st["x"].device)
        keep = bits.reshape(-1)[:rows * d].reshape(rows, d) >= round(c["p"] * 2 ** 32)
        y = torch.where(keep, st["x"].to(F32) * (1.0 / (1.0 - c["p"])), 0.0)
        if st["residual"] is not None:
            y = y + st["residual"].to(F32)
        return y.to(DTYPES[c["y"]])
    if op == "norms_fwd":
        x = st["x"].to(F32)
        a = x * _rstd(x) * st["post"]
        if st["gate"] is not None:
            a = a * st["gate"]
        s = (c["alpha"] * st["residual"].to(F32) + a).to(DTYPES[c["s"]])
        v = s.to(F32)  # the norm of the stream as it is stored
        return [s, (v * _rstd(v) * st["pre"]).to(BF16)]
    if op == "norms_bwd":
        v, dy, x = st["s"].to(F32), st["dy"].to(F32), st["x"].to(F32)
        rstd = _rstd(v)
        n = v * rstd
        g = dy * st["pre"]
        ds = rstd * (g - n * (g * n).mean(dim=1, keepdim=True))
        if st["ds"] is not None:
            ds = ds + st["ds"].to(F32)
        dpre = (dy * n).sum(dim=0)
        rstd = _rstd(x)
        n = x * rstd
        da = ds if st["gate"] is None else ds * st["gate"]
        q = da * st["post"]
        dx = rstd * (q - n * (q * n).mean(dim=1, keepdim=True))
        out = [dx.to(DTYPES[c["x"]]), (c["alpha"] * ds).to(DTYPES[c["s"]]), (da * n).sum(dim=0),
               dpre]
        if st["gate"] is not None:
            out.append((ds * n * st["post"]).sum(dim=0) if c["gate"] == "channel" else
                       (ds * n * st["post"]).sum(dim=1, keepdim=True))
        return out
    x, w, off = st["x"], st["w"], st["bounds"]
    groups = [(e, off[e], off[e + 1]) for e in range(c["E"])]
    if op == "grouped_fwd":
        y = torch.empty(c["rows"], c["N"], dtype=DTYPES[c["out"]], device=x.device)
        for e, a, b in groups:
            if b > a:
                y[a:b] = x[a:b].to(F32) @ w[e].to(F32).t()
        return y
    dx = torch.empty(c["rows"], c["K"], dtype=DTYPES[c["out"]], device=x.device)
    dw = torch.zeros(c["E"], c["N"], c["K"], dtype=F32, device=x.device)
    for e, a, b in groups:
        if b > a:
            dy = st["dy"][a:b].to(F32)
            dx[a:b] = dy @ w[e].to(F32)
            dw[e] = dy.t() @ x[a:b].to(F32)
    return [dx, dw]


# ------------------------------------------------------------------- work --

def _size(kind):
    return 4 if kind == "f32" else 2


def work(case):
    c = case
    op = c["op"]
    if op.startswith("drop"):
        n = c["rows"] * c["d"]
        return {"bytes": n * (_size(c["x"]) + _size(c["y"]) * (2 if c["residual"] else 1)),
                "flops": 2 * n}
    if op.startswith("norms"):
        n, d = c["rows"] * c["d"], c["d"]
        gate = {"none": 0, "channel": 4 * d, "token": 4 * c["rows"]}[c["gate"]]
        if op == "norms_fwd":
            # the branch and the stream in, the stream and its norm out
            return {"bytes": n * (_size(c["x"]) + 2 * _size(c["s"]) + 2) + 8 * d + gate,
                    "flops": 12 * n}
        # dy, the branch and the stream in (and its gradient), both gradients out
        b = n * (_size(c["dy"]) + 2 * _size(c["x"]) + _size(c["s"]) * (3 if c["skip"] else 2))
        return {"bytes": b + 16 * d + 2 * gate, "flops": 28 * n}
    rows, N, K = c["rows"], c["N"], c["K"]
    if c["split"] == "one":
        used = rows
    else:  # experts with rows, on average
        used = sum(1.0 - (1.0 - p) ** rows for p in _shares(c))
    weights = int(used * N * K)
    if op == "grouped_fwd":
        return {"bytes": 2 * weights + rows * (2 * K + _size(c["out"]) * N),
                "flops": 2 * rows * N * K}
    return {"bytes": 2 * weights + 4 * c["E"] * N * K
            + rows * (2 * N + 2 * K + _size(c["out"]) * K), "flops": 4 * rows * N * K}


# ------------------------------------------------------------------ exact --

def _words(rng, count, device):
    """The generator's first `count` words, by 16-bit limbs (no product passes 48 bits)."""
    seed, step = (int(v) for v in rng.tolist())
    mask = (1 << 32) - 1

    def product(v, m):  # (high, low) words of v m
        lo = (v & 0xFFFF) * m
        hi = (v >> 16) * m + (lo >> 16)
        return hi >> 16, ((hi & 0xFFFF) << 16) | (lo & 0xFFFF)

    block = torch.arange((count + 3) // 4, dtype=torch.int64, device=device)
    ctr = [block & mask, block >> 32, torch.full_like(block, step & mask),
           torch.full_like(block, SITE)]
    for r in range(10):
        key = [((seed & mask) + r * 0x9E3779B9) & mask,
               ((seed >> 32 & mask) + r * 0xBB67AE85) & mask]
        h0, l0 = product(ctr[0], 0xD2511F53)
        h1, l1 = product(ctr[2], 0xCD9E8D57)
        ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
    out = torch.empty(block.numel(), 4, dtype=torch.int64, device=device)
    for j in range(4):
        out[:, j] = ctr[j]
    return out.flatten()[:count]


def exact(case, seed):
    c, st = case, prepare(case, seed)
    op = c["op"]
    if op.startswith("drop"):
        x = st["x"].to(F64)
        u = _words(st["rng"], x.numel(), x.device).to(F64).view(c["rows"], c["d"])
        y = x / (1.0 - c["p"])
        y[u < float(round(c["p"] * 2 ** 32))] = 0.0
        return y if st["residual"] is None else y.add_(st["residual"].to(F64))
    if op.startswith("norms"):
        d, x, post, pre = c["d"], st["x"].to(F64), st["post"].to(F64), st["pre"].to(F64)
        gate = 1.0 if st["gate"] is None else st["gate"].to(F64)
        mx = (x.pow(2).sum(1, keepdim=True) / d + EPS).sqrt()
        if op == "norms_fwd":
            s = c["alpha"] * st["residual"].to(F64) + gate * post * x / mx
            v = s.to(DTYPES[c["s"]]).to(F64)  # the second norm is of the stream as it is stored
            ms = (v.pow(2).sum(1, keepdim=True) / d + EPS).sqrt()
            return [s, pre * v / ms]
        v, dy = st["s"].to(F64), st["dy"].to(F64)
        ms = (v.pow(2).sum(1, keepdim=True) / d + EPS).sqrt()
        ds = dy * pre / ms - v * (dy * pre * v).sum(1, keepdim=True) / (d * ms.pow(3))
        if st["ds"] is not None:
            ds += st["ds"].to(F64)
        q = ds * gate * post
        dx = q / mx - x * (q * x).sum(1, keepdim=True) / (d * mx.pow(3))
        out = [dx, c["alpha"] * ds, (ds * gate * x / mx).sum(0), (dy * v / ms).sum(0)]
        if c["gate"] == "channel":
            out.append(post * (ds * x / mx).sum(0))
        elif c["gate"] == "token":
            out.append((ds * post * x / mx).sum(1, keepdim=True))
        return out
    x, w, off = st["x"], st["w"], st["bounds"]
    parts, grads = [], torch.zeros(c["E"], c["N"], c["K"], dtype=F64, device=x.device) \
        if op == "grouped_bwd" else None
    for e in range(c["E"]):
        rows = slice(off[e], off[e + 1])
        if op == "grouped_fwd":
            parts.append(torch.einsum("rk,nk->rn", x[rows].to(F64), w[e].to(F64)))
        else:
            dy = st["dy"][rows].to(F64)
            parts.append(torch.einsum("rn,nk->rk", dy, w[e].to(F64)))
            grads[e] = torch.einsum("rn,rk->nk", dy, x[rows].to(F64))
    y = torch.cat(parts)
    return y if op == "grouped_fwd" else [y, grads]
