"""Plain references in 64 bits of the operators around the layer, and the error
bounds their tests use.

Bounds: u32 = 2^-24 is fp32's unit roundoff, u16 = 2^-8 bf16's (half a step of
2^-7 at 1: 8 significant bits, round to nearest).  A sum of n fp32 products is within 2 n u32 of the sum
of their magnitudes (twice n u32, for accumulators that truncate); the bounds
below add to that the final rounding and, where an exponential takes part, the
hardware exponential's 2 ulp and the rounding of its argument.
"""
import math

import torch

F64 = torch.float64
U32, U16 = 2.0 ** -24, 2.0 ** -8


def rounding(dtype):
    return U16 if dtype == torch.bfloat16 else U32


def add_rmsnorm(x, weight, residual, eps):
    """(s, y in 64 bits) with s rounded to the stream's type as stored."""
    if residual is None:
        s = x
    else:
        # an fp32 sum of two bf16 or fp32 values, then the stream's rounding
        s = (x.float() + residual.float()).to(residual.dtype)
    v = s.to(F64)
    rstd = (v.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    return s, v * rstd * weight.to(F64)


def add_rmsnorm_backward(dy, s, weight, ds, eps):
    v, w, g = s.to(F64), weight.to(F64), dy.to(F64)
    rstd = (v.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    n = v * rstd
    gw = g * w
    dx = rstd * (gw - n * (gw * n).mean(1, keepdim=True))
    if ds is not None:
        dx = dx + ds.to(F64)
    return dx, (g * n).sum(0)


def router_balance(logits, idx, mask, balance_coef, z_coef):
    T, E = logits.shape
    l = logits.to(F64)
    l = torch.where(l < math.inf, l, torch.full_like(l, -math.inf))  # NaN and +inf
    some = (l > -math.inf).any(1)
    m = torch.ones(T, dtype=F64, device=l.device) if mask is None else (mask != 0).to(F64)
    p = torch.where(some[:, None], torch.softmax(torch.where(some[:, None], l, torch.zeros_like(l)),
                                                 1), torch.zeros_like(l))
    lse = torch.logsumexp(l, 1)
    n = int(m.sum())
    rows = idx[m > 0].reshape(-1).long()
    counts = torch.bincount(rows[(rows >= 0) & (rows < E)], minlength=E)
    nn = max(n, 1)
    prob = (m[:, None] * p).sum(0) / nn
    f = counts.to(F64) / (nn * idx.shape[1])
    loss = torch.stack([balance_coef * E * (f * prob).sum(),
                        z_coef * (m * torch.where(some, lse, torch.zeros_like(lse)) ** 2).sum() / nn])
    return loss, counts.to(torch.int32), prob, lse, n, p, m, f, some


def router_balance_backward(dloss, logits, idx, mask, balance_coef, z_coef):
    _, _, _, lse, n, p, m, f, some = router_balance(logits, idx, mask, balance_coef, z_coef)
    E = logits.shape[1]
    nn = max(n, 1)
    lse = torch.where(some, lse, torch.zeros_like(lse))
    u = dloss.to(F64)
    d = p * (u[0] * balance_coef * E * (f - (p @ f)[:, None]) + u[1] * 2 * z_coef * lse[:, None])
    return d / nn * m[:, None]


def act(z, name):
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if name == "silu":
        a, da = z, torch.ones_like(z)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        a, da = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z ** 2)
    s = torch.sigmoid(a)
    return z * s, s + z * s * (1 - s) * da


def linear(x, w, bias, name, residual):
    """(y, z, bound of |z| errors): the sum of magnitudes a sum's error scales with."""
    z = x.to(F64) @ w.to(F64).T
    mag = x.to(F64).abs() @ w.to(F64).abs().T
    if bias is not None:
        z = z + bias.to(F64)
        mag = mag + bias.to(F64).abs()
    y = act(z, name)[0]
    if residual is not None:
        y = y + residual.to(F64)
    return y, z, mag


def linear_backward(dy, x, w, z, name):
    """(dx, dw, db) and the magnitudes of their sums."""
    dz = dy.to(F64)
    if name != "none":
        dz = dz * act(z.to(F64), name)[1]
    x, w = x.to(F64), w.to(F64)
    return (dz @ w, dz.T @ x, dz.sum(0)), (dz.abs() @ w.abs(), dz.abs().T @ x.abs(),
                                           dz.abs().sum(0))


def pow2(e):
    """2^e in 64 bits, exactly (a library power may be an ulp off), for integers e."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def mx_values(v):
    """MXFP8 values of 64-bit rows in blocks of 32 columns, with codes' scale bytes."""
    b = v.reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(2, keepdim=True)
    _, e = torch.frexp(amax)
    shared = (e - 9).clamp(-127, 127)
    shared = torch.where(amax > 0, shared, torch.full_like(shared, -127))
    t = b * pow2(-shared)
    _, q = torch.frexp(t)
    step = pow2((q - 1).clamp(min=-6) - 3)
    t = (torch.round(t / step) * step).clamp(-448, 448)
    return (t * pow2(shared)).reshape(v.shape), (shared + 127).squeeze(2).to(torch.uint8)


def decode(codes, scales):
    """The bf16 values of E4M3 codes [rows, d] and E8M0 bytes [rows, d/32]."""
    q = codes.view(torch.float8_e4m3fn).to(F64).reshape(codes.shape[0], -1, 32)
    return (q * pow2(scales.to(torch.int32).unsqueeze(2) - 127)).reshape(codes.shape)
