"""Plain references in 64 bits of dropout, the norms after and before a block and
the products grouped by expert, and the error bounds their tests use.

Bounds: as _block_ref.py's.  u32 = 2^-24 and u16 = 2^-8 are half a step of fp32 and
bf16 at 1.  A sum of n fp32 products in any order is within 2 n u32 of the sum of
their magnitudes, and what is computed from it inherits that with its own few
roundings (16 u32 hold the reciprocal root's 2 and every product's).
"""
import torch

from _block_ref import F64, U32, rounding

MASK = 0xFFFFFFFF


def philox4x32_10(ctr, key):
    """Philox4x32-10 of one counter (four words) and key (two), in Python integers."""
    c, k = list(ctr), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & MASK, (a >> 32) ^ c[3] ^ k[1], a & MASK]
        k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
    return c


def dropout_words(seed, step, site, first, count, device="cpu"):
    """Words of elements first .. first + count - 1 (first a multiple of 4), int64."""
    block = first // 4 + torch.arange((count + 3) // 4, dtype=torch.int64, device=device)
    c = [block & MASK, block >> 32, torch.full_like(block, step & MASK),
         torch.full_like(block, site)]
    k0, k1 = seed & MASK, (seed >> 32) & MASK

    def mul(v, m):  # 16-bit limbs: nothing passes 2^49
        lo = (v & 0xFFFF) * m
        hi = (v >> 16) * m + (lo >> 16)
        return hi >> 16, ((hi & 0xFFFF) << 16) | (lo & 0xFFFF)

    for _ in range(10):
        ah, al = mul(c[0], 0xD2511F53)
        bh, bl = mul(c[2], 0xCD9E8D57)
        c = [bh ^ c[1] ^ k0, bl, ah ^ c[3] ^ k1, al]
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    return torch.stack(c, 1).reshape(-1)[:count]


def dropout(x, p, seed, step, site, residual, dtype):
    """(y, bound, kept)."""
    rows, d = x.shape
    keep = dropout_words(seed, step, site, 0, rows * d, x.device).reshape(rows, d) \
        >= round(p * 2 ** 32)
    v = torch.where(keep, x.to(F64) / (1 - p) if p < 1 else 0.0, 0.0)
    y = v if residual is None else v + residual.to(F64)
    # the scale's rounding, the fused product's, and the output's
    return y, v.abs() * 2 * U32 + y.abs() * (rounding(dtype) + 2 * U32) + 1e-38, keep


def _rstd(v, eps):
    return (v.pow(2).mean(1, keepdim=True) + eps).rsqrt()


def post_pre(x, r, w1, w2, gate, alpha, eps, dtype):
    """(s, its bound, a map from the stored s to (y, its bound))."""
    d = x.shape[1]
    x, r, w1, w2 = x.to(F64), r.to(F64), w1.to(F64), w2.to(F64)
    a = x * _rstd(x, eps) * w1
    if gate is not None:
        a = a * gate.to(F64)
    s = alpha * r + a
    bound = a.abs() * (2 * d + 16) * U32 + s.abs() * (1.01 * rounding(dtype) + 2 * U32) \
        + (alpha * r).abs() * 2 * U32 + 1e-30

    def norm(stored):
        v = stored.to(F64)
        y = v * _rstd(v, eps) * w2
        return y, y.abs() * (1.01 * rounding(torch.bfloat16) + (2 * d + 16) * U32) + 1e-30
    return s, bound, norm


def post_pre_backward(dy, x, s, w1, w2, gate, ds, alpha, eps):
    """([dx, dresidual, dpost, dpre, dgate], their bounds without the outputs' rounding)."""
    rows, d = x.shape
    dy, x, s, w1, w2 = (t.to(F64) for t in (dy, x, s, w1, w2))
    z = torch.ones((), dtype=F64, device=x.device) if gate is None else gate.to(F64)
    r2, r1 = _rstd(s, eps), _rstd(x, eps)
    m, n, g = s * r2, x * r1, dy * w2
    t = r2 * (g - m * (g * m).mean(1, keepdim=True))
    u = (2 * d + 32) * U32
    bt = r2 * (g.abs() + m.abs() * (g * m).abs().mean(1, keepdim=True)) * u
    if ds is not None:
        t = t + ds.to(F64)
        bt = bt + ds.to(F64).abs() * 2 * U32
    q = t * z * w1
    bq = (bt + t.abs() * 4 * U32) * (z * w1).abs()
    dx = r1 * (q - n * (q * n).mean(1, keepdim=True))
    bx = r1 * (bq + n.abs() * (bq * n.abs()).mean(1, keepdim=True)
               + u * (q.abs() + n.abs() * (q * n).abs().mean(1, keepdim=True)))
    rest = u + 2 * rows * U32  # of a column sum: n's and the sum's own errors
    out = [dx, alpha * t, (t * z * n).sum(0), (dy * m).sum(0)]
    bounds = [bx, abs(alpha) * (bt + t.abs() * 2 * U32),
              ((bt * (z * n).abs()).sum(0) + rest * (t * z * n).abs().sum(0)),
              rest * (dy * m).abs().sum(0)]
    if gate is not None:
        dim = 0 if gate.dim() == 1 else 1
        e = t * w1 * n
        be = (bt * (w1 * n).abs() + e.abs() * (u + 2 * max(rows, d) * U32)).sum(dim)
        out.append(e.sum(dim).reshape(gate.shape))
        bounds.append(be.reshape(gate.shape))
    return out, bounds
