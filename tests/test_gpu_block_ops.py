"""The operators around the layer against plain references in 64 bits: the
residual addition with RMS norm, the router's auxiliary losses, the dense
product; each with its gradient, at the sizes, types, strides and masks where
it can go wrong.  Bounds are derived in _block_ref.py."""
import ctypes
import math

import pytest
import torch

import _block_ref as ref
from _block_ref import F64, U16, U32
from routing_dispatch_grouped_router_gb300 import _lib, api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def randn(seed, *shape, dtype=BF16, scale=1.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = (torch.randn(*shape[:-1], shape[-1] + pad, generator=g, device="cuda") * scale).to(dtype)
    return t[..., :shape[-1]] if pad else t


def close(got, want, bound):
    """|got - want| <= bound everywhere, and equal where either is not finite."""
    got = got.to(F64)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine)
    d = (got - want).abs()[fine]
    b = (bound.expand_as(want) if torch.is_tensor(bound) else torch.full_like(want, bound))[fine]
    worst = (d - b).max().item() if d.numel() else 0.0
    assert worst <= 0, (worst, d.max().item())


# ------------------------------------------------------------- add_rmsnorm --

NORM_SHAPES = [(1, 1), (1, 7168), (3, 31), (5, 32), (2, 257), (7, 1000), (4, 1024), (9, 2880),
               (700, 160), (1300, 2048), (3, 8200), (2, 16384), (1, 16383)]


@pytest.mark.parametrize("rows,d", NORM_SHAPES)
@pytest.mark.parametrize("xt,st,wt,pad", [(BF16, BF16, F32, 0), (F32, BF16, BF16, 8),
                                          (BF16, F32, F32, 3), (F32, F32, BF16, 0)])
def test_add_rmsnorm(rows, d, xt, st, wt, pad):
    x = randn(1, rows, d, dtype=xt, pad=pad)
    r = randn(2, rows, d, dtype=st, scale=3.0, pad=pad)
    w = randn(3, d, dtype=wt)
    s, y = api.add_rmsnorm(x, w, r, eps=1e-5)
    s0, y0 = ref.add_rmsnorm(x, w, r, 1e-5)
    assert torch.equal(s, s0) and s.dtype == st
    # rstd: a sum of d squares (positive terms) and a reciprocal root of 2 ulp
    close(y, y0, y0.abs() * (1.01 * U16 + (2 * d + 16) * U32) + 1e-30)


@pytest.mark.parametrize("rows,d", [(1, 65), (40, 67), (9, 16376), (700, 2373), (3000, 130),
                                    (7, 16381), (1217, 4094), (8, 1001)])
@pytest.mark.parametrize("xt,st,wt", [(BF16, BF16, F32), (F32, BF16, BF16), (BF16, F32, F32),
                                      (F32, F32, BF16)])
@pytest.mark.parametrize("lds", [(0, 0, 0, 0), (8, 0, 16, 24), (4, 0, 0, 4), (1, 1, 1, 1),
                                 (0, 3, 0, 0)])
def test_add_rmsnorm_strided_rows(rows, d, xt, st, wt, lds):
    """Strides of their own: NaN between the rows of the inputs, and nothing written
    between those of s and y."""
    def strided(seed, pad, dtype):
        t = torch.full((rows, d + pad), math.nan, dtype=dtype, device="cuda")
        t[:, :d] = randn(seed, rows, d, dtype=dtype)
        return t[:, :d]
    x, r = strided(1, lds[0], xt), strided(2, lds[1], st)
    w = randn(3, d, dtype=wt)
    sb = torch.full((rows, d + lds[2]), 7.0, dtype=st, device="cuda")
    yb = torch.full((rows, d + lds[3]), 7.0, dtype=BF16, device="cuda")
    s, y = api.add_rmsnorm(x, w, r, eps=1e-5, s=sb[:, :d], y=yb[:, :d])
    assert (sb[:, d:] == 7).all() and (yb[:, d:] == 7).all()
    s0, y0 = ref.add_rmsnorm(x, w, r, 1e-5)
    assert torch.equal(s, s0)
    close(y, y0, y0.abs() * (1.01 * U16 + (2 * d + 16) * U32) + 1e-30)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rmsnorm_without_residual(dtype):
    x = randn(4, 37, 2048, dtype=dtype)
    w = randn(5, 2048, dtype=F32)
    s, y = api.add_rmsnorm(x, w)
    assert s is x
    _, y0 = ref.add_rmsnorm(x, w, None, 1e-6)
    close(y, y0, y0.abs() * (1.01 * U16 + 5000 * U32))


def test_add_rmsnorm_in_place():
    """The stream's new value may go over the residual or over x."""
    for over in ("residual", "x"):
        x, r, w = randn(6, 33, 7168), randn(7, 33, 7168), randn(8, 7168, dtype=F32)
        s0, y0 = api.add_rmsnorm(x, w, r)
        s, y = api.add_rmsnorm(x, w, r, s=r if over == "residual" else x)
        assert torch.equal(s, s0) and torch.equal(y, y0)


def test_add_rmsnorm_zero_and_non_finite_rows():
    x = randn(9, 6, 1000)
    x[1] = 0
    x[2, 5] = math.inf
    x[3, 7] = math.nan
    w = torch.ones(1000, device="cuda")
    _, y = api.add_rmsnorm(x, w, torch.zeros_like(x), eps=0.5)
    assert (y[1] == 0).all()
    # an infinite element: rstd is 0, the other elements are 0, its own inf * 0
    assert torch.isnan(y[2, 5]) and (y[2, :5] == 0).all()
    assert torch.isnan(y[3]).all()
    assert torch.isfinite(y[[0, 4, 5]]).all()


@pytest.mark.parametrize("rows,d", [(1, 32), (3, 96), (5, 2880), (130, 4096), (2, 16384),
                                    (650, 224)])
@pytest.mark.parametrize("xt,st,pad", [(BF16, BF16, 0), (F32, BF16, 3), (F32, F32, 0)])
def test_add_rmsnorm_mx(rows, d, xt, st, pad):
    x = randn(11, rows, d, dtype=xt, pad=pad)
    r = randn(12, rows, d, dtype=st, scale=3.0)
    r[0, :32] = 0
    x[0, :32] = 0  # a block of zeros
    w = randn(13, d, dtype=F32)
    values = torch.empty(rows, d, dtype=BF16, device="cuda")
    y = torch.empty(rows, d, dtype=BF16, device="cuda")
    s, codes, scales = api.add_rmsnorm_mx(x, w, r, values=values, y=y)
    s0, y0 = ref.add_rmsnorm(x, w, r, 1e-6)
    assert torch.equal(s, s0)
    assert torch.equal(y, api.add_rmsnorm(x, w, r)[1])
    # the values are exactly what codes and scales stand for
    assert torch.equal(values.to(F64), ref.decode(codes, scales))
    v0, sc0 = ref.mx_values(y0)
    assert scales[0, 0] == 0 and (values[0, :32] == 0).all()
    # an fp32 norm beside a rounding boundary may fall on its other side: one
    # E4M3 step there (2^-3 of the value or 2^-9 of the scale), equal elsewhere
    small = ref.pow2(sc0.to(torch.int32).unsqueeze(2) - 127 - 8)
    step = v0.abs() / 4 + small.expand(-1, -1, 32).reshape(rows, d)
    assert ((values.to(F64) - v0).abs() <= step).all()
    off = (values.to(F64) != v0).double().mean().item()
    assert off <= 64 * (2 * d + 16) * U32, off  # 16 steps per octave, 2 sides, margin 2
    assert (scales != sc0).double().mean().item() <= 64 * (2 * d + 16) * U32 + 1e-12


def test_mx_form_is_the_quantiser_s():
    """Codes of a norm that bf16 holds exactly are mok_mx_quantize's of it."""
    x = torch.ones(64, 256, device="cuda", dtype=BF16)
    w = ref.pow2(torch.randint(-9, 9, (256,), device="cuda")).float()
    y = torch.empty_like(x)
    _, codes, scales = api.add_rmsnorm_mx(x, w, eps=0.0, y=y)
    c2 = torch.empty_like(codes)
    s2 = torch.empty_like(scales)
    api.mx_quantize(y, False, codes=c2, scales=s2)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)


@pytest.mark.parametrize("rows,d", NORM_SHAPES + [(1217, 96)])
@pytest.mark.parametrize("yt,st,wt,skip,pad", [(BF16, BF16, F32, True, 0),
                                               (F32, BF16, BF16, True, 8),
                                               (BF16, F32, F32, False, 5),
                                               (F32, F32, F32, True, 0)])
def test_add_rmsnorm_backward(rows, d, yt, st, wt, skip, pad):
    dy = randn(21, rows, d, dtype=yt, pad=pad)
    s = randn(22, rows, d, dtype=st, scale=3.0, pad=pad)
    ds = randn(23, rows, d, dtype=st) if skip else None
    w = randn(24, d, dtype=wt)
    dx, dw = api.add_rmsnorm_backward(dy, s, w, ds, eps=1e-5)
    dx0, dw0 = ref.add_rmsnorm_backward(dy, s, w, ds, 1e-5)
    v = s.to(F64)
    rstd = (v.pow(2).mean(1, keepdim=True) + 1e-5).rsqrt()
    gw = (dy.to(F64) * w.to(F64)).abs()
    mag = rstd * (gw + (v * rstd).abs() * (gw * (v * rstd).abs()).mean(1, keepdim=True))
    if ds is not None:
        mag = mag + ds.to(F64).abs()
    close(dx, dx0, dx0.abs() * 1.01 * ref.rounding(st) + mag * (4 * d + 32) * U32)
    magw = (dy.to(F64) * v * rstd).abs().sum(0)
    close(dw, dw0, magw * (2 * rows + 2 * d + 32) * U32)


@pytest.mark.parametrize("rows,d", [(1, 513), (40, 515), (9, 16376), (1300, 2373), (2600, 1001),
                                    (3000, 644), (7, 16381), (1217, 4094)])
@pytest.mark.parametrize("yt,st,skip", [(BF16, BF16, True), (F32, BF16, False), (BF16, F32, True),
                                        (F32, F32, True)])
@pytest.mark.parametrize("lds", [(0, 0, 0, 0), (8, 0, 16, 24), (4, 0, 0, 4), (1, 1, 1, 1),
                                 (0, 3, 0, 0)])
def test_add_rmsnorm_backward_rows_at_a_shift(rows, d, yt, st, skip, lds):
    """Rows whose beginnings are alike in every tensor, or not; NaN between the rows
    of the inputs and nothing written between those of dx."""
    def strided(seed, pad, dtype, scale=1.0):
        t = torch.full((rows, d + pad), math.nan, dtype=dtype, device="cuda")
        t[:, :d] = randn(seed, rows, d, dtype=dtype, scale=scale)
        return t[:, :d]
    dy, s = strided(21, lds[0], yt), strided(22, lds[1], st, 3.0)
    ds = strided(23, lds[2], st) if skip else None
    w = randn(24, d, dtype=F32)
    buf = torch.full((rows, d + lds[3]), 7.0, dtype=st, device="cuda")
    dx, dw = api.add_rmsnorm_backward(dy, s, w, ds, eps=1e-5, dx=buf[:, :d])
    assert (buf[:, d:] == 7).all()
    dx0, dw0 = ref.add_rmsnorm_backward(dy, s, w, ds, 1e-5)
    v = s.to(F64)
    rstd = (v.pow(2).mean(1, keepdim=True) + 1e-5).rsqrt()
    gw = (dy.to(F64) * w.to(F64)).abs()
    mag = rstd * (gw + (v * rstd).abs() * (gw * (v * rstd).abs()).mean(1, keepdim=True))
    if ds is not None:
        mag = mag + ds.to(F64).abs()
    close(dx, dx0, dx0.abs() * 1.01 * ref.rounding(st) + mag * (4 * d + 32) * U32)
    magw = (dy.to(F64) * v * rstd).abs().sum(0)
    close(dw, dw0, magw * (2 * rows + 2 * d + 32) * U32)
    assert torch.equal(dw, api.add_rmsnorm_backward(dy, s, w, ds, eps=1e-5, dx=buf[:, :d])[1])


def test_add_rmsnorm_backward_accumulates_and_repeats():
    dy, s, ds = randn(25, 1000, 2880), randn(26, 1000, 2880), randn(27, 1000, 2880)
    w = randn(28, 2880, dtype=F32)
    dx, dw = api.add_rmsnorm_backward(dy, s, w, ds)
    dx2, dw2 = api.add_rmsnorm_backward(dy, s, w, ds)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    api.add_rmsnorm_backward(dy, s, w, ds, dx=ds, dweight=dw2, accumulate=True)  # dx over ds
    assert torch.equal(ds, dx) and torch.equal(dw2, dw + dw)


def test_add_rmsnorm_gradient_against_differences():
    x, w, dy = randn(29, 3, 200, dtype=F32), randn(30, 200, dtype=F32), randn(31, 3, 200, dtype=F32)
    dx, dw = api.add_rmsnorm_backward(dy, x, w, eps=1e-5)
    h = 1e-6
    for arg, grad in (("x", dx), ("w", dw)):
        v = torch.randn_like(grad, dtype=F64)
        val = []
        for sign in (1, -1):
            xx = x.to(F64) + (sign * h * v if arg == "x" else 0)
            ww = w.to(F64) + (sign * h * v if arg == "w" else 0)
            y = xx * (xx.pow(2).mean(1, keepdim=True) + 1e-5).rsqrt() * ww
            val.append((y * dy.to(F64)).sum())
        want = ((val[0] - val[1]) / (2 * h)).item()
        got = (grad.to(F64) * v).sum().item()
        assert abs(got - want) <= 1e-5 * (grad.to(F64) * v).abs().sum().item()


def test_empty_rows():
    w = torch.ones(256, device="cuda")
    x = torch.empty(0, 256, device="cuda", dtype=BF16)
    s, y = api.add_rmsnorm(x, w, x.clone())
    assert s.shape == y.shape == (0, 256)
    dx, dw = api.add_rmsnorm_backward(x, x, w)
    assert dx.shape == (0, 256) and (dw == 0).all()
    dw.fill_(3.0)
    api.add_rmsnorm_backward(x, x, w, dweight=dw, accumulate=True)
    assert (dw == 3.0).all()


# ---------------------------------------------------------- router_balance --

def routing(seed, T, E, k, masked=0.0, pad=0):
    l = randn(seed, T, E, dtype=F32, pad=pad)
    l += randn(seed + 1, E, dtype=F32)
    idx = torch.topk(l, k, 1).indices.to(torch.int32)
    mask = None
    if masked:
        g = torch.Generator(device="cuda").manual_seed(seed + 2)
        mask = (torch.rand(T, generator=g, device="cuda") >= masked).to(torch.uint8)
    return l, idx, mask


def check_balance(l, idx, mask, a=1e-2, b=1e-3):
    loss, counts, prob, lse, n = api.router_balance(l, idx, mask, balance_coef=a, z_coef=b)
    loss0, counts0, prob0, lse0, n0, p, m, f, some = ref.router_balance(l, idx, mask, a, b)
    T, E = l.shape
    assert torch.equal(counts, counts0) and int(n) == n0
    # softmax: E positive terms, exponentials of arguments up to |l - max|
    top = torch.where(some[:, None] & (l.to(F64) > -math.inf) & (l.to(F64) < math.inf),
                      l.to(F64).abs(), torch.zeros_like(l, dtype=F64)).amax().item() if T else 0.0
    soft = (2 * E + 4 * top + 64) * U32
    close(prob, prob0, prob0 * (soft + 2 * T * U32) + 1e-30)
    close(lse, lse0, (2 * E + 64) * U32 + torch.where(some, lse0, torch.zeros_like(lse0)).abs()
          * 4 * U32 + 4 * top * U32)
    close(loss, loss0, loss0.abs() * (2 * soft + (4 * T + 2 * E + 64) * U32) + 1e-30)
    u = torch.tensor([1.25, -0.75], device="cuda")
    dl = api.router_balance_backward(u, l, lse, counts, n, idx.shape[1], mask, balance_coef=a,
                                     z_coef=b)
    dl0 = ref.router_balance_backward(u, l, idx, mask, a, b)
    nn = max(n0, 1)
    mag = p * (1.25 * a * E * (f + (p @ f)[:, None] + 1.0 / E) +
               0.75 * 2 * b * torch.where(some, lse0, torch.zeros_like(lse0)).abs()[:, None]) / nn
    close(dl, dl0, mag * (2 * soft + (4 * E + 64) * U32) + 1e-30)
    if mask is not None:
        assert (dl[mask == 0] == 0).all()
    return loss, counts, prob, lse, n, dl


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (256, 8, 2), (33, 3, 2), (1000, 16, 4),
                                   (77, 17, 8), (4096, 64, 8), (999, 100, 5), (5000, 128, 8),
                                   (300, 255, 8), (1234, 384, 8), (700, 509, 3), (640, 512, 8)])
@pytest.mark.parametrize("masked,pad", [(0.0, 0), (0.4, 4), (0.1, 1)])
def test_router_balance(T, E, k, masked, pad):
    l, idx, mask = routing(100 + T, T, E, k, masked, pad)
    check_balance(l, idx, mask)
    assert api.device_status(api.operator_status()) == 0


def test_router_balance_masks_everything():
    l, idx, _ = routing(7, 500, 64, 8)
    mask = torch.zeros(500, dtype=torch.bool, device="cuda")
    loss, counts, prob, _, n, dl = check_balance(l, idx, mask)
    assert (loss == 0).all() and (counts == 0).all() and (prob == 0).all() and int(n) == 0
    assert (dl == 0).all()


def test_router_balance_no_tokens():
    l = torch.empty(0, 16, device="cuda")
    loss, counts, prob, lse, n = api.router_balance(
        l, torch.empty(0, 2, dtype=torch.int32, device="cuda"), balance_coef=1.0, z_coef=1.0)
    assert (loss == 0).all() and (counts == 0).all() and (prob == 0).all() and int(n) == 0


def test_router_balance_infinities():
    """-inf logits (experts out of the routing), also in whole rows; garbage in
    masked rows leaves no trace."""
    l, idx, mask = routing(8, 300, 40, 4, 0.3)
    l[:, 37:] = -math.inf
    idx = torch.topk(l, 4, 1).indices.to(torch.int32)
    l[11] = -math.inf
    check_balance(l, idx, mask)
    # a row masked with the type's lowest value: uniform (its lse^2 is beyond
    # fp32, so without the z loss)
    low = l.clone()
    low[12] = torch.finfo(F32).min
    low[13, :36] = torch.finfo(F32).min
    loss = check_balance(low, idx, mask, b=0.0)[0]
    assert loss[1] == 0
    dead = torch.nonzero(mask == 0).flatten()[:3]
    l[dead[0]], l[dead[1]] = math.nan, math.inf
    idx[dead[2]] = -7
    check_balance(l, idx, mask)
    assert api.device_status(api.operator_status()) == 0


def test_router_balance_reports_bad_input():
    word = api.operator_status()
    try:
        for what in ("nan", "inf", "index"):
            word.zero_()
            l, idx, _ = routing(9, 300, 40, 4)
            if what == "index":
                idx[5, 1], idx[6, 0] = 40, -1
            else:
                l[17, 3] = math.nan if what == "nan" else math.inf
            check_balance(l, idx, None)
            assert api.device_status(word) == (17 if what == "index" else 16)
    finally:
        word.zero_()


def test_router_balance_repeats_bitwise():
    l, idx, mask = routing(10, 20000, 384, 8, 0.2)
    first = check_balance(l, idx, mask)
    for _ in range(5):
        again = api.router_balance(l, idx, mask, balance_coef=1e-2, z_coef=1e-3)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_router_balance_gradient_against_differences():
    """Against central differences of the losses with the counts held (their
    derivative is zero almost everywhere)."""
    l, idx, mask = routing(11, 50, 24, 3, 0.2)
    *_, dl = check_balance(l, idx, mask, a=0.5, b=0.25)
    v = torch.randn(50, 24, dtype=F64, device="cuda")
    h = 1e-6
    val = []
    for sign in (1, -1):
        loss = ref.router_balance(l.to(F64) + sign * h * v, idx, mask, 0.5, 0.25)[0]
        val.append(1.25 * loss[0] - 0.75 * loss[1])
    want = ((val[0] - val[1]) / (2 * h)).item()
    assert abs((dl.to(F64) * v).sum().item() - want) <= 1e-5 * (dl.to(F64) * v).abs().sum().item()


# ----------------------------------------------------------------- linear --

LINEAR_SHAPES = [(1, 1, 8), (1, 2048, 7168), (2, 130, 72), (16, 128, 512), (17, 60, 136),
                 (64, 1000, 2048), (65, 384, 64), (128, 257, 1024), (129, 264, 200),
                 (200, 8, 4096), (255, 1024, 2880), (257, 33, 1000), (300, 2880, 96),
                 (1000, 4096, 256), (2049, 520, 1032)]


def check_linear(M, N, K, act, bias, residual, out, keep_z, pad=0, seed=50):
    x = randn(seed, M, K, pad=pad)
    w = randn(seed + 1, N, K, scale=1 / math.sqrt(K))
    b = randn(seed + 2, N, dtype=F32) if bias else None
    r = randn(seed + 3, M, N, dtype=out) if residual else None
    got = api.linear(x, w, b, act=act, residual=r, out_dtype=out, keep_z=keep_z)
    y0, z0, mag = ref.linear(x, w, b, act, r)
    y = got[0] if keep_z else got
    assert y.dtype == out
    dz = mag * (2 * K + 8) * U32
    # slopes of the activations stay below 1.13; the exponential's argument is
    # within |a| 2^-23, a up to 2|z| + z^3/7 but at most 100 where the result matters
    act_err = 0.0 if act in ("none", "relu") else act_bound(z0)
    close(y, y0, y0.abs() * 1.01 * ref.rounding(out) + 1.13 * dz + act_err
          + (r.to(F64).abs() * 2 * U32 if residual else 0.0) + 1e-30)
    if keep_z:
        close(got[1], z0, z0.abs() * 1.01 * ref.rounding(out) + dz + 1e-30)
    return x, w, b, r, y


def act_bound(z):
    a = (2 * z.abs() + z.abs() ** 3 / 7).clamp(max=100)
    return z.abs() * (8 + 4 * a) * U32


@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES)
@pytest.mark.parametrize("act,bias,residual,out,keep_z,pad",
                         [("none", False, False, BF16, False, 0), ("silu", True, True, BF16, True, 8),
                          ("gelu", True, True, F32, True, 0), ("relu", False, True, F32, False, 16)])
def test_linear(M, N, K, act, bias, residual, out, keep_z, pad):
    check_linear(M, N, K, act, bias, residual, out, keep_z, pad)
    assert api.device_status(api.operator_status()) == 0


@pytest.mark.parametrize("M", [1, 40, 300])
def test_linear_repeats_bitwise_and_in_place(M):
    x, w, b, r, y = check_linear(M, 2048, 1024, "silu", True, True, BF16, False)
    for _ in range(5):
        assert torch.equal(api.linear(x, w, b, act="silu", residual=r), y)
    api.linear(x, w, b, act="silu", residual=r, y=r)  # y over the residual
    assert torch.equal(r, y)


@pytest.mark.parametrize("M", [3, 200])
def test_linear_takes_any_alignment_of_its_epilogue(M):
    """bias, residual, y and z at odd element offsets give the aligned call's bits
    or bounds (another path may sum in another order)."""
    N, K = 264, 520
    x, w = randn(60, M, K), randn(61, N, K, scale=1 / math.sqrt(K))
    flat = lambda seed, n, dtype: randn(seed, n + 1, dtype=dtype)[1:]  # noqa: E731
    b = flat(62, N, F32)
    r = flat(63, M * N, BF16).view(M, N)
    y = torch.empty(M * N + 1, dtype=BF16, device="cuda")[1:].view(M, N)
    api.linear(x, w, b, act="gelu", residual=r, y=y)
    y0, z0, mag = ref.linear(x, w, b, "gelu", r)
    close(y, y0, y0.abs() * 1.01 * U16 + 1.13 * mag * (2 * K + 8) * U32 + act_bound(z0)
          + r.to(F64).abs() * 2 * U32)


@pytest.mark.parametrize("M,N", [(130, 1), (200, 5), (257, 13), (131, 39), (300, 129), (192, 270),
                                 (400, 301)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_linear_rows_of_any_alignment(M, N, out):
    """y, z and the residual at element offsets of their own in rows of odd
    lengths: values, and nothing written around them."""
    K = 200
    for oy, oz, orr in ((0, 0, 0), (1, 1, 1), (3, 5, 2), (7, 0, 4)):
        x, w, b = randn(54, M, K), randn(55, N, K, scale=1 / math.sqrt(K)), randn(56, N, dtype=F32)
        bufs = [torch.full((M * N + 32,), 7.0, dtype=out, device="cuda") for _ in range(2)]
        y, z = (t[8 + o:8 + o + M * N].view(M, N) for t, o in zip(bufs, (oy, oz)))
        r = randn(57, M * N + 8, dtype=out)[orr:orr + M * N].view(M, N)
        api.linear(x, w, b, act="silu", residual=r, y=y, z=z)
        y0, z0, mag = ref.linear(x, w, b, "silu", r)
        dz = mag * (2 * K + 8) * U32
        close(z, z0, z0.abs() * 1.01 * ref.rounding(out) + dz + 1e-30)
        close(y, y0, y0.abs() * 1.01 * ref.rounding(out) + 1.13 * dz + act_bound(z0)
              + r.to(F64).abs() * 2 * U32 + 1e-30)
        for t, o in zip(bufs, (oy, oz)):
            assert (t[:8 + o] == 7).all() and (t[8 + o + M * N:] == 7).all()


def test_linear_writes_its_own_elements_only():
    """Nothing before or behind y and z, at sizes that end inside a tile."""
    for M, N in ((1, 130), (70, 61), (130, 136), (300, 264)):
        x, w = randn(64, M, 200), randn(65, N, 200)
        buf = torch.full((2, M * N + 512), 7.0, dtype=BF16, device="cuda")
        y, z = (buf[i, 256:256 + M * N].view(M, N) for i in range(2))
        api.linear(x, w, act="silu", y=y, z=z)
        assert (buf[:, :256] == 7).all() and (buf[:, 256 + M * N:] == 7).all()
        assert not (y == 7).all(1).any()


def test_linear_non_finite():
    """A NaN or infinity reaches its own row (x) or column (w) only."""
    for M in (5, 300):
        x, w = randn(66, M, 256), randn(67, 136, 256)
        x[2, 3], x[4, 200] = math.nan, math.inf
        y = api.linear(x, w, act="silu")
        bad = ~torch.isfinite(y).all(1)
        assert bad[2] and bad[4] and bad.sum() == 2


def test_activation_limits():
    """Far tails: no NaN from inf * 0 where the limit is finite."""
    z = torch.tensor([-3e38, -1e20, -200.0, -30.0, 0.0, 30.0, 200.0, 1e20, 3e38], device="cuda")
    x = torch.zeros(1, 8, dtype=BF16, device="cuda")
    w = torch.zeros(9, 8, dtype=BF16, device="cuda")
    for act in ("relu", "silu", "gelu"):
        y = api.linear(x, w, z, act=act, out_dtype=F32)[0]
        want = ref.act(z.to(F64).clamp(-1e15, 1e15), act)[0]
        assert torch.isfinite(y).all()
        neg = z <= 0
        assert (y[neg].to(F64) - want[neg]).abs().max() <= 1e-10
        assert torch.allclose(y[~neg], z[~neg], rtol=1e-6)
        dz = api.linear_backward(torch.ones(1, 9, device="cuda"), x, w, z.view(1, 9), act=act,
                                 bias=True)[2]
        slope = (z > 0).to(F32)
        if act != "relu":
            slope[4] = 0.5
        assert torch.allclose(dz, slope, atol=1e-6)


@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES)
@pytest.mark.parametrize("act,dyt,dxt,bias", [("none", BF16, BF16, True), ("silu", BF16, BF16, False),
                                              ("gelu", F32, F32, True), ("relu", BF16, F32, True),
                                              ("none", F32, F32, False)])
def test_linear_backward(M, N, K, act, dyt, dxt, bias):
    x = randn(70, M, K, pad=8 if M % 2 else 0)
    w = randn(71, N, K, scale=1 / math.sqrt(K))
    dy, z = randn(72, M, N, dtype=dyt), randn(73, M, N, dtype=dyt)
    dx, dw, db = api.linear_backward(dy, x, w, z if act != "none" else None, act=act, bias=bias,
                                     dx_dtype=dxt)
    (dx0, dw0, db0), (mx, mw, mb) = ref.linear_backward(dy, x, w, z, act)
    # dz: the activation's slope (exponential as in the forward; slopes near
    # zero are differences, so the bound is absolute: u32 per unit of |dy|)
    slope = 0.0 if act in ("none", "relu") else 64 * U32
    dza = dy.to(F64).abs() * slope
    # two bf16 parts leave u16 of u16 of dz
    parts = U16 * U16 if dxt == BF16 else U32
    close(dx, dx0, dx0.abs() * 1.01 * ref.rounding(dxt) + mx * (2 * 3 * N * U32 + parts)
          + dza @ w.to(F64).abs() + 1e-30)
    close(dw, dw0, mw * (2 * 3 * M + 16) * U32 + dza.T @ x.to(F64).abs() + 1e-30)
    if bias:
        close(db, db0, mb * (2 * M + 16) * U32 + dza.sum(0) + 1e-30)
    else:
        assert db is None
    assert api.device_status(api.operator_status()) == 0


@pytest.mark.parametrize("M", [1, 2, 3, 4, 7, 8, 9])
@pytest.mark.parametrize("N,K", [(1, 8), (40, 136), (513, 264), (1300, 1032), (2050, 40008)])
def test_linear_backward_of_few_tokens(M, N, K):
    """Slices of N and their sum, accumulation, and each gradient without the others."""
    x, w = randn(90, M, K, pad=8), randn(91, N, K, scale=1 / math.sqrt(K))
    dy, z = randn(92, M, N, dtype=F32), randn(93, M, N, dtype=F32)
    dx, dw, db = api.linear_backward(dy, x, w, z, act="silu", bias=True, dx_dtype=F32)
    (dx0, dw0, db0), (mx, mw, mb) = ref.linear_backward(dy, x, w, z, "silu")
    dza = dy.to(F64).abs() * 64 * U32
    close(dx, dx0, mx * (2 * 3 * N * U32 + U32) + dza @ w.to(F64).abs() + 1e-30)
    close(dw, dw0, mw * (2 * 3 * M + 16) * U32 + dza.T @ x.to(F64).abs() + 1e-30)
    close(db, db0, mb * (2 * M + 16) * U32 + dza.sum(0) + 1e-30)
    again = [t.clone() for t in (dx, dw, db)]
    api.linear_backward(dy, x, w, z, act="silu", dx=again[0], dw=again[1], dbias=again[2],
                        accumulate=True)
    assert all(torch.equal(a + a, b) for a, b in zip((dx, dw, db), again))


@pytest.mark.parametrize("M,K", [(5, 136), (5, 40008), (40, 520)])
def test_linear_gradients_alone(M, K):
    """Through the C entry: any of dx, dw and dbias may be NULL."""
    N = 1300
    x, w = randn(94, M, K), randn(95, N, K)
    dy = randn(96, M, N)
    want = api.linear_backward(dy, x, w, bias=True)
    d = _lib.LinearDesc(M=M, N=N, K=K)
    n = ctypes.c_size_t()
    f = _lib.load()
    assert f.mok_linear_workspace_size(d, 1, n) == 0
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    for i in range(3):
        got = torch.zeros_like(want[i])
        out = [got.data_ptr() if i == j else None for j in range(3)]
        stream = torch.cuda.current_stream().cuda_stream
        assert f.mok_linear_backward(d, dy.data_ptr(), x.data_ptr(), w.data_ptr(), None, *out,
                                     ws.data_ptr() if n.value else None, n.value, None,
                                     stream) == 0
        assert torch.equal(got, want[i])


def test_linear_backward_accumulates_and_repeats():
    for M, N, K in ((40, 60, 136), (3000, 264, 512), (9000, 64, 256)):
        x, w, dy = randn(80, M, K), randn(81, N, K), randn(82, M, N, dtype=F32)
        one = api.linear_backward(dy, x, w, bias=True, dx_dtype=F32)
        two = api.linear_backward(dy, x, w, bias=True, dx_dtype=F32)
        assert all(torch.equal(a, b) for a, b in zip(one, two))
        api.linear_backward(dy, x, w, dx=two[0], dw=two[1], dbias=two[2], accumulate=True)
        assert all(torch.equal(b, a + a) for a, b in zip(one, two))


def test_linear_backward_no_tokens():
    x = torch.empty(0, 64, device="cuda", dtype=BF16)
    w = randn(83, 40, 64)
    assert api.linear(x, w).shape == (0, 40)
    dx, dw, db = api.linear_backward(torch.empty(0, 40, device="cuda", dtype=BF16), x, w, bias=True)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    dw += 2
    api.linear_backward(torch.empty(0, 40, device="cuda", dtype=BF16), x, w, dw=dw,
                        dx=torch.empty(0, 64, device="cuda"), accumulate=True)
    assert (dw == 2).all()


def test_linear_gradient_against_differences():
    M, N, K = 20, 24, 40
    x, w = randn(84, M, K), randn(85, N, K, scale=0.2)
    b, dy = randn(86, N, dtype=F32), randn(87, M, N, dtype=F32)
    y, z = api.linear(x, w, b, act="gelu", out_dtype=F32, keep_z=True)
    dx, dw, db = api.linear_backward(dy, x, w, z, act="gelu", bias=True, dx_dtype=F32)
    h = 1e-6
    for i, grad in enumerate((dx, dw, db)):
        v = torch.randn(grad.shape, dtype=F64, device="cuda")
        val = []
        for sign in (1, -1):
            args = [x.to(F64), w.to(F64), b.to(F64)]
            args[i] = args[i] + sign * h * v
            val.append((ref.act(args[0] @ args[1].T + args[2], "gelu")[0] * dy.to(F64)).sum())
        want = ((val[0] - val[1]) / (2 * h)).item()
        got = (grad.to(F64) * v).sum().item()
        assert abs(got - want) <= 1e-5 * (grad.to(F64) * v).abs().sum().item()


# --------------------------------------------------- streams, graphs, misuse --

def test_on_another_stream():
    """Calls on a stream of their own, behind slow work there, while the default
    stream is idle: every tensor a call makes belongs to that stream."""
    st = torch.cuda.Stream()
    x, r, w = randn(90, 512, 1024), randn(91, 512, 1024), randn(92, 1024, dtype=F32)
    wl = randn(93, 256, 1024)
    s0, y0 = api.add_rmsnorm(x, w, r)
    l0 = api.linear(y0, wl, out_dtype=F32)
    idx = torch.topk(l0, 4, 1).indices.to(torch.int32)
    b0 = api.router_balance(l0, idx, balance_coef=1.0, z_coef=1.0)
    g0 = api.linear_backward(l0, y0, wl, bias=True)
    n0 = api.add_rmsnorm_backward(g0[0], s0, w)
    torch.cuda.synchronize()
    xs, rs = torch.zeros_like(x), torch.zeros_like(r)
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        xs.copy_(x)
        rs.copy_(r)
    s, y = api.add_rmsnorm(xs, w, rs, stream=st)
    l = api.linear(y, wl, out_dtype=F32, stream=st)
    b = api.router_balance(l, idx, balance_coef=1.0, z_coef=1.0, stream=st)
    g = api.linear_backward(l, y, wl, bias=True, stream=st)
    n = api.add_rmsnorm_backward(g[0], s, w, stream=st)
    # memory handed out on the default stream meanwhile must not be theirs
    trash = [torch.full((1 << 18,), 3e38, device="cuda") for _ in range(16)]
    st.synchronize()
    del trash
    for got, want in zip((s, y, l, *b, *g, *n), (s0, y0, l0, *b0, *g0, *n0)):
        assert torch.equal(got, want)


def test_in_a_cuda_graph():
    x, r, w = randn(94, 300, 512), randn(95, 300, 512), randn(96, 512, dtype=F32)
    wl = randn(97, 64, 512)

    def step():
        s, y = api.add_rmsnorm(x, w, r)
        l = api.linear(y, wl, out_dtype=F32)
        b = api.router_balance(l, idx, balance_coef=1.0, z_coef=1.0)
        g = api.linear_backward(l, y, wl, bias=True)
        return (s, y, l, *b, *g, *api.add_rmsnorm_backward(g[0], s, w))

    idx = torch.randint(0, 64, (300, 4), dtype=torch.int32, device="cuda")
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    x, w = randn(98, 4, 64), torch.ones(64, device="cuda")
    bad = [
        lambda: api.add_rmsnorm(x, w[:32]),
        lambda: api.add_rmsnorm(x.half(), w),
        lambda: api.add_rmsnorm(x, w, x[:2]),
        lambda: api.add_rmsnorm(x.t(), w[:4]),
        lambda: api.add_rmsnorm(x.cpu(), w),
        lambda: api.add_rmsnorm(x, w.cpu()),
        lambda: api.add_rmsnorm(x, w, x, s=x.float()),
        lambda: api.add_rmsnorm(x[:1].expand(4, 64), w),
        lambda: api.add_rmsnorm_mx(x[:, :40], w[:40]),
        lambda: api.add_rmsnorm_backward(x, x, w, x.float()),
        lambda: api.add_rmsnorm_backward(x, x, w, accumulate=True),
        lambda: api.router_balance(x, torch.zeros(4, 2, dtype=torch.int32, device="cuda"),
                                   balance_coef=1.0),
        lambda: api.router_balance(x.float(), torch.zeros(4, 2, dtype=torch.int64, device="cuda"),
                                   balance_coef=1.0),
        lambda: api.linear(x, randn(99, 8, 32)),
        lambda: api.linear(x, randn(99, 8, 64), act="tanh"),
        lambda: api.linear(x, randn(99, 8, 64), residual=x),
        lambda: api.linear(x, randn(99, 8, 64), w),
        lambda: api.linear_backward(randn(99, 4, 8), x, randn(99, 8, 64), act="silu"),
        lambda: api.linear_backward(randn(99, 4, 8), x, randn(99, 8, 64), accumulate=True),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    refused = [
        (2, lambda: api.add_rmsnorm(torch.zeros(1, 16385, device="cuda"),
                                    torch.zeros(16385, device="cuda"))),
        (1, lambda: api.add_rmsnorm(x, w, eps=-1.0)),
        (1, lambda: api.add_rmsnorm(x, w, eps=math.nan)),
        (2, lambda: api.router_balance(torch.zeros(2, 513, device="cuda"),
                                       torch.zeros(2, 2, dtype=torch.int32, device="cuda"),
                                       balance_coef=1.0)),
        (2, lambda: api.router_balance(torch.zeros(2, 16, device="cuda"),
                                       torch.zeros(2, 9, dtype=torch.int32, device="cuda"),
                                       balance_coef=1.0)),
        (2, lambda: api.linear(x[:, :12].contiguous(), randn(99, 8, 12))),
        (1, lambda: api.linear(x[:, 1:57], randn(99, 8, 56))),
        (2, lambda: api.linear_backward(randn(99, 4, 8), x, randn(99, 8, 64), accumulate=True,
                                        dx=torch.zeros_like(x), dw=torch.zeros(8, 64, device="cuda"))),
        (3, lambda: api.linear_backward(randn(99, 40, 8), randn(99, 40, 64), randn(99, 8, 64),
                                        workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
    ]
    for code, call in refused:
        with pytest.raises(_lib.MokError) as e:
            call()
        assert e.value.code == code
