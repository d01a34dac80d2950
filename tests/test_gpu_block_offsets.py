"""The operators around the layer on tensors of more than 2^32 bytes or 2^31
elements, and at the sizes that mok.h states as the largest: rows at both ends
and about the boundary against 64-bit references, sums over all rows against the
sums of two halves.  Bounds as in _block_ref.py."""
import math

import pytest
import torch

import _block_ref as ref
from _block_ref import F64, U16, U32
from routing_dispatch_grouped_router_gb300 import api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def randn(seed, *shape, dtype=BF16, scale=1.0):
    """Normal values, made without an fp32 copy of all of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, scale, generator=g)


def within(got, want, bound):
    d = (got.to(F64) - want).abs() - bound
    assert torch.isfinite(got).all()
    assert d.max().item() <= 0, (d.max().item(), (got.to(F64) - want).abs().max().item())


def ends(rows, cols):
    """Row ranges at both ends and about element 2^31 and 2^32."""
    at = [0, rows - 3] + [min(max(e // cols - 1, 0), rows - 3) for e in (1 << 31, 1 << 32)]
    return [slice(a, a + 3) for a in sorted(set(at))]


@pytest.mark.parametrize("d", [8192, 8191])
def test_norm_of_more_than_two_to_the_31_elements(d):
    rows = (1 << 32) // 8192 + 700
    x, r = randn(1, rows, d), randn(2, rows, d, scale=3.0)
    w = 1 + randn(3, d, dtype=F32, scale=0.1)
    s, y = api.add_rmsnorm(x, w, r)
    if d % 32 == 0:
        values = torch.empty(rows, d, dtype=BF16, device="cuda")
        _, codes, scales = api.add_rmsnorm_mx(x, w, r, values=values)
    dx, dw = api.add_rmsnorm_backward(x, s, w, r)
    for q in ends(rows, d):
        s0, y0 = ref.add_rmsnorm(x[q], w, r[q], 1e-6)
        assert torch.equal(s[q], s0)
        within(y[q], y0, y0.abs() * (1.01 * U16 + (2 * d + 16) * U32) + 1e-30)
        if d % 32 == 0:
            assert torch.equal(values[q].to(F64), ref.decode(codes[q], scales[q]))
            # the exact norm's codes, but where it lies within 2^-42 of a boundary
            lo, hi = (ref.mx_values(y0 * (1 + e))[0] for e in (-2.0 ** -42, 2.0 ** -42))
            assert torch.equal(values[q].to(F64)[lo == hi], lo[lo == hi])
        dx0, _ = ref.add_rmsnorm_backward(x[q], s[q], w, r[q], 1e-6)
        v = s[q].to(F64)
        n = v * (v.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt()
        rstd = (v.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt()
        g = (x[q].to(F64) * w.to(F64)).abs()
        mag = rstd * (g + n.abs() * (g * n.abs()).mean(1, keepdim=True)) + r[q].to(F64).abs()
        within(dx[q], dx0, dx0.abs() * 1.01 * U16 + mag * (4 * d + 32) * U32)
    h = rows // 2
    _, a = api.add_rmsnorm_backward(x[:h], s[:h], w, r[:h])
    _, b = api.add_rmsnorm_backward(x[h:], s[h:], w, r[h:])
    # sums of half a million terms that do not line up, in blocks: 1e-4 of their size
    rms = lambda t: t.pow(2).mean().sqrt().item()  # noqa: E731
    assert rms(dw - (a + b)) <= 1e-4 * rms(dw)


@pytest.mark.parametrize("N", [8192, 8190, 8191])
def test_linear_of_more_than_two_to_the_31_outputs(N):
    M, K = (1 << 32) // 8192 + 300, 64
    x, w = randn(11, M, K), randn(12, N, K, scale=1 / math.sqrt(K))
    b, r = randn(13, N, dtype=F32), randn(14, M, N)
    y, z = api.linear(x, w, b, act="relu", residual=r, keep_z=True)
    dx, dw, db = api.linear_backward(r, x, w, z, act="relu", bias=True)
    for q in ends(M, N):
        y0, z0, mag = ref.linear(x[q], w, b, "relu", r[q])
        dz = mag * (2 * K + 8) * U32
        within(z[q], z0, z0.abs() * 1.01 * U16 + dz + 1e-30)
        within(y[q], y0, y0.abs() * 1.01 * U16 + dz + r[q].to(F64).abs() * 2 * U32 + 1e-30)
        (dx0, _, _), (mx, _, _) = ref.linear_backward(r[q], x[q], w, z[q], "relu")
        within(dx[q], dx0, dx0.abs() * 1.01 * U16 + mx * (6 * N * U32 + U16 * U16) + 1e-30)
    h = M // 2
    half = [api.linear_backward(r[q], x[q], w, z[q], act="relu", bias=True)[1:]
            for q in (slice(0, h), slice(h, M))]
    rms = lambda t: t.pow(2).mean().sqrt().item()  # noqa: E731
    for got, p, q in zip((dw, db), *half):
        assert rms(got - (p + q)) <= 1e-4 * rms(got)


def test_balance_of_many_tokens():
    T, E, k = (1 << 27) // 8 * 3, 96, 8  # 4.8e9 logits
    l = randn(21, T, E, dtype=F32)
    idx = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(22))
    loss, counts, prob, lse, n = api.router_balance(l, idx, balance_coef=1.0, z_coef=1.0)
    assert int(n) == T
    assert torch.equal(counts.long(), torch.bincount(idx.view(-1), minlength=E))
    u = torch.ones(2, device="cuda")
    dl = api.router_balance_backward(u, l, lse, counts, n, k, balance_coef=1.0, z_coef=1.0)
    f = counts.to(F64) / (T * k)
    for q in ends(T, E):
        p = torch.softmax(l[q].to(F64), 1)
        lse0 = torch.logsumexp(l[q].to(F64), 1)
        within(lse[q], lse0, (2 * E + 64) * U32 + lse0.abs() * 4 * U32 + 64 * U32)
        want = p * (E * (f - (p @ f)[:, None]) + 2 * lse0[:, None]) / T
        mag = p * (E * (f + (p @ f)[:, None] + 1 / E) + 2 * lse0.abs()[:, None]) / T
        within(dl[q], want, mag * (2 * (2 * E + 128) + 4 * E + 64) * U32 + 1e-30)
    # means over fifty million tokens, added by 152 blocks' threads one after the
    # other (some 10^4 terms each): 1e-4
    want = torch.zeros(E, dtype=F64, device="cuda")
    z = 0.0
    for c in l.split(1 << 22):
        p = torch.softmax(c, 1)
        want += p.sum(0, dtype=F64)
        z += torch.logsumexp(c, 1).to(F64).pow(2).sum()
    assert ((prob.to(F64) - want / T).abs() <= 1e-4 / E).all()
    assert abs(loss[1].item() - z.item() / T) <= 1e-4 * z.item() / T


@pytest.mark.parametrize("M,N", [(1 << 24, 8), (16, 1 << 24), (3, 1 << 24), (300, 1 << 24)])
def test_linear_at_its_largest_sizes(M, N):
    """As many tokens or features as mok.h takes."""
    K = 8
    x, w = randn(31, M, K), randn(32, N, K)
    y = api.linear(x, w)
    dx, dw, db = api.linear_backward(y, x, w, bias=True, dx_dtype=F32)
    assert api.device_status(api.operator_status()) == 0
    if M > N:
        for q in ends(M, N):
            y0, _, mag = ref.linear(x[q], w, None, "none", None)
            within(y[q], y0, y0.abs() * 1.01 * U16 + mag * (2 * K + 8) * U32 + 1e-30)
            (dx0, _, _), (mx, _, _) = ref.linear_backward(y[q], x[q], w, None, "none")
            within(dx[q], dx0, mx * (2 * N + 2) * U32 + 1e-30)
    else:
        for n0 in (0, N // 2 - 100, N - 200):
            q = slice(n0, n0 + 200)
            y0, _, mag = ref.linear(x, w[q], None, "none", None)
            within(y[:, q], y0, y0.abs() * 1.01 * U16 + mag * (2 * K + 8) * U32 + 1e-30)
            (_, dw0, db0), (_, mw, mb) = ref.linear_backward(y[:, q], x, w[q], None, "none")
            within(dw[q], dw0, mw * (6 * M + 16) * U32 + 1e-30)
            within(db[q], db0, mb * (2 * M + 16) * U32 + 1e-30)
