"""The branch operators on more than 2^32 elements and at the largest row counts:
offsets that pass 32 bits, checked where they do (the last rows, the last experts)."""
import pytest
import torch

import _branch_ref as ref
from _block_ref import F64, U16, U32
from routing_dispatch_grouped_router_gb300 import api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def randn(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    return t.normal_(std=scale, generator=g)


def close(got, want, bound):
    d = (got.to(F64) - want).abs()
    assert bool((d <= bound).all()), (d - bound).max().item()


@pytest.mark.parametrize("d", [8192, 8183, 16384])
def test_post_pre_past_32_bits(d):
    rows = (1 << 32) // d + 5
    x, r = randn(1, rows, d), randn(2, rows, d, scale=3.0)
    w1, w2 = randn(3, d, dtype=F32), randn(4, d, dtype=F32)
    gate = randn(5, rows, 1, dtype=F32)
    s, y = api.post_pre_rmsnorm(x, r, w1, w2, gate, s=r)  # in the residual's place
    tail = slice(rows - 3, rows)
    r0 = randn(2, rows, d, scale=3.0)[tail].clone()
    s0, bound, norm = ref.post_pre(x[tail], r0, w1, w2, gate[tail], 1.0, 1e-6, BF16)
    close(s[tail], s0, bound)
    close(y[tail], *norm(s[tail]))
    dx, dr, dw1, dw2, dg = api.post_pre_rmsnorm_backward(y, x, s, w1, w2, gate)
    want, bounds = ref.post_pre_backward(y[tail], x[tail], s[tail], w1, w2, gate[tail], None, 1.0,
                                         1e-6)
    for o, i in ((dx[tail], 0), (dr[tail], 1)):
        close(o, want[i], bounds[i] + want[i].abs() * 1.01 * U16 + 1e-30)
    close(dg[tail], want[4], bounds[4] + want[4].abs() * 1.01 * U32 + 1e-30)
    assert bool(torch.isfinite(dw1).all()) and bool(torch.isfinite(dw2).all())


def test_grouped_outputs_past_32_bits():
    """y and dx of more than 2^32 elements, the last groups at their ends."""
    R, N, K = (1 << 20) + 77, 4104, 64
    off = torch.tensor([0, 1 << 19, R - 130, R - 1, R], dtype=torch.int32, device="cuda")
    x, w = randn(1, R, K), randn(2, 4, N, K, scale=0.125)
    y = api.grouped_linear(x, w, off)
    for a, b, e in ((R - 130, R - 1, 2), (R - 1, R, 3), ((1 << 19) - 3, 1 << 19, 0)):
        want = x[a:b].to(F64) @ w[e].to(F64).T
        mag = x[a:b].to(F64).abs() @ w[e].to(F64).abs().T
        close(y[a:b], want, mag * 2 * K * U32 + want.abs() * 1.01 * U16 + 1e-30)
    dx, dw = api.grouped_linear_backward(y, x, w, off)
    a = R - 130
    want = y[a:R - 1].to(F64) @ w[2].to(F64)
    mag = y[a:R - 1].to(F64).abs() @ w[2].to(F64).abs()
    close(dx[a:R - 1], want, mag * 2 * N * U32 + want.abs() * 1.01 * U16 + 1e-30)
    want = y[a:R - 1].to(F64).T @ x[a:R - 1].to(F64)
    close(dw[2], want, (y[a:R - 1].to(F64).abs().T @ x[a:R - 1].to(F64).abs()) * 2 * 129 * U32 + 1e-30)
    assert api.device_status(api.operator_status()) == 0


def test_grouped_weights_past_32_bits():
    """Weights and their gradient of more than 2^32 elements, rows at the last expert."""
    E, N, K = 65, 8192, 8200
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = 3
    off[E] = 20
    w = randn(1, E, N, K, scale=K ** -0.5)
    x, dy = randn(2, 20, K), randn(3, 20, N)
    y = api.grouped_linear(x, w, off, out_dtype=F32)
    dx, dw = api.grouped_linear_backward(dy, x, w, off, dx_dtype=F32)
    for rows, e in ((slice(0, 3), 0), (slice(3, 20), E - 1)):
        a, g, we = x[rows].to(F64), dy[rows].to(F64), w[e].to(F64)
        close(y[rows], a @ we.T, (a.abs() @ we.abs().T) * 2 * K * U32)
        close(dx[rows], g @ we, (g.abs() @ we.abs()) * 2 * N * U32)
        close(dw[e], g.T @ a, (g.abs().T @ a.abs()) * 2 * 17 * U32 + 1e-30)
    assert not dw[E // 2].any()


@pytest.mark.parametrize("ends", [[1 << 24], [5, (1 << 24) - 9, 1 << 24]])
def test_grouped_of_the_most_rows(ends):
    R, N, K = 1 << 24, 16, 24
    off = torch.tensor([0] + ends, dtype=torch.int32, device="cuda")
    E = len(ends)
    x, dy, w = randn(1, R, K), randn(2, R, N), randn(3, E, N, K, scale=0.2)
    y = api.grouped_linear(x, w, off)
    dx, dw = api.grouped_linear_backward(dy, x, w, off)
    assert api.device_status(api.operator_status()) == 0
    o = off.tolist()
    for e in range(E):
        b = o[e + 1]
        a = max(o[e], b - 1000)
        want = x[a:b].to(F64) @ w[e].to(F64).T
        mag = x[a:b].to(F64).abs() @ w[e].to(F64).abs().T
        close(y[a:b], want, mag * 2 * K * U32 + want.abs() * 1.01 * U16 + 1e-30)
        want = dy[a:b].to(F64) @ w[e].to(F64)
        mag = dy[a:b].to(F64).abs() @ w[e].to(F64).abs()
        close(dx[a:b], want, mag * 2 * N * U32 + want.abs() * 1.01 * U16 + 1e-30)
        r = slice(o[e], b)
        want = dy[r].to(F64).T @ x[r].to(F64)
        assert ((dw[e].to(F64) - want).pow(2).mean() / want.pow(2).mean()).sqrt() < 2e-6


def test_dropout_rows_of_the_largest_sizes():
    """One long row, and rows of one element."""
    n = (1 << 31) - 1
    x = torch.ones(1, n, dtype=BF16, device="cuda")
    rng = torch.tensor([9, 1], device="cuda")
    y = api.dropout(x, 0.5, rng, 2)
    first = n // 4 * 4 - 4096
    keep = ref.dropout_words(9, 1, 2, first, n - first, "cuda") >= 1 << 31
    assert torch.equal(y[0, first:] != 0, keep)
    y2 = api.dropout(x.view(n, 1), 0.5, rng, 2, y=y.view(n, 1))
    assert torch.equal(y2[first:, 0] != 0, keep)


def test_dropout_of_rows_of_one_element():
    """2^31 - 1 rows of one element at a stride of two: more than 2^31 groups, so that
    places are counted in 64 bits, and what lies between the rows stays."""
    n = (1 << 31) - 1
    x = torch.ones(n, 1, dtype=BF16, device="cuda")
    rng = torch.tensor([9, 1], device="cuda")
    out = torch.full((n, 2), 7.0, dtype=BF16, device="cuda")
    api.dropout(x, 0.5, rng, 2, y=out[:, :1])
    for first in (0, 1 << 30, n // 4 * 4 - 4096):
        count = min(4096, n - first)
        keep = ref.dropout_words(9, 1, 2, first, count, "cuda") >= 1 << 31
        assert torch.equal(out[first:first + count, 0],
                           torch.where(keep, 2.0, 0.0).to(BF16))
    for part in out[:, 1].split(1 << 28):
        assert bool((part == 7).all())


@pytest.mark.parametrize("rows,d,pad", [((1 << 21) + 1, 8200, 0), ((1 << 21) + 1, 8200, 8),
                                        ((1 << 21) + 1, 8201, 1)])
def test_dropout_past_2_to_the_34_elements(rows, d, pad):
    """More than 2^34 elements, where the counter's second word is not 0, in place:
    contiguous, in rows of whole words, in rows at an odd stride."""
    x = torch.ones(rows, d + pad, dtype=BF16, device="cuda")
    rng = torch.tensor([9, 1], device="cuda")
    v = x[:, :d]
    assert api.dropout(v, 0.25, rng, 2, y=v) is v
    for r0 in (0, rows // 2, rows - 4):
        a = r0 * d // 4 * 4
        w = ref.dropout_words(9, 1, 2, a, 4 * d + 8, "cuda")[r0 * d - a:][:4 * d].reshape(4, d)
        assert torch.equal(v[r0:r0 + 4] != 0, w >= 1 << 30)
    assert bool((x[::97, d:] == 1).all())
