"""The products grouped by expert against plain references in 64 bits: ragged and
empty groups, widths that no tile divides, strides, values that must not cross a
group's border.

Bounds: a sum of n products accumulated in fp32 is within 2 n u32 of the sum of
their magnitudes (twice n u32: the tensor cores truncate), and the output's
rounding."""
import ctypes
import math

import pytest
import torch

from _block_ref import F64, U32, rounding
from routing_dispatch_grouped_router_gb300 import _lib, api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def randn(seed, *shape, dtype=BF16, scale=1.0, pad=0):
    """Normal values; with `pad`, in rows with NaN behind them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)
    if not pad:
        return t
    b = torch.full((*shape[:-1], shape[-1] + pad), math.nan, dtype=dtype, device="cuda")
    b[..., :shape[-1]] = t
    return b[..., :shape[-1]]


def table(sizes, lead=0):
    """Offsets of groups of these sizes after `lead` rows."""
    o = [lead]
    for n in sizes:
        o.append(o[-1] + n)
    return o, torch.tensor(o, dtype=torch.int32, device="cuda")


def close(got, want, mag, n, dtype):
    bound = mag * 2 * n * U32 + want.abs() * 1.01 * rounding(dtype) + 1e-30
    d = (got.to(F64) - want).abs()
    assert bool((d <= bound).all()), (d - bound).max().item()


def check(sizes, N, K, dtype, lead=0, behind=0, pad=0, seed=1):
    o, off = table(sizes, lead)
    E, R = len(sizes), o[-1] + behind
    x = randn(seed, R, K, pad=pad)
    dy = randn(seed + 1, R, N, pad=pad)
    w = randn(seed + 2, E, N, K, scale=K ** -0.5)
    for t in (x, dy):  # rows of no group, and the weights of no rows, are not read
        t[:lead] = math.nan
        t[o[-1]:] = math.inf
    for e, n in enumerate(sizes):
        if n == 0:
            w[e] = math.nan
    yb = torch.full((R, N + pad), 7.0, dtype=dtype, device="cuda")
    xb = torch.full((R, K + pad), 7.0, dtype=dtype, device="cuda")
    y = api.grouped_linear(x, w, off, y=yb[:, :N])
    dx, dw = api.grouped_linear_backward(dy, x, w, off, dx=xb[:, :K])
    for b, cols in ((yb, N), (xb, K)):
        assert bool((b[:, cols:] == 7).all()) and bool((b[:lead] == 7).all())
        assert bool((b[o[-1]:] == 7).all())
    for e, n in enumerate(sizes):
        r = slice(o[e], o[e + 1])
        if n == 0:
            assert not dw[e].any()
            continue
        a, g, we = x[r].to(F64), dy[r].to(F64), w[e].to(F64)
        close(y[r], a @ we.T, a.abs() @ we.abs().T, K, dtype)
        close(dx[r], g @ we, g.abs() @ we.abs(), N, dtype)
        close(dw[e], g.T @ a, g.abs().T @ a.abs(), n, F32)
    assert api.device_status(api.operator_status()) == 0
    return x, dy, w, off, y, dx, dw


SIZES = [[1], [5], [128], [130, 0, 1], [0, 0, 300, 64], [16, 17, 15, 1, 31, 32, 33, 63, 64, 65],
         [127, 129, 256, 255, 257, 2], [700, 3, 0, 90], [1] * 40, [0] * 9 + [8] + [0] * 30,
         [577, 1153]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("N,K", [(8, 8), (64, 72), (136, 200), (264, 520), (600, 1032)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_grouped(sizes, N, K, dtype):
    check(sizes, N, K, dtype)


@pytest.mark.parametrize("lead,behind,pad", [(3, 0, 0), (0, 5, 8), (130, 70, 24), (1, 200, 0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_grouped_rows_of_no_group_and_strides(lead, behind, pad, dtype):
    check([70, 0, 129, 30], 328, 264, dtype, lead, behind, pad)
    check([0, 0], 72, 64, dtype, lead, behind, pad)


def test_grouped_many_experts():
    g = torch.Generator().manual_seed(3)
    check(torch.randint(0, 9, (512,), generator=g).tolist(), 72, 136, F32)
    check([0] * 511 + [200], 72, 136, BF16)
    check([200] + [0] * 511, 72, 136, BF16)


@pytest.mark.parametrize("sizes,N,K", [([3000, 1, 0, 2047], 1400, 2888),
                                       ([512] * 24, 1024, 1536), ([9000, 40], 2048, 512)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_grouped_large(sizes, N, K, dtype):
    """Several tiles per CTA; fp32 results to 1e-6 rms, which one accumulation over
    1400 values or more (2e-6) does not meet."""
    x, dy, w, off, y, dx, dw = check(sizes, N, K, dtype)
    o = off.tolist()

    def rms(got, want):
        return ((got.to(F64) - want).pow(2).mean() / want.pow(2).mean()).sqrt().item()

    for e, n in enumerate(sizes):
        if n == 0:
            continue
        r = slice(o[e], o[e + 1])
        a, g, we = x[r].to(F64), dy[r].to(F64), w[e].to(F64)
        assert rms(dw[e], g.T @ a) < 1e-6
        if dtype == F32:
            assert rms(y[r], a @ we.T) < 1e-6 and rms(dx[r], g @ we) < 1e-6


@pytest.mark.parametrize("sizes,N,K", [([20000], 64, 72), ([9000, 0, 13], 136, 64),
                                       ([4097, 1, 2222], 8, 200), ([1030], 256, 128)])
def test_grouped_weight_gradient_in_parts(sizes, N, K):
    """Few tiles and many rows: dw summed in parts of the rows, to 1e-6 rms, added into
    dw after their sum; one group's values in no other's."""
    x, dy, w, off, y, dx, dw = check(sizes, N, K, BF16)
    o = off.tolist()
    for e, n in enumerate(sizes):
        if n:
            r = slice(o[e], o[e + 1])
            want = dy[r].to(F64).T @ x[r].to(F64)
            assert ((dw[e].to(F64) - want).pow(2).mean() / want.pow(2).mean()).sqrt() < 1e-6
    acc = dw.clone()
    api.grouped_linear_backward(dy, x, w, off, dw=acc, accumulate=True)
    assert torch.equal(acc, 2 * dw)
    if len(sizes) > 1:
        x2 = x.clone()
        x2[o[-2]:] = math.nan
        assert torch.equal(api.grouped_linear_backward(dy, x2, w, off)[1][:-1], dw[:-1])


def test_grouped_values_stay_in_their_group():
    """NaN and Inf in one group's rows or weights reach no other group's results."""
    sizes = [33, 7, 129, 64, 1, 250]
    x, dy, w, off, y, dx, dw = check(sizes, 136, 328, F32)
    o = off.tolist()
    for bad, value in ((1, math.nan), (2, math.inf), (4, math.nan)):
        x2, dy2, w2 = x.clone(), dy.clone(), w.clone()
        r = slice(o[bad], o[bad + 1])
        x2[r], dy2[r], w2[bad] = value, value, value
        y2 = api.grouped_linear(x2, w2, off, out_dtype=F32)
        dx2, dw2 = api.grouped_linear_backward(dy2, x2, w2, off, dx_dtype=F32)
        keep = torch.ones(o[-1], dtype=torch.bool, device="cuda")
        keep[r] = False
        assert torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])
        assert not torch.isfinite(y2[r]).any() and not torch.isfinite(dx2[r]).any()
        for e in range(len(sizes)):
            assert torch.equal(dw2[e], dw[e]) if e != bad else not torch.isfinite(dw2[e]).any()


def test_grouped_is_bitwise_repeatable_and_a_rows_result_its_own():
    """The same call gives the same bits, and a group's result does not depend on
    the groups beside it."""
    sizes = [300, 41, 129]
    x, dy, w, off, y, dx, dw = check(sizes, 264, 392, BF16)
    for _ in range(3):
        assert torch.equal(api.grouped_linear(x, w, off), y)
        a, b = api.grouped_linear_backward(dy, x, w, off)
        assert torch.equal(a, dx) and torch.equal(b, dw)
    o = off.tolist()
    off2 = torch.tensor([o[1], o[2]], dtype=torch.int32, device="cuda")
    y2 = api.grouped_linear(x, w[1:2].contiguous(), off2)
    assert torch.equal(y2[o[1]:o[2]], y[o[1]:o[2]])


def test_grouped_accumulates():
    sizes = [70, 0, 129, 30]
    x, dy, w, off, y, dx, dw = check(sizes, 136, 264, BF16)
    acc = dw.clone()
    acc[1] = 3.0
    api.grouped_linear_backward(dy, x, w, off, dw=acc, accumulate=True)
    assert torch.equal(acc[[0, 2, 3]], 2 * dw[[0, 2, 3]]) and bool((acc[1] == 3).all())


@pytest.mark.parametrize("raw,taken", [([0, 40, 20, 100], [0, 40, 40, 100]),
                                       ([-5, 10, 50, 1000], [0, 10, 50, 128]),
                                       ([200, 3, 4, 5], [128, 128, 128, 128])])
def test_grouped_offsets_out_of_order(raw, taken):
    """Taken as mok.h says, and reported; nothing outside of the rows is touched."""
    x, w = randn(1, 128, 72), randn(2, 3, 136, 72)
    word = api.operator_status()
    bad = torch.tensor(raw, dtype=torch.int32, device="cuda")
    good = torch.tensor(taken, dtype=torch.int32, device="cuda")
    outs = []
    for off in (good, bad):
        y = torch.full((128, 136), 7.0, dtype=BF16, device="cuda")
        dx = torch.full((128, 72), 7.0, dtype=BF16, device="cuda")
        api.grouped_linear(x, w, off, y=y)
        outs.append((y,) + api.grouped_linear_backward(y, x, w, off, dx=dx))
        code = api.device_status(word)
        word.zero_()
        torch.cuda.synchronize()
        assert code == (0 if off is good else 17)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_grouped_streams_and_graphs():
    """On another stream, and captured: replays read the offsets that memory holds."""
    x, dy, w = randn(1, 512, 264), randn(2, 512, 136), randn(3, 4, 136, 264)
    plans = [torch.tensor(o, dtype=torch.int32, device="cuda")
             for o in ([0, 100, 100, 300, 512], [0, 1, 510, 511, 512], [0, 0, 0, 0, 512])]
    want = [(api.grouped_linear(x, w, o),) + api.grouped_linear_backward(dy, x, w, o)
            for o in plans]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (api.grouped_linear(x, w, plans[0], stream=side),) + \
        api.grouped_linear_backward(dy, x, w, plans[0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want[0]):
        assert torch.equal(a, b)
    off = plans[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = api.grouped_linear(x, w, off)
        dx, dw = api.grouped_linear_backward(dy, x, w, off)
    for o, t in zip(plans, want):
        off.copy_(o)
        graph.replay()
        for a, b in zip((y, dx, dw), t):
            assert torch.equal(a, b)


def test_grouped_empty_and_refused():
    w, off = randn(1, 3, 64, 72), torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = randn(2, 0, 72), randn(2, 0, 64)
    assert api.grouped_linear(x, w, off).shape == (0, 64)
    dx, dw = api.grouped_linear_backward(dy, x, w, off)
    assert dx.shape == (0, 72) and not dw.any()
    x, dy = randn(2, 10, 72), randn(2, 10, 64)
    odd = torch.empty(10 * 72 + 8, dtype=BF16, device="cuda")[1:721].view(10, 72)
    with pytest.raises(_lib.MokError):
        api.grouped_linear(odd, w, off)  # not 16-byte aligned
    many = torch.zeros(514, dtype=torch.int32, device="cuda")
    with pytest.raises(_lib.MokError):
        api.grouped_linear(x, randn(1, 513, 64, 72), many)
    for call in (lambda: api.grouped_linear(x, w[:, :, :64], off),
                 lambda: api.grouped_linear(x[:, :64], w, off),
                 lambda: api.grouped_linear(x, w[0], off),
                 lambda: api.grouped_linear(x, w, off[:3]),
                 lambda: api.grouped_linear(x, w, off.long()),
                 lambda: api.grouped_linear(x, w, off.cpu()),
                 lambda: api.grouped_linear(x.float(), w, off),
                 lambda: api.grouped_linear(x, w.float(), off),
                 lambda: api.grouped_linear(x, w, off, out_dtype=torch.float16),
                 lambda: api.grouped_linear(x, w, off, y=randn(1, 9, 64)),
                 lambda: api.grouped_linear(randn(1, 10, 70), randn(1, 3, 64, 70), off),
                 lambda: api.grouped_linear(randn(1, 10, 75)[:, :72], w, off),
                 lambda: api.grouped_linear_backward(dy.float(), x, w, off),
                 lambda: api.grouped_linear_backward(dy[:9], x, w, off),
                 lambda: api.grouped_linear_backward(dy, x, w, off, accumulate=True),
                 lambda: api.grouped_linear_backward(dy, x, w, off, dw=w)):
        with pytest.raises(ValueError):
            call()


def test_grouped_on_a_dispatch_plan():
    """The offsets that the layer's dispatch plan writes."""
    T, d, E, I, k = 300, 128, 16, 128, 4
    desc = api.make_desc(T, d, E, I, k)
    g = torch.Generator(device="cuda").manual_seed(5)
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    pos = torch.empty(T, k, dtype=torch.int32, device="cuda")
    rows = torch.empty(T * k, dtype=torch.int32, device="cuda")
    ws = torch.empty(api.stage_workspace_size(desc), dtype=torch.uint8, device="cuda")
    api.dispatch_plan(desc, idx.contiguous(), counts, off, pos, rows, ws)
    x, w = randn(6, T, d), randn(7, E, 264, d)
    y = api.grouped_linear(x[rows.long()], w, off, out_dtype=F32)
    got = y[pos.long()]  # [T, k, N]
    want = torch.einsum("td,tknd->tkn", x.to(F64), w.to(F64)[idx.long()])
    mag = torch.einsum("td,tknd->tkn", x.to(F64).abs(), w.to(F64).abs()[idx.long()])
    assert bool(((got.to(F64) - want).abs() <= mag * 2 * d * U32 + want.abs() * U32).all())


def test_grouped_long_sums():
    """2^20 values of one sign into bf16: half a step, and what sums of 4096 values on
    the tensor cores (truncated: twice u32 a value), added in fp32, may lose.  (One
    accumulation loses 6.7e-3 here, over two of the half steps.)"""
    R, n, m = 32, 1 << 20, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.rand(R, n, generator=g, device="cuda").bfloat16()
    b = (torch.rand(1, m, n, generator=g, device="cuda") * n ** -0.5).bfloat16()
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    want = a.to(F64) @ b[0].to(F64).T  # (every term is positive: its own magnitude)
    bound = want * (1.01 * rounding(BF16) + (2 * 4096 + n / 4096) * U32)
    y = api.grouped_linear(a, b, off)
    dx, _ = api.grouped_linear_backward(a, a[:, :m].contiguous(), b.transpose(1, 2).contiguous(),
                                        off)
    for got in (y, dx):
        d = (got.to(F64) - want).abs()
        assert bool((d <= bound).all()), (d / want).max().item()


@pytest.mark.parametrize("sizes,cols", [([20, 0, 13], 264), ([100] * 160, 256),
                                        ([5000, 130], 264)])
def test_grouped_long_sums_of_every_tile(sizes, cols):
    """Just past 2^14 values, by narrow tiles, wide ones and pairs: rows of bf16 and fp32
    results in 64 bits, bf16 ones within half a step and the loss of 4096 values in one
    accumulation."""
    n = 16456
    _, off = table(sizes)
    R, E = sum(sizes), len(sizes)
    a, b = randn(1, R, n), randn(2, E, cols, n, scale=n ** -0.5)
    out = torch.full((R, cols + 8), 7.0, dtype=BF16, device="cuda")
    y = api.grouped_linear(a, b, off, y=out[:, :cols])
    y32 = api.grouped_linear(a, b, off, out_dtype=F32)
    x, w = torch.zeros(R, cols, dtype=BF16, device="cuda"), b.transpose(1, 2).contiguous()
    dx, _ = api.grouped_linear_backward(a, x, w, off)
    dx32, _ = api.grouped_linear_backward(a, x, w, off, dx_dtype=F32)
    assert bool((out[:, cols:] == 7).all())
    for r in (0, R // 2, R - 1):
        e = (off[1:] <= r).sum().item()
        want = b[e].to(F64) @ a[r].to(F64)
        mag = b[e].to(F64).abs() @ a[r].to(F64).abs()
        for got, m in ((y, 4096), (y32, 576), (dx, 4096), (dx32, 576)):
            close(got[r], want, mag, m + n / m, got.dtype)


RAGGED = [517, 1, 0, 700, 63, 480, 530, 16, 1033, 500, 0, 799, 401, 512, 31, 900, 640, 333, 777, 2,
          15, 1200, 600, 257]


@pytest.mark.parametrize("sizes", [RAGGED, [n // 2 + 3 for n in RAGGED]])
@pytest.mark.parametrize("N,K", [(1024, 1536), (1088, 1600), (1096, 1600), (1088, 1608)])
def test_grouped_ragged_at_training_sizes(sizes, N, K):
    """Pairs of CTAs and wide single ones with groups' last rows below sixteen, widths
    of whole 64-column blocks (an odd number of them: the last box passes the map's end)
    and others."""
    check(sizes, N, K, BF16)


def test_grouped_lengths_of_every_remainder():
    """Every number of last rows, between neighbours of NaN, by pairs (fp32 dx too)."""
    check([400 + i for i in range(16)] + [800 + 3 * i for i in range(16)], 512, 256, F32)
