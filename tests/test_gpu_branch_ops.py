"""Dropout and the norms after and before a block against plain references in 64
bits, at the sizes, types, strides and values where they can go wrong.  Bounds are
derived in _branch_ref.py."""
import math

import pytest
import torch

import _branch_ref as ref
from _block_ref import F64, U32, rounding
from routing_dispatch_grouped_router_gb300 import _lib, api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
SEED = 0x1234_5678_9ABC_DEF1


def randn(seed, *shape, dtype=BF16, scale=1.0, pad=0):
    """Normal values; with `pad`, in rows with NaN behind them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)
    if not pad:
        return t
    b = torch.full((*shape[:-1], shape[-1] + pad), math.nan, dtype=dtype, device="cuda")
    b[..., :shape[-1]] = t
    return b[..., :shape[-1]]


def rng(seed=SEED, step=3):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


def close(got, want, bound):
    """|got - want| <= bound everywhere, and alike where either is not finite."""
    got = got.to(F64)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine)
    d, b = (got - want).abs()[fine], bound.expand_as(want)[fine]
    assert d.numel() == 0 or bool((d <= b).all()), ((d - b).max().item(), d.max().item())


def rms(got, want):
    return ((got.to(F64) - want).pow(2).mean() / want.pow(2).mean().clamp(min=1e-300)).sqrt().item()


# ---------------------------------------------------------------- dropout --

@pytest.mark.parametrize("rows,d", [(1, 1), (1, 7), (3, 4), (5, 13), (1000, 1), (7, 4099),
                                    (64, 2048), (130, 72), (2, 16385)])
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("pad,res", [(0, False), (0, True), (8, True), (1, True), (4, False)])
def test_dropout(rows, d, xt, yt, pad, res):
    p = 0.3
    x = randn(1, rows, d, dtype=xt, pad=pad)
    r = randn(2, rows, d, dtype=yt, scale=3.0, pad=pad) if res else None
    y = api.dropout(x, p, rng(), 9, residual=r, out_dtype=yt)
    y0, bound, keep = ref.dropout(x, p, SEED, 3, 9, r, yt)
    assert y.dtype == yt and y.shape == x.shape
    close(y, y0, bound)
    if not res:
        assert not y[~keep].any()
        # its backward is the same map
        assert torch.equal(api.dropout_backward(x, p, rng(), 9, dx_dtype=yt), y)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -33, 2.0 ** -32, 0.5, 0.9, 1.0 - 2.0 ** -33, 1.0])
def test_dropout_probabilities(p):
    x = randn(1, 33, 515, dtype=F32)
    y = api.dropout(x, p, rng(), 0)
    y0, bound, keep = ref.dropout(x, p, SEED, 3, 0, None, F32)
    if round(p * 2 ** 32) == 2 ** 32:
        assert not y.any()
    else:
        close(y, y0, bound)
    if p in (0.0, 2.0 ** -33):
        assert bool(keep.all())


def test_dropout_rate_and_independence():
    """Kept shares within five standard deviations, also of pairs of masks."""
    n, p = 1 << 24, 0.2
    x = torch.ones(4096, 4096, device="cuda")
    base = api.dropout(x, p, rng(), 0) != 0
    others = [api.dropout(x, p, rng(step=4), 0) != 0, api.dropout(x, p, rng(), 1) != 0,
              api.dropout(x, p, rng(seed=SEED + 1), 0) != 0,
              api.dropout(x, p, rng(seed=SEED ^ (1 << 40)), 0) != 0]
    for m, q in [(base, 0.8)] + [(base & o, 0.64) for o in others] + \
            [(base[:, 1:] & base[:, :-1], 0.64), (base[1:] & base[:-1], 0.64)]:
        k = m.numel()
        assert abs(m.sum().item() - q * k) < 5 * math.sqrt(k * q * (1 - q)) * 1.5
    assert base.numel() == n


def test_dropout_of_a_place_is_the_same_for_any_stride_and_type():
    x = torch.ones(37, 51, device="cuda")
    m = api.dropout(x, 0.5, rng(), 2) != 0
    for xt in (BF16, F32):
        for pad in (0, 1, 5, 13):
            v = torch.ones(37, 51 + pad, device="cuda", dtype=xt)[:, :51]
            assert torch.equal(api.dropout(v, 0.5, rng(), 2, out_dtype=BF16) != 0, m)


def test_dropout_keeps_what_is_dropped_out_of_y():
    x = randn(1, 64, 256, dtype=F32)
    _, _, keep = ref.dropout(x, 0.4, SEED, 3, 1, None, F32)
    bad = x.clone()
    bad[~keep] = math.nan
    bad[::2][~keep[::2]] = math.inf
    assert torch.equal(api.dropout(bad, 0.4, rng(), 1), api.dropout(x, 0.4, rng(), 1))


def test_dropout_in_place_and_between_rows():
    for pad in (0, 3):
        x, r = randn(1, 40, 77, pad=pad), randn(2, 40, 77, pad=pad)
        want = api.dropout(x, 0.3, rng(), residual=r)
        for target in (x, r):
            x2 = torch.as_strided(x._base.clone() if pad else x.clone(), x.shape, x.stride())
            r2 = torch.as_strided(r._base.clone() if pad else r.clone(), r.shape, r.stride())
            y = x2 if target is x else r2
            assert api.dropout(x2, 0.3, rng(), residual=r2, y=y) is y
            assert torch.equal(y, want)
        out = torch.full((40, 80), 7.0, dtype=BF16, device="cuda")
        api.dropout(x, 0.3, rng(), residual=r, y=out[:, :77])
        assert torch.equal(out[:, :77], want) and bool((out[:, 77:] == 7).all())


def test_dropout_captured_draws_by_the_step_in_memory():
    x = randn(1, 128, 192)
    state = rng(step=0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        api.dropout(x, 0.5, state, 4)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = api.dropout(x, 0.5, state, 4)
        dx = api.dropout_backward(y, 0.5, state, 4)
        state[1] += 1
    seen = []
    for step in (0, 1, 2):
        graph.replay()
        assert torch.equal(y, api.dropout(x, 0.5, rng(step=step), 4))
        assert torch.equal(dx, api.dropout_backward(y, 0.5, rng(step=step), 4))
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_dropout_past_32_bits():
    """More than 2^32 elements, contiguous and strided: the last rows' places."""
    rows, d, p = (1 << 19) + 3, 8200, 0.25
    x = torch.ones(rows, d, dtype=BF16, device="cuda")
    y = api.dropout(x, p, rng(), 5)
    r0 = rows - 4
    first = r0 * d  # (a multiple of four)
    keep = ref.dropout_words(SEED, 3, 5, first, 4 * d, "cuda").reshape(4, d) >= round(p * 2 ** 32)
    assert torch.equal(y[r0:] != 0, keep)
    v = x[:, :8197]
    y2 = api.dropout(v, p, rng(), 5, y=y[:, :8197])
    first = r0 * 8197 // 4 * 4
    w = ref.dropout_words(SEED, 3, 5, first, 4 * 8197 + 4, "cuda")[r0 * 8197 - first:]
    assert torch.equal(y2[r0:] != 0, w[:4 * 8197].reshape(4, 8197) >= round(p * 2 ** 32))


def test_dropout_empty_and_refused():
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    assert api.dropout(x, 0.5, rng()).shape == (0, 64)
    x = randn(1, 4, 64)
    for call in (lambda: api.dropout(x, -0.1, rng()), lambda: api.dropout(x, 1.1, rng()),
                 lambda: api.dropout(x, math.nan, rng()), lambda: api.dropout(x[0], 0.1, rng()),
                 lambda: api.dropout(x, 0.1, rng().cpu()), lambda: api.dropout(x, 0.1, None),
                 lambda: api.dropout(x, 0.1, rng().int()), lambda: api.dropout(x, 0.1, rng(), -1),
                 lambda: api.dropout(x, 0.1, rng(), 1 << 32), lambda: api.dropout(x.half(), 0.1, rng()),
                 lambda: api.dropout(x.t(), 0.1, rng()),
                 lambda: api.dropout(x, 0.1, rng(), residual=x.float(), out_dtype=BF16),
                 lambda: api.dropout(x, 0.1, rng(), residual=x[:2]),
                 lambda: api.dropout(x, 0.1, rng(), y=x.float(), out_dtype=BF16),
                 lambda: api.dropout(x[:1].expand(4, 64), 0.1, rng()),
                 lambda: api.dropout_backward(x, 0.1, rng(), dx=x[:, :32])):
        with pytest.raises(ValueError):
            call()


# -------------------------------------------------------- post_pre_rmsnorm --

def gate_of(kind, rows, d, dtype):
    if kind == "none":
        return None
    shape = (d,) if kind == "channel" else (rows, 1)
    return randn(9, *shape, dtype=dtype)


SHAPES = [(1, 1), (1, 7168), (3, 31), (5, 32), (2, 257), (7, 1000), (4, 1024), (9, 2880),
          (700, 160), (1300, 2048), (3, 8200), (2, 16384), (1, 16383), (700, 2373), (9, 8192)]
TYPES = [(BF16, BF16, F32, F32), (F32, BF16, BF16, F32), (BF16, F32, F32, BF16),
         (F32, F32, BF16, BF16)]


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("xt,st,wt,gt", TYPES)
@pytest.mark.parametrize("kind,pad", [("none", 0), ("channel", 8), ("token", 3)])
def test_post_pre(rows, d, xt, st, wt, gt, kind, pad):
    x = randn(1, rows, d, dtype=xt, scale=0.5, pad=pad)
    r = randn(2, rows, d, dtype=st, scale=3.0, pad=pad)
    w1, w2, gate = randn(3, d, dtype=wt), randn(4, d, dtype=wt), gate_of(kind, rows, d, gt)
    sb = torch.full((rows, d + pad), 7.0, dtype=st, device="cuda")
    yb = torch.full((rows, d + pad), 7.0, dtype=BF16, device="cuda")
    s, y = api.post_pre_rmsnorm(x, r, w1, w2, gate, residual_scale=0.75, eps=1e-5, s=sb[:, :d],
                                y=yb[:, :d])
    assert bool((sb[:, d:] == 7).all()) and bool((yb[:, d:] == 7).all())
    s0, bound, norm = ref.post_pre(x, r, w1, w2, gate, 0.75, 1e-5, st)
    close(s, s0, bound)
    close(y, *norm(s))
    again = api.post_pre_rmsnorm(x, r, w1, w2, gate, residual_scale=0.75, eps=1e-5,
                                 s=torch.empty_like(sb)[:, :d], y=torch.empty_like(yb)[:, :d])
    assert torch.equal(again[0], s) and torch.equal(again[1], y)
    # contiguous outputs: rows that begin elsewhere may be summed in another order
    s2, y2 = api.post_pre_rmsnorm(x, r, w1, w2, gate, residual_scale=0.75, eps=1e-5)
    assert s2.dtype == st
    close(s2, s0, bound)
    close(y2, *norm(s2))


@pytest.mark.parametrize("rows,d", SHAPES + [(40, 67), (9, 16376), (3000, 130), (1217, 4094),
                                             (2500, 1032), (8, 1001), (1000, 4096)])
@pytest.mark.parametrize("yt,xt,st,wt,gt", [(BF16, BF16, BF16, F32, F32),
                                            (F32, BF16, F32, BF16, BF16),
                                            (BF16, F32, BF16, BF16, F32),
                                            (F32, F32, F32, F32, BF16),
                                            (BF16, F32, F32, F32, F32)])
@pytest.mark.parametrize("kind,pad,skip", [("none", 0, True), ("channel", 8, False),
                                           ("token", 3, True), ("channel", 0, True)])
def test_post_pre_backward(rows, d, yt, xt, st, wt, gt, kind, pad, skip):
    x = randn(1, rows, d, dtype=xt, scale=0.5, pad=pad)
    s = randn(2, rows, d, dtype=st, scale=3.0, pad=pad)
    dy = randn(5, rows, d, dtype=yt, pad=pad)
    ds = randn(6, rows, d, dtype=st, pad=pad) if skip else None
    w1, w2, gate = randn(3, d, dtype=wt), randn(4, d, dtype=wt), gate_of(kind, rows, d, gt)
    xb = torch.full((rows, d + pad), 7.0, dtype=BF16, device="cuda")
    rb = torch.full((rows, d + pad), 7.0, dtype=st, device="cuda")
    got = api.post_pre_rmsnorm_backward(dy, x, s, w1, w2, gate, ds, residual_scale=0.75, eps=1e-5,
                                        dx=xb[:, :d], dresidual=rb[:, :d])
    assert bool((xb[:, d:] == 7).all()) and bool((rb[:, d:] == 7).all())
    want, bounds = ref.post_pre_backward(dy, x, s, w1, w2, gate, ds, 0.75, 1e-5)
    assert (got[4] is None) == (gate is None)
    for o, w, b in zip(got, want, bounds):
        close(o, w, b + w.abs() * 1.01 * rounding(o.dtype) + 1e-30)
    again = api.post_pre_rmsnorm_backward(dy, x, s, w1, w2, gate, ds, residual_scale=0.75,
                                          eps=1e-5, dx=torch.empty_like(xb)[:, :d],
                                          dresidual=torch.empty_like(rb)[:, :d])
    for a, b in zip(again, got):
        assert a is b or torch.equal(a, b)
    # contiguous outputs: rows that begin elsewhere may be summed in another order
    other = api.post_pre_rmsnorm_backward(dy, x, s, w1, w2, gate, ds, residual_scale=0.75,
                                          eps=1e-5)
    assert other[0].dtype == xt
    for o, w, b in zip(other, want, bounds):
        close(o, w, b + w.abs() * 1.01 * rounding(o.dtype) + 1e-30)


def test_post_pre_sums_over_many_rows():
    """fp32 sums over 20000 rows: to 5e-7 rms (a sum of partial sums of 130 rows
    each loses at most some eight roundings' rms, 4e-7)."""
    rows, d = 20000, 1536
    x, s, dy, ds = (randn(i, rows, d, dtype=F32) for i in range(1, 5))
    w1, w2, gate = randn(5, d, dtype=F32), randn(6, d, dtype=F32), randn(7, d, dtype=F32)
    got = api.post_pre_rmsnorm_backward(dy, x, s, w1, w2, gate, ds)
    want, _ = ref.post_pre_backward(dy, x, s, w1, w2, gate, ds, 1.0, 1e-6)
    for o, w in zip(got, want):
        assert rms(o, w) < 5e-7


@pytest.mark.parametrize("kind", ["channel", "token"])
def test_post_pre_backward_accumulates(kind):
    rows, d = 37, 264
    x, s, dy = (randn(i, rows, d, dtype=F32) for i in range(1, 4))
    w1, w2, gate = randn(5, d, dtype=F32), randn(6, d, dtype=F32), gate_of(kind, rows, d, F32)
    one = api.post_pre_rmsnorm_backward(dy, x, s, w1, w2, gate)
    acc = [t.clone() for t in one[2:]]
    api.post_pre_rmsnorm_backward(dy, x, s, w1, w2, gate, dpost=acc[0], dpre=acc[1], dgate=acc[2],
                                  accumulate=True)
    for a, o in zip(acc, one[2:]):
        assert torch.equal(a, 2 * o)


@pytest.mark.parametrize("d", [96, 2048, 2051])
def test_post_pre_in_place(d):
    rows = 600
    x, r, dy = randn(1, rows, d), randn(2, rows, d), randn(3, rows, d)
    w1, w2 = randn(5, d, dtype=F32), randn(6, d, dtype=F32)
    s, y = api.post_pre_rmsnorm(x, r, w1, w2)
    for target in (0, 1):
        x2, r2 = x.clone(), r.clone()
        s2, y2 = api.post_pre_rmsnorm(x2, r2, w1, w2, s=(x2, r2)[target])
        assert s2 is (x2, r2)[target] and torch.equal(s2, s) and torch.equal(y2, y)
    ds = randn(4, rows, d)
    want = api.post_pre_rmsnorm_backward(dy, x, s, w1, w2, None, ds)
    for target in (0, 1):
        x2, dy2, ds2 = x.clone(), dy.clone(), ds.clone()
        got = api.post_pre_rmsnorm_backward(dy2, x2, s, w1, w2, None, ds2,
                                            dx=(x2, dy2)[target], dresidual=ds2)
        for a, b in zip(got[:4], want[:4]):
            assert torch.equal(a, b)


def test_post_pre_rows_of_zeros_infinities_and_nan():
    """A row's values reach no other row."""
    rows, d = 8, 520
    x, r = randn(1, rows, d, dtype=F32), randn(2, rows, d, dtype=F32)
    w1, w2 = randn(5, d, dtype=F32), randn(6, d, dtype=F32)
    base = api.post_pre_rmsnorm(x, r, w1, w2)
    bad = x.clone()
    bad[1] = 0
    bad[3, 5] = math.nan
    bad[5, 7] = math.inf
    s, y = api.post_pre_rmsnorm(bad, r, w1, w2)
    assert torch.equal(s[1], r[1]) and bool(torch.isfinite(y[1].float()).all())
    assert bool(torch.isnan(s[3]).all()) and bool(torch.isnan(y[5].float()).any())
    for i in (0, 2, 4, 6, 7):
        assert torch.equal(s[i], base[0][i]) and torch.equal(y[i], base[1][i])
    # zero rows and eps 0: as the formula has them, not a number
    s, y = api.post_pre_rmsnorm(torch.zeros_like(x), r, w1, w2, eps=0.0)
    assert bool(torch.isnan(s).all())


def test_post_pre_streams_and_graphs():
    rows, d = 333, 1024
    x, r, dy = randn(1, rows, d), randn(2, rows, d), randn(3, rows, d)
    w1, w2, gate = randn(5, d, dtype=F32), randn(6, d, dtype=F32), randn(7, rows, 1, dtype=F32)
    s, y = api.post_pre_rmsnorm(x, r, w1, w2, gate)
    want = (s, y) + api.post_pre_rmsnorm_backward(dy, x, s, w1, w2, gate)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s2, y2 = api.post_pre_rmsnorm(x, r, w1, w2, gate, stream=side)
    got = (s2, y2) + api.post_pre_rmsnorm_backward(dy, x, s2, w1, w2, gate, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s3, y3 = api.post_pre_rmsnorm(x, r, w1, w2, gate)
        got = (s3, y3) + api.post_pre_rmsnorm_backward(dy, x, s3, w1, w2, gate)
    for _ in range(3):
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_post_pre_empty_and_refused():
    d = 64
    x, w = randn(1, 4, d), randn(2, d)
    e = x[:0]
    s, y = api.post_pre_rmsnorm(e, e, w, w)
    assert s.shape == y.shape == (0, d)
    out = api.post_pre_rmsnorm_backward(e, e, e, w, w, w)
    assert out[0].shape == (0, d) and not any(t.any() for t in out[2:])
    big = randn(1, 2, 16392)
    with pytest.raises(_lib.MokError):
        api.post_pre_rmsnorm(big, big, randn(1, 16392), randn(1, 16392))
    for call in (lambda: api.post_pre_rmsnorm(x, x, w, w.float()),
                 lambda: api.post_pre_rmsnorm(x, x[:2], w, w),
                 lambda: api.post_pre_rmsnorm(x, x, w[:32], w),
                 lambda: api.post_pre_rmsnorm(x, x, w, w, randn(1, 4)),
                 lambda: api.post_pre_rmsnorm(x, x, w, w, randn(1, 3, 1)),
                 lambda: api.post_pre_rmsnorm(x, x, w, w, randn(1, 4, d)),
                 lambda: api.post_pre_rmsnorm(x, x, w, w, w.half()),
                 lambda: api.post_pre_rmsnorm(x, x.half(), w, w),
                 lambda: api.post_pre_rmsnorm(x, x, w, w, s=x.float()),
                 lambda: api.post_pre_rmsnorm(x, x, w, w, y=x.float()),
                 lambda: api.post_pre_rmsnorm(x, None, w, w),
                 lambda: api.post_pre_rmsnorm_backward(x, x, x, w, w, None, x.float()),
                 lambda: api.post_pre_rmsnorm_backward(x, x, x, w, w, accumulate=True),
                 lambda: api.post_pre_rmsnorm_backward(x, x, x, w, w, dgate=randn(1, d, dtype=F32)),
                 lambda: api.post_pre_rmsnorm_backward(x, x, x, w, w, dx=x.half()),
                 lambda: api.post_pre_rmsnorm_backward(x, x, x, w, w, dx_dtype=torch.float16)):
        with pytest.raises(ValueError):
            call()


# -------------------------------------- more rows than the norms' rings hold --

# (rows, d): 5 to 20 rows a block, more than a ring's slots (at most four), so that these
# are filled again; the second at a shift, rows of odd length
RINGS = [(4000, 4096), (6001, 2051), (7003, 1032)]


@pytest.mark.parametrize("rows,d", RINGS)
@pytest.mark.parametrize("xt,st", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("kind", ["none", "channel", "token"])
def test_post_pre_many_rows(rows, d, xt, st, kind):
    x, r = randn(1, rows, d, dtype=xt, scale=0.5), randn(2, rows, d, dtype=st, scale=3.0)
    w1, w2, gate = randn(3, d, dtype=F32), randn(4, d, dtype=F32), gate_of(kind, rows, d, F32)
    s, y = api.post_pre_rmsnorm(x, r, w1, w2, gate, residual_scale=0.75, eps=1e-5)
    s0, bound, norm = ref.post_pre(x, r, w1, w2, gate, 0.75, 1e-5, st)
    close(s, s0, bound)
    close(y, *norm(s))
    dy, ds = randn(5, rows, d), randn(6, rows, d, dtype=st)
    got = api.post_pre_rmsnorm_backward(dy, x, s, w1, w2, gate, ds, residual_scale=0.75, eps=1e-5)
    want, bounds = ref.post_pre_backward(dy, x, s, w1, w2, gate, ds, 0.75, 1e-5)
    for o, w, b in zip(got, want, bounds):
        close(o, w, b + w.abs() * 1.01 * rounding(o.dtype) + 1e-30)
    # in the places that mok.h allows, on another stream, and from a graph: the same bits
    for target in (0, 1):
        x2, r2 = x.clone(), r.clone()
        if target == 0 and xt != st:
            continue
        s2, y2 = api.post_pre_rmsnorm(x2, r2, w1, w2, gate, residual_scale=0.75, eps=1e-5,
                                      s=(x2, r2)[target])
        assert s2 is (x2, r2)[target] and torch.equal(s2, s) and torch.equal(y2, y)
    for target in (0, 1):
        x2, dy2, ds2 = x.clone(), dy.clone(), ds.clone()
        place = (x2, dy2)[target]
        if place.dtype != got[0].dtype:
            continue
        again = api.post_pre_rmsnorm_backward(dy2, x2, s, w1, w2, gate, ds2, residual_scale=0.75,
                                              eps=1e-5, dx=place, dresidual=ds2)
        assert again[0] is place and again[1] is ds2
        for a, b in zip(again, got):
            assert a is b or torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = api.post_pre_rmsnorm(x, r, w1, w2, gate, residual_scale=0.75, eps=1e-5, stream=side)
    other += api.post_pre_rmsnorm_backward(dy, x, other[0], w1, w2, gate, ds, residual_scale=0.75,
                                           eps=1e-5, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = api.post_pre_rmsnorm(x, r, w1, w2, gate, residual_scale=0.75, eps=1e-5)
        kept += api.post_pre_rmsnorm_backward(dy, x, kept[0], w1, w2, gate, ds,
                                              residual_scale=0.75, eps=1e-5)
    graph.replay()
    graph.replay()
    for a, b, c in zip(other, kept, (s, y) + tuple(got)):
        assert (a is None and b is None) or (torch.equal(a, c) and torch.equal(b, c))
