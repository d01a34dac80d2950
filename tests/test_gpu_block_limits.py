"""The operators around the layer where a first form of them went wrong: logits
far from zero, tensors of more rows or features than one grid dimension holds,
norms beside a rounding boundary of E4M3, calls from several host threads.  Bounds
as in _block_ref.py, and as derived at each test."""
import ctypes
import math
import threading

import pytest
import torch

import _block_ref as ref
from _block_ref import F64, U16, U32
from routing_dispatch_grouped_router_gb300 import _lib, api, block

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def randn(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def within(got, want, bound):
    """|got - want| <= bound everywhere; the largest excess otherwise."""
    d = (got.to(F64) - want).abs() - bound
    assert torch.isfinite(got).all()
    assert d.max().item() <= 0, (d.max().item(), (got.to(F64) - want).abs().max().item())


# ---------------------------------------------------------- router_balance --

@pytest.mark.parametrize("T,E,k", [(60, 40, 4), (33, 8, 2), (50, 130, 8), (9, 512, 8), (40, 17, 1),
                                   (21, 300, 3)])
@pytest.mark.parametrize("offset", [0.0, 1e4, -1e4, 3e6, -1e8, -3e37])
def test_balance_gradient_of_rows_far_from_zero(T, E, k, offset):
    """A row's softmax does not change with an offset of all its logits, however
    large its lse: every other row of the batch is moved far away."""
    l = randn(1000 + T, T, E, dtype=F32)
    l[::2] += offset
    idx = torch.topk(l, k, 1).indices.to(torch.int32)
    check_gradient(l, idx, None, 0.5, 1e-3)


def check_gradient(l, idx, mask, a, b):
    T, E = l.shape
    u = torch.tensor([1.25, -0.75], device="cuda")
    _, counts, prob, lse, n = api.router_balance(l, idx, mask, balance_coef=a, z_coef=b)
    dl = api.router_balance_backward(u, l, lse, counts, n, idx.shape[1], mask, balance_coef=a,
                                     z_coef=b)
    _, counts0, prob0, lse0, n0, p, m, f, some = ref.router_balance(l, idx, mask, a, b)
    assert torch.equal(counts, counts0)
    x = torch.where(some[:, None], l.to(F64), torch.zeros_like(l, dtype=F64))
    # softmax: E positive terms; an exponential of l - max (one rounding of an
    # argument that matters down to -104), for each row by itself
    far = (x - x.amax(1, keepdim=True)).abs().clamp(max=104.0).amax(1, keepdim=True)
    soft = (2 * E + 4 * far + 64) * U32
    within(prob, prob0, prob0 * (soft.amax() + 2 * T * U32) + 1e-30)
    dl0 = ref.router_balance_backward(u, l, idx, mask, a, b)
    z0 = torch.where(some, lse0, torch.zeros_like(lse0)).abs()[:, None]
    mag = p * (1.25 * a * E * (f + (p @ f)[:, None] + 1.0 / E) + 0.75 * 2 * b * z0) / max(n0, 1)
    within(dl, dl0, mag * (2 * soft + (4 * E + 64) * U32) + 1e-30)
    return dl


def test_balance_gradient_of_rows_of_the_lowest_value():
    """Rows masked with the type's lowest value, whole or in part, with and
    without the z loss in the gradient."""
    low = torch.finfo(F32).min
    l = randn(1100, 64, 40, dtype=F32)
    l[3] = low
    l[5, :36] = low
    l[8] = low / 2
    l[9, 1:] = -math.inf
    l[11] = -math.inf
    idx = torch.topk(l, 4, 1).indices.to(torch.int32)
    for b in (0.0, 1e-3):
        dl = check_gradient(l, idx, None, 0.5, b)
        assert (dl[11] == 0).all()
    mask = torch.ones(64, dtype=torch.uint8, device="cuda")
    mask[5:9] = 0
    assert (check_gradient(l, idx, mask, 0.5, 0.0)[5:9] == 0).all()


# ----------------------------------------------------------------- linear --

@pytest.mark.parametrize("act,dyt,bias", [("none", F32, True), ("silu", BF16, False)])
def test_linear_backward_of_two_million_tokens(act, dyt, bias):
    """More than 65535 blocks of 32 rows: dz, its column sums and products."""
    M, N, K = 65535 * 32 + 33, 8, 8
    x, w = randn(1200, M, K), randn(1201, N, K)
    dy, z = randn(1202, M, N, dtype=dyt), randn(1203, M, N, dtype=dyt)
    dx, dw, db = api.linear_backward(dy, x, w, z, act=act, bias=bias, dx_dtype=F32)
    assert api.device_status(api.operator_status()) == 0
    (dx0, dw0, db0), (mx, mw, mb) = ref.linear_backward(dy, x, w, z, act)
    dza = dy.to(F64).abs() * (0.0 if act == "none" else 64 * U32)
    within(dx, dx0, mx * (6 * N + 1) * U32 + dza @ w.to(F64).abs() + 1e-30)
    # 36 products to an accumulation, then sums in fp32 over the chunks of a split
    # and over the splits: errors that do not line up, so well below M U32
    rms = lambda t: t.pow(2).mean().sqrt().item()  # noqa: E731
    assert rms(dw.to(F64) - dw0) <= 1e-4 * rms(dw0)
    if bias:
        assert rms(db.to(F64) - db0) <= 1e-4 * rms(db0)


@pytest.mark.parametrize("M", [1, 5, 16, 100])
def test_linear_of_more_features_than_a_grid_dimension(M):
    """N beyond 65535 tiles of 128 features, few tokens."""
    N, K = 65535 * 128 + 130, 8
    x, w = randn(1300, M, K), randn(1301, N, K)
    y = api.linear(x, w)
    assert api.device_status(api.operator_status()) == 0
    for n0 in (0, 65534 * 128, N - 200):
        n1 = min(n0 + 300, N)
        y0, _, mag = ref.linear(x, w[n0:n1], None, "none", None)
        within(y[:, n0:n1], y0, y0.abs() * 1.01 * U16 + mag * (2 * K + 8) * U32 + 1e-30)


# ------------------------------------------------------- status, arguments --

def test_operator_status_is_one_word_however_the_device_is_named():
    word = api.operator_status()
    i = torch.cuda.current_device()
    for name in ("cuda", f"cuda:{i}", i, torch.device("cuda"), torch.device("cuda", i)):
        assert api.operator_status(name).data_ptr() == word.data_ptr()
    for name in ("cpu", torch.device("cpu")):
        with pytest.raises(ValueError):
            api.operator_status(name)


def test_arguments_without_a_truth_value():
    """A tensor of several elements for a flag raises ValueError, and no call is made."""
    x, w, b = randn(1500, 4, 64), randn(1501, 8, 64), torch.zeros(8, device="cuda")
    ones, dy = torch.ones(64, device="cuda"), randn(1502, 4, 8)
    dw = torch.zeros(64, device="cuda")
    for call in (lambda: api.linear(x, w, keep_z=b),
                 lambda: api.linear_backward(dy, x, w, bias=b),
                 lambda: api.add_rmsnorm_backward(x, x, ones, dweight=dw, accumulate=b)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert (dw == 0).all()


# ------------------------------------------------------------ host threads --

def test_norm_backward_from_several_host_threads():
    """The C entry from three threads at once, each with a width and a stream of its
    own: no call fails, and every result is the call's alone."""
    lib = _lib.load()
    fail, result = [], {}
    jobs = {}
    for i, d in enumerate((1024, 7168, 2048)):
        dy, s, w = randn(1400 + i, 64, d), randn(1410 + i, 64, d), randn(1420 + i, d, dtype=F32)
        dx0, dw0 = api.add_rmsnorm_backward(dy, s, w)
        desc = _lib.RmsnormDesc(rows=64, d=d, eps=1e-6, weight_elem=1)
        n = ctypes.c_size_t()
        assert lib.mok_add_rmsnorm_workspace_size(desc, n) == 0
        ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
        jobs[d] = (desc, dy, s, w, torch.zeros_like(dx0), torch.zeros_like(dw0), ws, dx0, dw0,
                   torch.cuda.Stream())
    torch.cuda.synchronize()
    go = threading.Barrier(len(jobs))

    def work(d):
        desc, dy, s, w, dx, dw, ws, _, _, st = jobs[d]
        go.wait()
        for _ in range(4000):
            rc = lib.mok_add_rmsnorm_backward(
                desc, dy.data_ptr(), s.data_ptr(), w.data_ptr(), None, dx.data_ptr(),
                dw.data_ptr(), ws.data_ptr(), ws.numel(), None, st.cuda_stream)
            if rc != 0:
                fail.append((d, rc))

    threads = [threading.Thread(target=work, args=(d,)) for d in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not fail, (len(fail), fail[:4])
    for d, (_, _, _, _, dx, dw, _, dx0, dw0, _) in jobs.items():
        assert torch.equal(dx, dx0) and torch.equal(dw, dw0), d


def test_a_refused_launch_leaves_no_pending_error():
    """A call that the runtime refuses (here: its stream's capture has been
    invalidated) says so in its status; the runtime's error does not wait for the
    next call of the process."""
    lib = _lib.load()
    stream = ctypes.c_void_p()
    assert lib.cudaStreamCreateWithFlags(ctypes.byref(stream), 1) == 0
    x, w = randn(1510, 4, 64), torch.ones(64, device="cuda")
    y = torch.empty_like(x)
    wl, out = randn(1511, 8, 64), torch.empty(4, 8, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    try:
        assert lib.cudaStreamBeginCapture(stream, 2) == 0  # relaxed: this stream alone
        assert lib.cudaStreamSynchronize(stream) != 0      # not allowed in a capture: ends it
        lib.cudaGetLastError()
        norm = _lib.RmsnormDesc(rows=4, d=64, eps=1e-6, weight_elem=1)
        assert lib.mok_add_rmsnorm_forward(norm, x.data_ptr(), None, w.data_ptr(), None,
                                           y.data_ptr(), None, None, None, stream) == 4
        assert lib.cudaPeekAtLastError() == 0
        lin = _lib.LinearDesc(M=4, N=8, K=64)
        assert lib.mok_linear_forward(lin, x.data_ptr(), wl.data_ptr(), None, None, out.data_ptr(),
                                      None, None, 0, None, stream) == 4
        assert lib.cudaPeekAtLastError() == 0
    finally:
        graph = ctypes.c_void_p()
        lib.cudaStreamEndCapture(stream, ctypes.byref(graph))
        lib.cudaStreamDestroy(stream)
        lib.cudaGetLastError()
    torch.cuda.synchronize()
    assert torch.equal(api.add_rmsnorm(x, w)[1], api.add_rmsnorm(x, w)[1])


# ------------------------------------------------------- precision of MXFP8 --

# The MXFP8 form of the norm: mean square, reciprocal root and products in pairs
# of fp32.  The root's Newton step leaves 3/8 of the square of rsqrtf's error
# (2 ulp: 2^-22.4 relative, so 2^-46), each product and sum some 2^-46: in all below
# 2^-42.  Codes and scales are those of the exact norm wherever no boundary of
# theirs lies that near.
MX_ERR = 2.0 ** -42


def check_mx(x, w, eps, residual=None):
    values = torch.empty(x.shape, dtype=BF16, device="cuda")
    _, codes, scales = api.add_rmsnorm_mx(x, w, residual, eps=eps, values=values)
    y0 = ref.add_rmsnorm(x, w, residual, eps)[1]
    (lo, slo), (hi, shi) = (ref.mx_values(y0 * (1 + e)) for e in (-MX_ERR, MX_ERR))
    sure, ssure = lo == hi, slo == shi
    assert sure.double().mean().item() > 0.999 and ssure.double().mean().item() > 0.99
    assert torch.equal(values.to(F64)[sure], lo[sure])
    assert torch.equal(scales[ssure], slo[ssure])
    assert torch.equal(values.to(F64), ref.decode(codes, scales))


@pytest.mark.parametrize("d", [32, 96, 2880, 4096, 16384])
@pytest.mark.parametrize("rows", [1, 700])
def test_mx_codes_of_norms_beside_a_rounding_boundary(rows, d):
    """Rows of one magnitude c: every square has the same rounding error in fp32.
    eps puts the norm 1e-10 above or below the middle of two codes."""
    b = 1.0625  # between the codes of 1 and 1.125
    w1 = torch.nextafter(torch.tensor(b), torch.tensor(2.0)).item()
    w = torch.full((d,), w1, device="cuda")
    g = w1 / b - 1
    sign = torch.where(randn(1600, rows, d, dtype=F32) < 0, -1.0, 1.0)
    for c in (1.2345678, 0.7654321, 3.3333333, 1.1, 0.01234567):
        c = torch.tensor(c, dtype=F32).item()
        for delta in (1e-10, -1e-10):
            eps = c * c * (((1 + g) / (1 + delta)) ** 2 - 1)
            eps = torch.tensor(eps, dtype=F32).item()
            x = sign * c
            y0 = ref.add_rmsnorm(x, w, None, eps)[1].abs()
            assert ((y0 / b - 1).abs() > MX_ERR).all() and ((y0 > b) == (delta > 0)).all()
            check_mx(x, w, eps)


@pytest.mark.parametrize("xt,st", [(F32, None), (BF16, F32), (F32, BF16), (BF16, BF16)])
def test_mx_codes_are_the_exact_norm_s(xt, st):
    """Eight million values of random rows, of which an fp32 norm rounds some eight
    the other way; a part of them in rows of odd strides."""
    x = randn(1700, 2048, 4096, dtype=xt)
    r = None if st is None else randn(1701, 2048, 4096, dtype=st, scale=3.0)
    w = 1 + randn(1702, 4096, dtype=F32, scale=0.1)
    check_mx(x, w, 1e-6, r)
    y = torch.empty(700, 4097, dtype=xt, device="cuda")[:, :4096]
    y.copy_(x[:700])
    check_mx(y, w, 1e-6, None if r is None else r[:700])


# ------------------------------------------- precision of weight gradients --

@pytest.mark.parametrize("M,N,K", [(16384, 128, 512), (4096, 256, 512), (12000, 130, 256),
                                   (9000, 64, 512), (600, 40, 1032)])
@pytest.mark.parametrize("act,dyt", [("none", F32), ("silu", BF16)])
def test_linear_backward_keeps_fp32_accuracy_over_many_tokens(M, N, K, act, dyt):
    """dw and an fp32 dx take all 24 bits of dz and few MMAs per accumulation.  A
    truncating MMA costs a sum up to 1.7e-8 of it, 36 of them 6e-7 (half of that
    on average, and less as the chunks' sums join: a chunk's error is relative to
    the chunk); the sums in fp32 beside it some 3e-7, the slope's exponential up to
    3e-7: in all 1.5e-6.  Two parts of dz alone would leave 2^-17 / sqrt(12) = 2.2e-6."""
    x, w = randn(1800, M, K), randn(1801, N, K, scale=1 / math.sqrt(K))
    dy, z = randn(1802, M, N, dtype=dyt), randn(1803, M, N, dtype=dyt)
    dx, dw, _ = api.linear_backward(dy, x, w, z, act=act, dx_dtype=F32)
    (dx0, dw0, _), _ = ref.linear_backward(dy, x, w, z, act)

    def err(got, want):
        return ((got.to(F64) - want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt()).item()

    assert err(dx, dx0) <= 1.5e-6 and err(dw, dw0) <= 1.5e-6, (err(dx, dx0), err(dw, dw0))
    # the bound tells two parts from three: two, in an exact product, are beyond it
    dz = dy.to(F64) if act == "none" else dy.to(F64) * ref.act(z.to(F64), act)[1]
    one = dz.to(BF16).to(F64)
    two = one + (dz - one).to(BF16).to(F64)
    assert err(two.T @ x.to(F64), dw0) > 1.5e-6 and err(two @ w.to(F64), dx0) > 1.5e-6


@pytest.mark.parametrize("M,N,K", [(40, 64, 136), (700, 264, 520), (3000, 1024, 256)])
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_linear_backward_of_a_plain_dy_in_the_stated_scratch(M, N, K, offset):
    """A bf16 dy without an activation, at an offset of its own, through the C entry
    in exactly the scratch that the size query states for it; less is refused."""
    x, w = randn(1900, M, K), randn(1901, N, K, scale=1 / math.sqrt(K))
    dy = randn(1902, M * N + 8)[offset:offset + M * N].view(M, N)
    dx, dw, db = (torch.empty(s, device="cuda") for s in ((M, K), (N, K), (N,)))
    d = _lib.LinearDesc(M=M, N=N, K=K, dx_elem=1)
    n, lib = ctypes.c_size_t(), _lib.load()
    assert lib.mok_linear_workspace_size(d, 1 if offset else 2, n) == 0
    buf = torch.full((n.value + 256,), 91, dtype=torch.uint8, device="cuda")
    ptrs = [t.data_ptr() for t in (dy, x, w)] + [None] + [t.data_ptr() for t in (dx, dw, db, buf)]
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.mok_linear_backward(d, *ptrs, n.value - 1, None, stream) == 3
    assert lib.mok_linear_backward(d, *ptrs, n.value, None, stream) == 0
    assert (buf[n.value:] == 91).all()
    (dx0, dw0, db0), (mx, mw, mb) = ref.linear_backward(dy, x, w, None, "none")
    within(dx, dx0, mx * (2 * N + 2) * U32 + 1e-30)
    within(dw, dw0, mw * (2 * M + 16) * U32 + 1e-30)
    within(db, db0, mb * (2 * M + 16) * U32 + 1e-30)
    for got, want in zip(api.linear_backward(dy, x, w, bias=True, dx_dtype=F32), (dx, dw, db)):
        assert torch.equal(got, want)


# ------------------------------------------------------------ the MoE block --

@pytest.mark.parametrize("dtype", [api.BF16, api.MXFP8, api.NVFP4])
def test_block_is_its_calls_in_every_type_of_the_layer(dtype):
    """MoEBlock gives, bit for bit, what its operators and a layer of that type give
    called one by one."""
    T, d, E, I, k, F = 200, 256, 8, 256, 2, 264
    w = {"norm": 1 + randn(2000, d, dtype=F32, scale=0.1), "w_router": randn(2001, E, d, scale=d ** -0.5),
         "w_gate_up": randn(2002, E, 2 * I, d, scale=d ** -0.5),
         "w_down": randn(2003, E, d, I, scale=I ** -0.5), "w_up": randn(2004, F, d, scale=d ** -0.5),
         "b_up": randn(2005, F, dtype=F32, scale=0.1), "w_out": randn(2006, d, F, scale=F ** -0.5),
         "b_out": randn(2007, d, dtype=F32, scale=0.1)}
    x, r, dout = randn(2008, T, d, dtype=F32), randn(2009, T, d), randn(2010, T, d)
    dloss = torch.tensor([1.5, 0.5], device="cuda")
    blk = block.MoEBlock(T, d, E, I, k, act="gelu", dtype=dtype)
    out, s, loss, counts = blk.forward(x, r, w)
    dx, g = blk.backward(dout, None, dloss, w)
    assert blk.status() == 0

    layer = api.MoELayer(T, d, E, I, k, dtype=dtype)
    s0, n = api.add_rmsnorm(x, w["norm"], r, eps=blk.eps)
    routed = layer.forward(n, w["w_router"], None, w["w_gate_up"], w["w_down"])
    logits = api.linear(n, w["w_router"], out_dtype=F32)
    idx = layer.saved_tensor("topk_idx", torch.int32, (T, k))
    loss0, counts0, _, lse, nv = api.router_balance(logits, idx, **blk.coefs)
    h, z = api.linear(n, w["w_up"], w["b_up"], act="gelu", keep_z=True)
    out0 = api.linear(h, w["w_out"], w["b_out"], residual=routed, out_dtype=F32)
    for got, want in ((out, out0), (s, s0), (loss, loss0), (counts, counts0)):
        assert torch.equal(got, want)
    dn, wr, wgu, wd = layer.backward(dout, n, w["w_router"], None, w["w_gate_up"], w["w_down"])
    dh, wo, bo = api.linear_backward(dout, h, w["w_out"], bias=True)
    _, wu, bu = api.linear_backward(dh, n, w["w_up"], z, act="gelu", bias=True, dx=dn,
                                    accumulate="dx")
    dl = api.router_balance_backward(dloss, logits, lse, counts, nv, k, **blk.coefs)
    api.linear_backward(dl, n, w["w_router"], dx=dn, dw=wr, accumulate=True)
    dx0, wn = api.add_rmsnorm_backward(dn, s, w["norm"], eps=blk.eps)
    assert torch.equal(dx, dx0)
    for name, want in (("norm", wn), ("w_router", wr), ("w_gate_up", wgu), ("w_down", wd),
                       ("w_up", wu), ("b_up", bu), ("w_out", wo), ("b_out", bo)):
        assert torch.equal(g[name], want), name
