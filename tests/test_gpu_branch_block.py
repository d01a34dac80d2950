"""The branch operators as a model uses them: the MoE block with a norm after the one
before it, its gate and residual scale and dropout (bars as the layer's: max|diff| <=
2e-2 rms per tensor), and experts of grouped products between a dispatch plan and the
next block's norms (a bound on the rms of the difference, derived at its test), each
against a plain float64 computation with autograd on the kernel's own routing and
masks."""
import pytest
import torch

import _branch_ref as bref
from _block_ref import U16
from routing_dispatch_grouped_router_gb300 import api, block
from test_gpu_moe_block import plain_block

pytestmark = pytest.mark.gpu
F32, F64 = torch.float32, torch.float64
SEED, STEP = 77, 5


def within(got, want, name):
    want = want.detach()
    rms = want.pow(2).mean().sqrt().item()
    err = (got.to(F64) - want).abs().max().item() / rms
    assert err <= 2e-2 * max(1.0, (want.abs().max().item() / rms) / 4), (name, err)


def mask_of(rows, d, p, site):
    keep = bref.dropout_words(SEED, STEP, site, 0, rows * d, "cuda").reshape(rows, d) \
        >= round(p * 2 ** 32)
    return keep.to(F64) / (1 - p)


def norm(v, w, eps):
    return v * (v.pow(2).mean(1, keepdim=True) + eps).rsqrt() * w


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,d,E,I,k,F", [(256, 128, 8, 256, 2, 192), (130, 160, 5, 224, 3, 72)])
def test_block_with_post_norm_and_dropout(T, d, E, I, k, F, gated):
    gen = torch.Generator(device="cuda").manual_seed(T)

    def rnd(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    w = {"norm": 1 + rnd(d, scale=0.1, dtype=F32), "post": 1 + rnd(d, scale=0.1, dtype=F32),
         "w_router": rnd(E, d, scale=d ** -0.5), "w_gate_up": rnd(E, 2 * I, d, scale=d ** -0.5),
         "w_down": rnd(E, d, I, scale=I ** -0.5), "w_up": rnd(F, d, scale=d ** -0.5),
         "b_up": rnd(F, scale=0.1, dtype=F32), "w_out": rnd(d, F, scale=F ** -0.5),
         "b_out": rnd(d, scale=0.1, dtype=F32)}
    if gated:
        w["gate"] = 0.5 + rnd(d, scale=0.2, dtype=F32)
    x, residual = rnd(T, d, dtype=F32), rnd(T, d, scale=2.0, dtype=F32)
    dout, ds = rnd(T, d), rnd(T, d, dtype=F32)
    dloss = torch.tensor([3.0, 5.0], device="cuda") * T
    mask = (torch.rand(T, generator=gen, device="cuda") > 0.2).to(torch.uint8)
    p, alpha, site = 0.25, 0.8, 3
    blk = block.MoEBlock(T, d, E, I, k, balance_coef=0.5, z_coef=0.25, post_norm=True,
                         residual_scale=alpha, dropout=p, site=site)
    rng = torch.tensor([SEED, STEP], device="cuda")
    with pytest.raises(ValueError):
        blk.forward(x, residual, w, mask)
    out, s, loss, counts = blk.forward(x, residual, w, mask, rng)
    dx, dresidual, g = blk.backward(dout, ds, dloss, w)
    assert blk.status() == 0
    idx = blk.layer.saved_tensor("topk_idx", torch.int32, (T, k)).long()
    ww = {n: t.to(F64).requires_grad_() for n, t in w.items()}
    xx, rr = x.to(F64).requires_grad_(), residual.to(F64).requires_grad_()
    s0 = alpha * rr + norm(xx, ww["post"], blk.eps) * (ww["gate"] if gated else 1.0)
    # plain_block adds its two inputs: the stream and nothing
    o0, _, l0 = plain_block(s0, torch.zeros_like(s0), ww, idx, k, mask, blk.act, blk.eps, 0.5, 0.25)
    o0 = o0 * mask_of(T, d, p, site)
    total = (o0 * dout.to(F64)).sum() + (s0 * ds.to(F64)).sum() + (l0 * dloss.to(F64)).sum()
    total.backward()
    for name, a, b in [("out", out, o0), ("s", s, s0), ("loss", loss, l0), ("dx", dx, xx.grad),
                       ("dresidual", dresidual, rr.grad)] + [(n, g[n], ww[n].grad) for n in w]:
        within(a, b, name)


@pytest.mark.parametrize("T,d,F,E,k", [(300, 128, 264, 16, 4), (1, 256, 72, 8, 2), (97, 136, 80, 5, 3)])
def test_grouped_experts_between_norms(T, d, F, E, k):
    """post_pre_rmsnorm -> plan -> grouped experts -> dropout -> post_pre_rmsnorm,
    forward and backward, and the same bits again from a captured graph.

    The bound: n1, z, h, do, dz are rounded to bf16, each a relative error of at most
    u16, uniform within it (rms u16 / sqrt(3)) and independent from element to element.
    The output that most of them reach is dw_up, the sum of dz n1: n1's enters it as
    an operand, through relu(z) in dz and, doubled by the square, through y in the
    norm's gradient, 1 + 1 + 2 at most; z's likewise 1 + 2; those of h, do and dz 1
    each, together sqrt((16 + 9 + 3) / 3) u16 = 3.06 u16 (the outputs' own rounding,
    of n2 or dx, in place of one of these).  A sum of terms with independent errors is
    off by the root of the sum of their squares, the size of a sum that does not
    cancel.  The gradients of the slots' weights do: the gradient of a norm's input is
    orthogonal to that input, of which they are its products with the parts.  They are
    compared at the size of the root of the sum of their terms' squares."""
    gen = torch.Generator(device="cuda").manual_seed(T)

    def rnd(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    p, site, alpha, eps = 0.2, 1, 0.9, 1e-6
    x, r = rnd(T, d), rnd(T, d, scale=2.0, dtype=F32)
    v1, v2, v3, v4 = (1 + rnd(d, scale=0.1, dtype=F32) for _ in range(4))
    gate = 0.5 + rnd(T, 1, scale=0.2, dtype=F32)
    wu, wd = rnd(E, F, d, scale=d ** -0.5), rnd(E, d, F, scale=F ** -0.5)
    idx = torch.stack([torch.randperm(E, generator=gen, device="cuda")[:k] for _ in range(T)]).int()
    tw = torch.softmax(rnd(T, k, dtype=F32), 1)
    dy, ds2 = rnd(T, d), rnd(T, d, dtype=F32)
    rng = torch.tensor([SEED, STEP], device="cuda")
    desc = api.make_desc(T, 128, E, 128, k)
    plan = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1)] + \
        [torch.empty(T, k, dtype=torch.int32, device="cuda"),
         torch.empty(T * k, dtype=torch.int32, device="cuda")]
    ws = torch.empty(api.stage_workspace_size(desc), dtype=torch.uint8, device="cuda")
    experts = block.GroupedExperts()

    def step():
        counts, off, pos, rows = plan
        api.dispatch_plan(desc, idx, counts, off, pos, rows, ws)
        s1, n1 = api.post_pre_rmsnorm(x, r, v1, v2, gate, residual_scale=alpha, eps=eps)
        y = experts.forward(n1, tw, off, rows, pos, wu, wd)
        b = api.dropout(y, p, rng, site)
        s2, n2 = api.post_pre_rmsnorm(b, s1, v3, v4, eps=eps)
        db, ds1, dv3, dv4, _ = api.post_pre_rmsnorm_backward(dy, b, s2, v3, v4, None, ds2, eps=eps)
        dyy = api.dropout_backward(db, p, rng, site)
        dn1, dtw, dwu, dwd = experts.backward(dyy, wu, wd)
        dx, dr, dv1, dv2, dgate = api.post_pre_rmsnorm_backward(
            dn1, x, s1, v1, v2, gate, ds1, residual_scale=alpha, eps=eps)
        return [n2, s2, dx, dr, dv1, dv2, dgate, dv3, dv4, dwu, dwd, dtw]

    got = step()
    assert api.device_status(api.operator_status()) == 0
    leaves = [t.to(F64).requires_grad_() for t in (x, r, v1, v2, gate, v3, v4, wu, wd, tw)]
    xx, rr, a1, a2, gg, a3, a4, uu, dd, tt = leaves
    s1 = alpha * rr + gg * norm(xx, a1, eps)
    n1 = norm(s1, a2, eps)
    h = torch.einsum("td,tkfd->tkf", n1, uu[idx.long()]).clamp(min=0) ** 2
    o = torch.einsum("tkf,tkdf->tkd", h, dd[idx.long()])
    y = torch.einsum("tk,tkd->td", tt, o)
    y.retain_grad()
    s2 = s1 + norm(y * mask_of(T, d, p, site), a3, eps)
    n2 = norm(s2, a4, eps)
    ((n2 * dy.to(F64)).sum() + (s2 * ds2.to(F64)).sum()).backward()
    want = [n2, s2] + [t.grad for t in leaves]
    names = ["n2", "s2", "dx", "dr", "dv1", "dv2", "dgate", "dv3", "dv4", "dwu", "dwd", "dtw"]
    for name, a, b in zip(names, got, want):
        b = b.detach()
        size = b.pow(2).mean() if name != "dtw" else \
            (y.grad.unsqueeze(1) * o.detach()).pow(2).sum(2).mean()
        err = ((a.to(F64) - b).pow(2).mean() / size).sqrt().item()
        assert err <= 3.06 * U16, (name, err)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = step()
    for _ in range(2):
        graph.replay()
    for name, a, b in zip(names, again, got):
        assert torch.equal(a, b), name


def test_grouped_experts_of_a_plan_with_bad_indices():
    """The plan reports them and skips their slots: as a plan of weight 0 there, with any
    value in the words that the plan leaves unwritten."""
    T, d, F, E, k = 61, 136, 80, 5, 3
    gen = torch.Generator(device="cuda").manual_seed(2)

    def rnd(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    x, dy = rnd(T, d), rnd(T, d, dtype=F32)
    wu, wd = rnd(E, F, d, scale=d ** -0.5), rnd(E, d, F, scale=F ** -0.5)
    idx = torch.stack([torch.randperm(E, generator=gen, device="cuda")[:k] for _ in range(T)]).int()
    bad = torch.rand(T, k, generator=gen, device="cuda") < 0.3
    bad[7] = True
    tw = torch.softmax(rnd(T, k, dtype=F32), 1)
    desc = api.make_desc(T, 128, E, 128, k)
    outs = []
    for skip in (False, True):
        counts, off = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1))
        pos = torch.empty(T, k, dtype=torch.int32, device="cuda")
        rows = torch.full((T * k,), (1 << 31) - 1, dtype=torch.int32, device="cuda")
        ws = torch.empty(api.stage_workspace_size(desc), dtype=torch.uint8, device="cuda")
        at = torch.where(bad, torch.where(idx > 2, -1, E), idx).int() if skip else idx
        api.dispatch_plan(desc, at, counts, off, pos, rows, ws)
        assert api.device_status(ws) == (17 if skip else 0)
        assert (pos < 0).sum().item() == (bad.sum().item() if skip else 0)
        experts = block.GroupedExperts()
        y = experts.forward(x, tw if skip else tw.masked_fill(bad, 0.0), off, rows, pos, wu, wd)
        outs.append((y,) + experts.backward(dy, wu, wd))
    assert api.device_status(api.operator_status()) == 0
    for a, b in zip(*outs):
        assert bool(torch.isfinite(b).all())
    # y, dx, the weights' gradients are sums of the same terms and zeros, in groups whose
    # rows lie elsewhere: fp32 sums of at most F, d or T k terms in another order, and
    # bf16 roundings (h, dz of equal fp32 values) that may fall to the other side
    (y0, dx0, dt0, du0, dd0), (y1, dx1, dt1, du1, dd1) = outs
    assert not dt1[bad].any()
    for a, b in ((y0, y1), (dx0, dx1), (dt0[~bad], dt1[~bad]), (du0, du1), (dd0, dd1)):
        err = ((a - b).pow(2).mean() / a.pow(2).mean()).sqrt().item()
        assert err <= U16, err
    assert not y1[7].any() and not dx1[7].any()


@pytest.mark.parametrize("T,k", [(1, 2), (40, 4), (4096, 8)])
def test_grouped_experts_do_not_follow_torchs_tf32(T, k):
    """Torch's switch for its own products changes nothing in fp32 here: the same bits."""
    d, F, E = 1024, 128, 16
    gen = torch.Generator(device="cuda").manual_seed(T)

    def rnd(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    x, dy = rnd(T, d), rnd(T, d, dtype=F32)
    wu, wd = rnd(E, F, d, scale=d ** -0.5), rnd(E, d, F, scale=F ** -0.5)
    idx = torch.stack([torch.randperm(E, generator=gen, device="cuda")[:k] for _ in range(T)])
    tw = torch.softmax(rnd(T, k, dtype=F32), 1)
    flat = idx.reshape(-1)
    order = torch.argsort(flat, stable=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    pos = torch.empty(T * k, dtype=torch.int32, device="cuda")
    pos[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    before, outs = torch.backends.cuda.matmul.allow_tf32, []
    try:
        for tf32 in (False, True):
            torch.backends.cuda.matmul.allow_tf32 = tf32
            experts = block.GroupedExperts()
            y = experts.forward(x, tw, off, (order // k).int(), pos.view(T, k), wu, wd)
            outs.append((y,) + experts.backward(dy, wu, wd))
    finally:
        torch.backends.cuda.matmul.allow_tf32 = before
    for a, b in zip(*outs):
        assert torch.equal(a, b)
