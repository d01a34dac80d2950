"""The MoE block (norm, layer, shared expert, auxiliary losses) against a plain
float64 computation with autograd, on the kernel's own routing; bars as the
layer's: max|diff| <= 2e-2 rms per tensor."""
import pytest
import torch

import _block_ref as ref
from routing_dispatch_grouped_router_gb300 import api, block

pytestmark = pytest.mark.gpu
F64 = torch.float64


def plain_block(x, residual, w, idx, k, mask, act, eps, a, b):
    s = x + residual
    n = s * (s.pow(2).mean(1, keepdim=True) + eps).rsqrt() * w["norm"]
    logits = n @ w["w_router"].T
    E, I = w["w_router"].shape[0], w["w_down"].shape[2]
    p = torch.softmax(logits.gather(1, idx), 1)
    routed = torch.zeros_like(n)
    for e in range(E):
        t, slot = torch.nonzero(idx == e, as_tuple=True)
        gu = n[t] @ w["w_gate_up"][e].T
        o = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ w["w_down"][e].T
        routed = routed.index_add(0, t, p[t, slot, None] * o)
    h = ref.act(n @ w["w_up"].T + w["b_up"], act)[0]
    out = routed + h @ w["w_out"].T + w["b_out"]
    m = mask.to(F64)
    prob = (m[:, None] * torch.softmax(logits, 1)).sum(0) / m.sum()
    f = torch.bincount(idx[mask > 0].reshape(-1), minlength=E).to(F64) / (m.sum() * k)
    loss = torch.stack([a * E * (f * prob).sum(),
                        b * (m * torch.logsumexp(logits, 1) ** 2).sum() / m.sum()])
    return out, s, loss


@pytest.mark.parametrize("T,d,E,I,k,F,act", [(256, 128, 8, 256, 2, 192, "silu"),
                                             (130, 160, 5, 224, 3, 72, "gelu"),
                                             (1, 256, 16, 128, 4, 264, "relu")])
def test_block(T, d, E, I, k, F, act):
    gen = torch.Generator(device="cuda").manual_seed(T)

    def rnd(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    w = {"norm": 1 + rnd(d, scale=0.1, dtype=torch.float32), "w_router": rnd(E, d, scale=d ** -0.5),
         "w_gate_up": rnd(E, 2 * I, d, scale=d ** -0.5), "w_down": rnd(E, d, I, scale=I ** -0.5),
         "w_up": rnd(F, d, scale=d ** -0.5), "b_up": rnd(F, scale=0.1, dtype=torch.float32),
         "w_out": rnd(d, F, scale=F ** -0.5), "b_out": rnd(d, scale=0.1, dtype=torch.float32)}
    x, residual = rnd(T, d, dtype=torch.float32), rnd(T, d, scale=2.0, dtype=torch.float32)
    dout, ds = rnd(T, d), rnd(T, d, dtype=torch.float32)
    dloss = torch.tensor([3.0, 5.0], device="cuda") * T
    mask = (torch.rand(T, generator=gen, device="cuda") > 0.2).to(torch.uint8)
    mask[0] = 1
    blk = block.MoEBlock(T, d, E, I, k, act=act, balance_coef=0.5, z_coef=0.25)
    out, s, loss, counts = blk.forward(x, residual, w, mask)
    dx, g = blk.backward(dout, ds, dloss, w)
    assert blk.status() == 0
    idx = blk.layer.saved_tensor("topk_idx", torch.int32, (T, k)).long()
    assert torch.equal(counts.long(), torch.bincount(idx[mask > 0].reshape(-1), minlength=E))

    ww = {n: t.to(F64).requires_grad_() for n, t in w.items()}
    xx = x.to(F64).requires_grad_()
    o0, s0, l0 = plain_block(xx, residual.to(F64), ww, idx, k, mask, act, blk.eps, 0.5, 0.25)
    total = (o0 * dout.to(F64)).sum() + (s0 * ds.to(F64)).sum() + (l0 * dloss.to(F64)).sum()
    total.backward()
    got = {"out": out, "loss": loss, "dx": dx, **g}
    want = {"out": o0, "loss": l0, "dx": xx.grad, **{n: t.grad for n, t in ww.items()}}
    for name in want:
        r = want[name].detach()
        rms = r.pow(2).mean().sqrt().item()
        # the router's gradient is a difference of terms that nearly cancel for
        # one token's softmax; all others the layer's bar
        err = (got[name].to(F64) - r).abs().max().item() / rms
        assert err <= 2e-2 * max(1.0, (r.abs().max().item() / rms) / 4), (name, err)


def test_norm_in_mxfp8_feeds_the_mxfp8_product():
    """The norm's codes and scales are what gemm_mxfp8 takes: the product of
    their values, to fp32 accuracy of its sums."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(256, 512, generator=g, device="cuda").bfloat16()
    r = torch.randn(256, 512, generator=g, device="cuda").bfloat16()
    w = (torch.randn(128, 512, generator=g, device="cuda") / 22).bfloat16()
    values = torch.empty_like(x)
    _, codes, scales = api.add_rmsnorm_mx(x, torch.ones(512, device="cuda"), r, values=values)
    wc = torch.empty(128, 512, dtype=torch.uint8, device="cuda")
    ws = torch.empty(128, 16, dtype=torch.uint8, device="cuda")
    wv = api.mx_quantize(w, False, codes=wc, scales=ws)
    out = torch.empty(256, 128, device="cuda")
    api.gemm_mxfp8(codes, scales, wc, ws, out, torch.zeros(256, dtype=torch.uint8, device="cuda"))
    want = values.to(F64) @ wv.to(F64).T
    mag = values.to(F64).abs() @ wv.to(F64).abs().T
    assert ((out.to(F64) - want).abs() <= mag * 2 * 512 * ref.U32).all()
