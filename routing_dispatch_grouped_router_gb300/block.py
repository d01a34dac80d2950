"""A pre-norm MoE block for training: the residual addition with its RMS norm,
the MoE layer, a shared expert beside the routed ones, and the router's
auxiliary losses; forward and backward.

    s = x + residual
    n = RMSNorm(s) * norm
    out = MoE(n) + act(n w_up^T + b_up) w_out^T + b_out
    loss = router balance loss and z loss of the logits n w_router^T

The next block takes (out, s) as its (x, residual).
"""
from __future__ import annotations

import torch

from . import api


class MoEBlock:
    """Calls the operators in order and keeps what the backward needs.

    Weights are a dict: norm fp32 [d], w_router bf16 [E, d], w_gate_up bf16
    [E, 2I, d], w_down bf16 [E, d, I], w_up bf16 [F, d], b_up fp32 [F], w_out
    bf16 [d, F], b_out fp32 [d].  Gradients come as a dict of the same names,
    fp32."""

    def __init__(self, T, d, E, I, k, *, act="silu", eps=1e-6, balance_coef=1e-2, z_coef=1e-3,
                 dtype=api.BF16):
        self.layer = api.MoELayer(T, d, E, I, k, dtype=dtype)
        self.T, self.k, self.act, self.eps = T, k, act, eps
        self.coefs = {"balance_coef": balance_coef, "z_coef": z_coef}
        self.kept = None

    def forward(self, x, residual, weights, mask=None):
        """(out fp32 [T, d], s, loss fp32 [2], counts int32 [E]).  x bf16 or
        fp32 [T, d], residual the stream (s is of its type), mask uint8 [T]: the
        tokens that the auxiliary losses count."""
        w = weights
        s, n = api.add_rmsnorm(x, w["norm"], residual, eps=self.eps)
        routed = self.layer.forward(n, w["w_router"], None, w["w_gate_up"], w["w_down"])
        logits = api.linear(n, w["w_router"], out_dtype=torch.float32)
        idx = self.layer.saved_tensor("topk_idx", torch.int32, (self.T, self.k))
        loss, counts, _, lse, n_valid = api.router_balance(logits, idx, mask, **self.coefs)
        h, z = api.linear(n, w["w_up"], w["b_up"], act=self.act, keep_z=True)
        out = api.linear(h, w["w_out"], w["b_out"], residual=routed, out_dtype=routed.dtype)
        self.kept = (s, n, logits, lse, counts, n_valid, mask, h, z)
        return out, s, loss, counts

    def backward(self, dout, ds, dloss, weights):
        """Gradients of the last forward from dout bf16 [T, d], ds (the
        gradient of s from the blocks above, of its type, or None) and dloss fp32
        [2]: (dx, gradients of the weights); dx is that of x and of the residual."""
        w, g = weights, {}
        s, n, logits, lse, counts, n_valid, mask, h, z = self.kept
        dn, g["w_router"], g["w_gate_up"], g["w_down"] = self.layer.backward(
            dout, n, w["w_router"], None, w["w_gate_up"], w["w_down"])
        dh, g["w_out"], g["b_out"] = api.linear_backward(dout, h, w["w_out"], bias=True)
        _, g["w_up"], g["b_up"] = api.linear_backward(dh, n, w["w_up"], z, act=self.act, bias=True,
                                                      dx=dn, accumulate="dx")
        dlogits = api.router_balance_backward(dloss, logits, lse, counts, n_valid, self.k, mask,
                                              **self.coefs)
        api.linear_backward(dlogits, n, w["w_router"], dx=dn, dw=g["w_router"], accumulate=True)
        dx, g["norm"] = api.add_rmsnorm_backward(dn, s, w["norm"], ds, eps=self.eps)
        return dx, g

    def status(self):
        """The layer's device status, else the operators' (0: no error)."""
        return self.layer.status() or api.device_status(api.operator_status())
