"""A MoE block for training: the residual addition with its RMS norm, the MoE
layer, a shared expert beside the routed ones, and the router's auxiliary losses;
forward and backward.

    s = x + residual                                            (pre-norm)
    s = residual_scale * residual + gate * RMSNorm(x) * post    (with post_norm)
    n = RMSNorm(s) * norm
    out = dropout(MoE(n) + act(n w_up^T + b_up) w_out^T + b_out)
    loss = router balance loss and z loss of the logits n w_router^T

The next block takes (out, s) as its (x, residual).

`GroupedExperts` are experts of another form than the layer's, of products grouped by
expert over the rows of a dispatch plan.
"""
from __future__ import annotations

import torch

from . import api


class MoEBlock:
    """Calls the operators in order and keeps what the backward needs.

    Weights are a dict: norm fp32 [d], w_router bf16 [E, d], w_gate_up bf16
    [E, 2I, d], w_down bf16 [E, d, I], w_up bf16 [F, d], b_up fp32 [F], w_out
    bf16 [d, F], b_out fp32 [d]; with post_norm also post fp32 [d] and, if there,
    gate fp32 [d].  Gradients come as a dict of the same names, fp32.

    dropout: the share of the output's elements that are dropped, by the
    generator state that `forward` is given and `site`, the block's number.
    residual_scale is the post_norm form's."""

    def __init__(self, T, d, E, I, k, *, act="silu", eps=1e-6, balance_coef=1e-2, z_coef=1e-3,
                 dtype=api.BF16, post_norm=False, residual_scale=1.0, dropout=0.0, site=0):
        if not post_norm and residual_scale != 1.0:
            raise ValueError("residual_scale needs post_norm")
        if not 0.0 <= dropout <= 1.0:
            raise ValueError(f"dropout must be from 0 to 1, got {dropout}")
        self.layer = api.MoELayer(T, d, E, I, k, dtype=dtype)
        self.T, self.k, self.act, self.eps = T, k, act, eps
        self.post_norm, self.residual_scale = post_norm, residual_scale
        self.dropout, self.site = dropout, site
        self.coefs = {"balance_coef": balance_coef, "z_coef": z_coef}
        self.kept = None

    def forward(self, x, residual, weights, mask=None, rng=None):
        """(out fp32 [T, d], s, loss fp32 [2], counts int32 [E]).  x bf16 or
        fp32 [T, d], residual the stream (s is of its type), mask uint8 [T]: the
        tokens that the auxiliary losses count.  rng: int64 [2] on the GPU, the seed
        and the step of the dropout, unchanged until the backward has run."""
        w = weights
        if self.dropout > 0 and rng is None:
            raise ValueError("dropout needs rng, the seed and the step on the GPU")
        if self.post_norm:
            s, n = api.post_pre_rmsnorm(x, residual, w["post"], w["norm"], w.get("gate"),
                                        residual_scale=self.residual_scale, eps=self.eps)
        else:
            s, n = api.add_rmsnorm(x, w["norm"], residual, eps=self.eps)
        routed = self.layer.forward(n, w["w_router"], None, w["w_gate_up"], w["w_down"])
        logits = api.linear(n, w["w_router"], out_dtype=torch.float32)
        idx = self.layer.saved_tensor("topk_idx", torch.int32, (self.T, self.k))
        loss, counts, _, lse, n_valid = api.router_balance(logits, idx, mask, **self.coefs)
        h, z = api.linear(n, w["w_up"], w["b_up"], act=self.act, keep_z=True)
        out = api.linear(h, w["w_out"], w["b_out"], residual=routed, out_dtype=routed.dtype)
        if self.dropout > 0:
            api.dropout(out, self.dropout, rng, self.site, y=out)
        self.kept = (x if self.post_norm else None, s, n, logits, lse, counts, n_valid, mask, h, z, rng)
        return out, s, loss, counts

    def backward(self, dout, ds, dloss, weights):
        """Gradients of the last forward from dout bf16 [T, d], ds (the
        gradient of s from the blocks above, of its type, or None) and dloss fp32
        [2]: (dx, gradients of the weights); dx is that of x and of the residual.
        With post_norm (dx bf16, dresidual, gradients of the weights)."""
        w, g = weights, {}
        x, s, n, logits, lse, counts, n_valid, mask, h, z, rng = self.kept
        if self.dropout > 0:
            dout = api.dropout_backward(dout, self.dropout, rng, self.site)
        dn, g["w_router"], g["w_gate_up"], g["w_down"] = self.layer.backward(
            dout, n, w["w_router"], None, w["w_gate_up"], w["w_down"])
        dh, g["w_out"], g["b_out"] = api.linear_backward(dout, h, w["w_out"], bias=True)
        _, g["w_up"], g["b_up"] = api.linear_backward(dh, n, w["w_up"], z, act=self.act, bias=True,
                                                      dx=dn, accumulate="dx")
        dlogits = api.router_balance_backward(dloss, logits, lse, counts, n_valid, self.k, mask,
                                              **self.coefs)
        api.linear_backward(dlogits, n, w["w_router"], dx=dn, dw=g["w_router"], accumulate=True)
        if self.post_norm:
            dx, dresidual, g["post"], g["norm"], dgate = api.post_pre_rmsnorm_backward(
                dn, x, s, w["post"], w["norm"], w.get("gate"), ds,
                residual_scale=self.residual_scale, eps=self.eps, dx_dtype=torch.bfloat16)
            if dgate is not None:
                g["gate"] = dgate
            return dx, dresidual, g
        dx, g["norm"] = api.add_rmsnorm_backward(dn, s, w["norm"], ds, eps=self.eps)
        return dx, g

    def status(self):
        """The layer's device status, else the operators' (0: no error)."""
        return self.layer.status() or api.device_status(api.operator_status())


class GroupedExperts:
    """Experts act(x w_up^T) w_down^T with relu^2 between the products, over the
    rows that a dispatch plan sorts by expert: w_up bf16 [E, F, d], w_down bf16 [E,
    d, F].  The plan (`api.dispatch_plan`): offsets int32 [E+1], token_of_row int32
    [T k], pos int32 [T, k]; topk_w fp32 [T, k] the slots' weights.

    A slot that the plan skipped for a bad index (pos -1; the plan's status tells) adds
    nothing and gets no gradient.  Such a plan has rows of no group, the last one among
    them: it stands for all skipped slots, as a row of zeros."""

    def __init__(self):
        self.kept = None

    @torch.no_grad()  # the products have no part in autograd's graph: nor has the rest
    def forward(self, x, topk_w, offsets, token_of_row, pos, w_up, w_down):
        """y fp32 [T, d] = the sum over a token's slots of topk_w times its
        expert's output.  x bf16 [T, d]."""
        # (words of rows of no group are unwritten)
        tokens = token_of_row.long().clamp(0, x.shape[0] - 1)
        rows = x[tokens]
        skipped = pos < 0
        slots = torch.where(skipped, rows.shape[0] - 1, pos).long()
        topk_w = topk_w.masked_fill(skipped, 0.0)
        z = api.grouped_linear(rows, w_up, offsets)
        h = torch.square(torch.relu(z.float())).to(torch.bfloat16)
        o = api.grouped_linear(h, w_down, offsets, out_dtype=torch.float32)
        o[-1:].masked_fill_(skipped.any(), 0.0)
        self.kept = (rows, z, h, o, topk_w, offsets, tokens, slots, skipped)
        # (weighted sums elementwise, here and in the backward, not by a library's product,
        # whose fp32 goes by torch's TF32 switch: 3e-4 off at 4096 x 8 x 4096)
        return o[slots].mul_(topk_w.unsqueeze(2)).sum(1)

    @torch.no_grad()
    def backward(self, dy, w_up, w_down):
        """(dx fp32 [T, d], dtopk_w fp32 [T, k], dw_up, dw_down fp32) of the last
        forward from dy fp32 [T, d]."""
        rows, z, h, o, topk_w, offsets, tokens, slots, skipped = self.kept
        row_w = topk_w.new_zeros(o.shape[0], 1)
        row_w[slots, 0] = topk_w
        dyr = dy[tokens]
        do = torch.mul(dyr, row_w, out=torch.empty_like(dyr, dtype=torch.bfloat16))
        dtopk_w = dyr.mul_(o).sum(1)[slots].masked_fill_(skipped, 0.0)
        dh, dw_down = api.grouped_linear_backward(do, h, w_down, offsets, dx_dtype=torch.float32)
        dz = (dh * 2 * torch.relu(z.float())).to(torch.bfloat16)
        dr, dw_up = api.grouped_linear_backward(dz, rows, w_up, offsets, dx_dtype=torch.float32)
        dr[-1:].masked_fill_(skipped.any(), 0.0)
        return dr[slots].sum(1), dtopk_w, dw_up, dw_down
