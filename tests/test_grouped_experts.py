"""`GroupedExperts` beside autograd, on the CPU with plain products in place of the
kernels: its results carry no part of a graph (one without the products' gradients
would give wrong ones), as those of the operators that it calls."""
import torch

from routing_dispatch_grouped_router_gb300 import api, block


def plain(x, w, offsets, transposed=False):
    ends = offsets.tolist()
    return torch.cat([x[a:b].float() @ (w[e].float() if transposed else w[e].float().T)
                      for e, (a, b) in enumerate(zip(ends, ends[1:]))])


def test_no_partial_graph(monkeypatch):
    def forward(x, w, offsets, *, out_dtype=None):
        with torch.no_grad():  # an operator's outputs are not autograd's
            return plain(x, w, offsets).to(out_dtype or torch.bfloat16)

    def backward(dy, x, w, offsets, *, dx_dtype=None):
        with torch.no_grad():
            return plain(dy, w, offsets, True).to(dx_dtype), torch.zeros(w.shape)

    monkeypatch.setattr(api, "grouped_linear", forward)
    monkeypatch.setattr(api, "grouped_linear_backward", backward)
    T, k, E, d, F = 3, 2, 2, 8, 16
    offsets = torch.tensor([0, 3, 6], dtype=torch.int32)
    rows = torch.tensor([0, 1, 2, 0, 1, 2], dtype=torch.int32)
    pos = torch.tensor([[0, 3], [1, 4], [2, 5]], dtype=torch.int32)
    x = torch.randn(T, d).bfloat16().requires_grad_()
    tw = torch.rand(T, k).requires_grad_()
    up = torch.randn(E, F, d).bfloat16().requires_grad_()
    down = torch.randn(E, d, F).bfloat16().requires_grad_()
    experts = block.GroupedExperts()
    y = experts.forward(x, tw, offsets, rows, pos, up, down)
    assert not y.requires_grad
    dy = torch.randn(T, d).requires_grad_()
    assert not any(t.requires_grad for t in experts.backward(dy, up, down))
