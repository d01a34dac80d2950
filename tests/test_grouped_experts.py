"""`GroupedExperts` beside autograd, on the CPU with plain products in place of the
kernels: its results carry no part of a graph (one without the products' gradients
would give wrong ones), as those of the operators that it calls."""
import math

import pytest
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


def plan_with_skipped(T, idx, E):
    """The plan of idx [T, k] as the dispatch plan has it: an index outside of the experts
    leaves -1 in pos, and the words behind the last group unwritten (here: any value)."""
    k = len(idx[0])
    slots = [[(t, s) for t in range(T) for s in range(k) if idx[t][s] == e] for e in range(E)]
    offsets = [0]
    for group in slots:
        offsets.append(offsets[-1] + len(group))
    pos = torch.full((T, k), -1, dtype=torch.int32)
    rows = torch.tensor([(1 << 30) - 1, -7] * (T * k))[:T * k].int()
    for r, (t, s) in enumerate(slot for group in slots for slot in group):
        pos[t, s] = r
        rows[r] = t
    return torch.tensor(offsets, dtype=torch.int32), rows, pos


@pytest.mark.parametrize("idx", [[[1, 9], [0, 1], [1, 0], [1, 1]], [[-1, 5], [1, 0], [2, -9], [0, 2]],
                                 [[3, 3], [-1, -1], [4, 7], [99, 3]], [[0, 1], [1, 0], [2, 1], [0, 2]]])
def test_skipped_slots(monkeypatch, idx):
    """A slot that the plan skipped adds nothing, whatever the rows of no group hold, and
    gets no gradient."""
    T, k, E, d, F = 4, 2, 3, 8, 16

    def rows_of(t, like):  # as the operator leaves them: rows of no group unwritten
        return torch.cat([t, torch.full((like.shape[0] - t.shape[0], t.shape[1]), math.nan)])

    def forward(x, w, offsets, *, out_dtype=None):
        return rows_of(plain(x, w, offsets), x).to(out_dtype or torch.bfloat16)

    def backward(dy, x, w, offsets, *, dx_dtype=None):
        ends = offsets.tolist()
        dw = torch.stack([dy[a:b].float().T @ x[a:b].float() for a, b in zip(ends, ends[1:])])
        return rows_of(plain(dy, w, offsets, True), dy).to(dx_dtype), dw

    monkeypatch.setattr(api, "grouped_linear", forward)
    monkeypatch.setattr(api, "grouped_linear_backward", backward)
    g = torch.Generator().manual_seed(3)
    # (small whole numbers: every product and sum is exact)
    x, dy = (torch.randint(-2, 3, (T, d), generator=g).float() for _ in range(2))
    up = torch.randint(-1, 2, (E, F, d), generator=g).float()
    down = torch.randint(-1, 2, (E, d, F), generator=g).float()
    tw = torch.randint(1, 4, (T, k), generator=g).float() / 4
    bad = tw.clone()
    for t in range(T):
        for s in range(k):
            if not 0 <= idx[t][s] < E:
                bad[t, s] = math.nan  # (nor does its weight matter)
    experts = block.GroupedExperts()
    y = experts.forward(x.bfloat16(), bad, *plan_with_skipped(T, idx, E), up.bfloat16(),
                        down.bfloat16())
    got = (y,) + experts.backward(dy, up.bfloat16(), down.bfloat16())
    leaves = [t.double().requires_grad_() for t in (x, tw, up, down)]
    xx, ww, uu, dd = leaves
    want = xx * 0
    for t in range(T):
        for s in range(k):
            if 0 <= idx[t][s] < E:
                h = torch.relu(uu[idx[t][s]] @ xx[t]) ** 2
                want = want + torch.nn.functional.one_hot(torch.tensor(t), T).double()[:, None] \
                    * (ww[t, s] * (dd[idx[t][s]] @ h))
    (want * dy.double()).sum().backward()
    zero = [torch.zeros_like(t) if t.grad is None else t.grad for t in leaves]
    for a, b in zip(got, [want] + zero):
        assert torch.equal(a.double(), b.detach())
