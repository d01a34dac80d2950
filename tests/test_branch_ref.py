"""The references of the branch operators: the generator's published answers and
the norms' gradient against differences."""
import pytest
import torch

import _branch_ref as ref

F64 = torch.float64


@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))])
def test_generator_known_answers(ctr, key, want):
    """The known answers of Philox4x32-10 that its authors published."""
    assert tuple(ref.philox4x32_10(ctr, key)) == want


def test_words_are_the_generators():
    seed, step, site, first = 0x123456789abcdef0, 0x1_0000_0007, 3, 4 * ((1 << 33) + 5)
    got = ref.dropout_words(seed, step, site, first, 9).tolist()
    want = []
    for b in range(first // 4, first // 4 + 3):
        want += ref.philox4x32_10((b & ref.MASK, b >> 32, 7, site), (seed & ref.MASK, seed >> 32))
    assert got == want[:9]


@pytest.mark.parametrize("kind", ["none", "channel", "token"])
def test_post_pre_gradient_against_differences(kind):
    """d/dh of sum(y dy) + sum(s ds) along a random direction of every input."""
    g = torch.Generator().manual_seed(1)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, dtype=F64)

    rows, d, alpha, eps = 5, 12, 0.7, 1e-3
    gate = {"none": None, "channel": rnd(d), "token": rnd(rows, 1)}[kind]
    x, r, w1, w2, dy, ds = rnd(rows, d), rnd(rows, d), rnd(d), rnd(d), rnd(rows, d), rnd(rows, d)

    def loss(x, r, w1, w2, gate):
        s, _, norm = ref.post_pre(x, r, w1, w2, gate, alpha, eps, F64)
        return (norm(s)[0] * dy).sum() + (s * ds).sum(), s

    _, s = loss(x, r, w1, w2, gate)
    (dx, dr, dw1, dw2, *dg), _ = ref.post_pre_backward(dy, x, s, w1, w2, gate, ds, alpha, eps)
    args = [x, r, w1, w2] + ([gate] if gate is not None else [])
    grads = [dx, dr, dw1, dw2] + dg
    for i, (v, gv) in enumerate(zip(args, grads)):
        h, e = 1e-6, rnd(*v.shape)
        up, down = list(args), list(args)
        up[i], down[i] = v + h * e, v - h * e
        pad = [] if gate is not None else [None]
        diff = (loss(*up, *pad)[0] - loss(*down, *pad)[0]) / (2 * h)
        # a central difference: h^2 of a third derivative of some hundreds, and 1e-16 / h
        assert abs(diff - (gv * e).sum()) < 1e-7 * (1 + abs(diff))
