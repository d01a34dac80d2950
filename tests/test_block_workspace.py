"""Scratch of the dense product's backward, by the size query alone (no GPU)."""
import ctypes

import pytest

from routing_dispatch_grouped_router_gb300 import _lib, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("M,N,K", [(8192, 7168, 2048), (4096, 1024, 2048), (300, 130, 512)])
def test_backward_keeps_the_parts_of_dz_that_it_uses(lib, M, N, K):
    """None of a bf16 dy that is dz itself, one of an unaligned one, three where
    the products take three."""
    def size(backward, **kw):
        n = ctypes.c_size_t()
        assert lib.mok_linear_workspace_size(_lib.LinearDesc(M=M, N=N, K=K, **kw), backward, n) == 0
        return n.value

    part = M * ((N + 63) // 64 * 64) * 2
    part = (part + 255) // 256 * 256
    plain, aligned = size(1), size(2)
    assert plain - aligned == (part if N % 8 == 0 else 0)
    for kw in (dict(act=2), dict(y_elem=1)):
        assert size(1, **kw) == size(2, **kw) >= 3 * part
    # beside the parts: column sums by 32 rows and partial products, which take a
    # split of K only where tiles are few
    if M * N >= 1 << 24:
        assert aligned < part / 8
