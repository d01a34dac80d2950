"""The operators around the layer without a GPU: size queries, argument checks
of the C entry points before any device call, and the Python module's refusals."""
import ctypes

import pytest
import torch

from routing_dispatch_grouped_router_gb300 import _lib, api, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


P = ctypes.c_void_p
A = P(4096)  # a well aligned address that no check follows


def norm(**kw):
    d = dict(rows=4, d=64, ld_x=0, ld_res=0, ld_s=0, ld_y=0, eps=1e-6, x_elem=0, s_elem=0,
             weight_elem=1, accumulate=0, reserved=0)
    d.update(kw)
    return _lib.RmsnormDesc(**d)


def balance(**kw):
    d = dict(T=8, ld_logits=0, E=16, k=2, balance_coef=1.0, z_coef=1.0)
    d.update(kw)
    return _lib.BalanceDesc(**d)


def linear(**kw):
    d = dict(M=4, N=16, K=64, ld_x=0, act=0, y_elem=0, dx_elem=0, accumulate=0)
    d.update(kw)
    return _lib.LinearDesc(**d)


def test_sizes_of_the_descriptors():
    assert ctypes.sizeof(_lib.RmsnormDesc) == 6 * 8 + 6 * 4
    assert ctypes.sizeof(_lib.BalanceDesc) == 2 * 8 + 4 * 4
    assert ctypes.sizeof(_lib.LinearDesc) == 4 * 8 + 4 * 4


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(d=0), 1), (dict(d=16385), 2), (dict(rows=1 << 31), 2),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(x_elem=2), 2), (dict(s_elem=-1), 2),
    (dict(weight_elem=5), 2), (dict(reserved=1), 2), (dict(ld_x=63), 1), (dict(ld_y=-64), 1)])
def test_norm_descriptors_refused(lib, kw, code):
    n = ctypes.c_size_t()
    assert lib.mok_add_rmsnorm_workspace_size(norm(**kw), n) == code
    assert lib.mok_add_rmsnorm_forward(norm(**kw), A, None, A, None, A, None, None, None, None) == code


def test_norm_pointers_refused(lib):
    f = lib.mok_add_rmsnorm_forward
    assert f(norm(), None, None, A, None, A, None, None, None, None) == 1  # no x
    assert f(norm(), A, None, None, None, A, None, None, None, None) == 1  # no weight
    assert f(norm(), A, A, A, None, A, None, None, None, None) == 1        # a sum without s
    assert f(norm(), A, None, A, None, None, None, None, None, None) == 1  # no output
    assert f(norm(), A, None, A, None, A, None, A, None, None) == 1        # codes without scales
    assert f(norm(s_elem=1), A, None, A, None, A, None, None, None, None) == 2
    assert f(norm(d=40), A, None, A, None, None, A, None, None, None) == 2  # MX: d % 32
    assert f(norm(), P(4097), None, A, None, A, None, None, None, None) == 1
    b = lib.mok_add_rmsnorm_backward
    assert b(norm(), A, A, A, None, A, A, None, 0, None, None) == 1        # no workspace
    assert b(norm(), A, A, A, None, A, A, A, 16, None, None) == 3
    assert b(norm(), A, A, A, None, None, None, None, 0, None, None) == 1  # no dx


def test_norm_workspace_covers_any_alignment(lib):
    n = ctypes.c_size_t()
    for rows, d in ((1, 64), (5, 7168), (100000, 4096), (100000, 1), (100000, 16384)):
        assert lib.mok_add_rmsnorm_workspace_size(norm(rows=rows, d=d), n) == 0
        assert n.value % (4 * d) == 0 and 1 <= n.value // (4 * d) <= min(rows, 152 * 16)
    assert lib.mok_add_rmsnorm_workspace_size(norm(rows=0), n) == 0 and n.value == 0


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(E=513), 2), (dict(k=9), 2),
    (dict(E=1, k=2), 2), (dict(T=1 << 30), 2), (dict(ld_logits=15), 1)])
def test_balance_descriptors_refused(lib, kw, code):
    n = ctypes.c_size_t()
    assert lib.mok_router_balance_workspace_size(balance(**kw), n) == code


def test_balance_pointers_refused(lib):
    n = ctypes.c_size_t()
    assert lib.mok_router_balance_workspace_size(balance(), n) == 0
    f = lib.mok_router_balance_forward
    assert f(balance(), None, A, None, A, A, A, A, A, A, 1 << 20, None, None) == 1
    many = balance(T=1 << 16)
    assert lib.mok_router_balance_workspace_size(many, n) == 0 and n.value > 0
    assert f(many, A, A, None, A, A, A, A, A, None, 1 << 20, None, None) == 1
    assert f(many, A, A, None, A, A, A, A, A, A, n.value - 1, None, None) == 3
    assert f(balance(), P(4098), A, None, A, A, A, A, A, A, 1 << 20, None, None) == 1
    b = lib.mok_router_balance_backward
    assert b(balance(), None, A, A, A, A, None, A, None) == 1
    assert b(balance(), A, A, A, A, A, None, None, None) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(K=12), 2), (dict(M=(1 << 24) + 1), 2),
    (dict(act=4), 2), (dict(y_elem=2), 2), (dict(dx_elem=-1), 2), (dict(ld_x=63), 1),
    (dict(ld_x=68), 2), (dict(accumulate=4), 2)])
def test_linear_descriptors_refused(lib, kw, code):
    n = ctypes.c_size_t()
    assert lib.mok_linear_workspace_size(linear(**kw), 0, n) == code
    assert lib.mok_linear_workspace_size(linear(**kw), 1, n) == code


def test_linear_pointers_refused(lib):
    f = lib.mok_linear_forward
    assert f(linear(), None, A, None, None, A, None, None, 0, None, None) == 1
    assert f(linear(), A, None, None, None, A, None, None, 0, None, None) == 1
    assert f(linear(), A, A, None, None, None, None, None, 0, None, None) == 1
    assert f(linear(), P(4104), A, None, None, A, None, None, 0, None, None) == 1  # x at 8 bytes
    n = ctypes.c_size_t()
    d = linear(M=256, N=256, K=4096)
    assert lib.mok_linear_workspace_size(d, 0, n) == 0 and n.value > 0
    assert f(d, A, A, None, None, A, None, None, 0, None, None) == 1
    assert f(d, A, A, None, None, A, None, A, n.value - 1, None, None) == 3
    b = lib.mok_linear_backward
    assert b(linear(), None, A, A, None, A, A, A, A, 1 << 30, None, None) == 1
    assert b(linear(act=2), A, A, A, None, A, A, A, A, 1 << 30, None, None) == 1   # no z
    assert b(linear(accumulate=1), A, A, A, None, A, A, A, A, 1 << 30, None, None) == 2  # bf16 dx
    d = linear(M=40)
    assert b(d, A, A, A, None, A, A, A, None, 1 << 30, None, None) == 1
    assert b(d, A, A, A, None, A, A, A, A, 16, None, None) == 3


def test_python_refusals_without_a_gpu(lib):
    """Tensors on the CPU, missing ones and wrong kinds raise ValueError."""
    x, w = torch.zeros(2, 8), torch.zeros(8)
    for call in (lambda: api.add_rmsnorm(x, w), lambda: api.add_rmsnorm(None, w),
                 lambda: api.add_rmsnorm(3, w), lambda: api.add_rmsnorm_mx(x, w),
                 lambda: api.add_rmsnorm_backward(x, x, w),
                 lambda: api.router_balance(x, x, balance_coef=1.0),
                 lambda: api.linear(x, x), lambda: api.linear(x, x, act="tanh"),
                 lambda: api.linear_backward(x, x, x),
                 lambda: api.linear_backward(x, x, x, accumulate="db")):
        with pytest.raises(ValueError):
            call()
