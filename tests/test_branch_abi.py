"""Dropout, the norms after and before a block and the products grouped by expert
without a GPU: size queries, argument checks of the C entry points before any device
call, and the Python module's refusals."""
import ctypes
import math

import pytest
import torch

from routing_dispatch_grouped_router_gb300 import _lib, api, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


P = ctypes.c_void_p
A = P(4096)  # a well aligned address that no check follows


def drop(**kw):
    d = dict(rows=4, d=64, ld_x=0, ld_res=0, ld_y=0, p=0.5, x_elem=0, y_elem=0, site=0, reserved=0)
    d.update(kw)
    return _lib.DropoutDesc(**d)


def norms(**kw):
    d = dict(rows=4, d=64, ld_x=0, ld_res=0, ld_s=0, ld_y=0, ld_dx=0, ld_dr=0, eps=1e-6,
             residual_scale=1.0, x_elem=0, s_elem=0, weight_elem=1, gate_elem=1, gate=0, y_elem=0,
             dx_elem=0, accumulate=0)
    d.update(kw)
    return _lib.PostPreDesc(**d)


def grouped(**kw):
    d = dict(rows=16, N=64, K=72, E=4, y_elem=0, dx_elem=0, accumulate=0, ld_x=0, ld_y=0, ld_dx=0)
    d.update(kw)
    return _lib.GroupedDesc(**d)


def test_sizes_of_the_descriptors():
    assert ctypes.sizeof(_lib.DropoutDesc) == 6 * 8 + 4 * 4
    assert ctypes.sizeof(_lib.PostPreDesc) == 8 * 8 + 10 * 4
    assert ctypes.sizeof(_lib.GroupedDesc) == 6 * 8 + 4 * 4


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(d=0), 1), (dict(rows=1 << 31), 2), (dict(d=1 << 31), 2),
    (dict(p=-0.1), 1), (dict(p=1.5), 1), (dict(p=math.nan), 1), (dict(x_elem=2), 2),
    (dict(y_elem=-1), 2), (dict(reserved=1), 2), (dict(ld_x=63), 1), (dict(ld_res=-1), 1),
    (dict(ld_y=8), 1)])
def test_dropout_descriptors_refused(lib, kw, code):
    assert lib.mok_dropout_forward(drop(**kw), A, A, A, A, None) == code
    assert lib.mok_dropout_backward(drop(**kw), A, A, A, None) == code


def test_dropout_pointers_refused(lib):
    f = lib.mok_dropout_forward
    assert f(None, A, None, A, A, None) == 1
    assert f(drop(), None, None, A, A, None) == 1
    assert f(drop(), A, None, None, A, None) == 1
    assert f(drop(), A, None, A, None, None) == 1
    assert f(drop(), P(4097), None, A, A, None) == 1
    assert f(drop(y_elem=1), A, P(4098), A, A, None) == 1
    assert f(drop(y_elem=1), A, None, A, P(4098), None) == 1
    assert f(drop(), A, None, P(4100), A, None) == 1
    assert lib.mok_dropout_backward(drop(), A, A, None, None) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(d=0), 1), (dict(d=16385), 2), (dict(rows=1 << 31), 2),
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(x_elem=2), 2), (dict(s_elem=2), 2),
    (dict(weight_elem=2), 2), (dict(gate_elem=2), 2), (dict(y_elem=2), 2), (dict(dx_elem=2), 2),
    (dict(gate=3), 2), (dict(gate=-1), 2), (dict(ld_x=63), 1), (dict(ld_dr=1), 1),
    (dict(ld_dx=-64), 1)])
def test_norms_descriptors_refused(lib, kw, code):
    n = ctypes.c_size_t()
    assert lib.mok_post_pre_rmsnorm_workspace_size(norms(**kw), n) == code
    assert lib.mok_post_pre_rmsnorm_forward(norms(**kw), A, A, A, A, None, A, A, None, None) == code


def test_norms_pointers_refused(lib):
    f = lib.mok_post_pre_rmsnorm_forward
    for missing in (0, 1, 2, 3, 5, 6):
        args = [A, A, A, A, None, A, A, None, None]
        args[missing] = None
        assert f(norms(), *args) == 1
    assert f(norms(gate=1), A, A, A, A, None, A, A, None, None) == 1  # no gate
    assert f(norms(), A, A, A, A, A, A, A, None, None) == 1           # one not asked for
    assert f(norms(), P(4097), A, A, A, None, A, A, None, None) == 1
    assert f(norms(), A, A, P(4098), A, None, A, A, None, None) == 1  # an fp32 weight at 2 bytes
    assert f(norms(), A, A, A, A, None, A, A, P(4098), None) == 1
    b = lib.mok_post_pre_rmsnorm_backward
    n = ctypes.c_size_t()
    assert lib.mok_post_pre_rmsnorm_workspace_size(norms(), n) == 0 and n.value >= 2 * 4 * 64
    ok = [A, A, A, A, A, None, A, A, A, A, A, None, A]
    for i in (0, 1, 2, 3, 4, 7, 8, 12):
        args = list(ok)
        args[i] = None
        assert b(norms(), *args, n.value, None, None) == 1
    assert b(norms(), *ok, n.value - 1, None, None) == 3
    args = list(ok)
    args[11] = A
    assert b(norms(), *args, n.value, None, None) == 1  # dgate without a gate


def test_norms_workspace_covers_any_alignment(lib):
    n = ctypes.c_size_t()
    for rows, d in ((1, 64), (5, 7168), (100000, 4096), (100000, 1), (100000, 16384)):
        assert lib.mok_post_pre_rmsnorm_workspace_size(norms(rows=rows, d=d), n) == 0
        assert n.value % (8 * d) == 0 and 1 <= n.value // (8 * d) <= min(rows, 152 * 16)
    assert lib.mok_post_pre_rmsnorm_workspace_size(norms(rows=0), n) == 0 and n.value == 0


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(N=0), 1), (dict(K=-8), 1), (dict(E=0), 1), (dict(E=513), 2),
    (dict(N=68), 2), (dict(K=76), 2), (dict(rows=(1 << 24) + 1), 2), (dict(N=(1 << 20) + 8), 2),
    (dict(y_elem=2), 2), (dict(dx_elem=2), 2), (dict(accumulate=1), 2), (dict(ld_x=64), 1),
    (dict(ld_x=76), 2), (dict(ld_y=68), 2), (dict(ld_dx=73), 2), (dict(ld_x=1 << 37), 2)])
def test_grouped_descriptors_refused(lib, kw, code):
    assert lib.mok_grouped_linear_forward(grouped(**kw), A, A, A, A, None, None) == code
    n = ctypes.c_size_t()
    assert lib.mok_grouped_linear_backward(grouped(**kw), A, A, A, A, A, A, None, 0, None,
                                           None) == code
    assert lib.mok_grouped_linear_workspace_size(grouped(**kw), n) == code


def test_grouped_pointers_refused(lib):
    f, b = lib.mok_grouped_linear_forward, lib.mok_grouped_linear_backward
    for i in range(4):
        args = [A] * 4
        args[i] = None
        assert f(grouped(), *args, None, None) == 1
        args[i] = P(4104)
        if i != 2:
            assert f(grouped(), *args, None, None) == 1  # at 8 bytes
    assert f(grouped(), A, A, P(4098), A, None, None) == 1
    for i in range(4):
        args = [A] * 6
        args[i] = None
        assert b(grouped(), *args, None, 0, None, None) == 1
    assert b(grouped(y_elem=1), *[A] * 6, None, 0, None, None) == 2  # fp32 dy
    assert b(grouped(), A, A, A, A, P(4104), A, None, 0, None, None) == 1
    assert b(grouped(), A, A, A, A, A, P(4104), None, 0, None, None) == 1
    n = ctypes.c_size_t()
    assert lib.mok_grouped_linear_workspace_size(grouped(), n) == 0 and n.value == 0
    long = grouped(rows=100000, E=1)
    assert lib.mok_grouped_linear_workspace_size(long, n) == 0 and n.value > 0
    assert b(long, *[A] * 6, None, n.value, None, None) == 1
    assert b(long, *[A] * 6, A, n.value - 1, None, None) == 3


def test_python_refusals_without_a_gpu(lib):
    """Tensors on the CPU, missing ones and wrong kinds raise ValueError."""
    x, w = torch.zeros(2, 8), torch.zeros(8)
    rng = torch.zeros(2, dtype=torch.int64)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: api.dropout(x, 0.5, rng), lambda: api.dropout(None, 0.5, rng),
                 lambda: api.dropout_backward(x, 0.5, rng), lambda: api.dropout(x, 0.5, 3),
                 lambda: api.post_pre_rmsnorm(x, x, w, w),
                 lambda: api.post_pre_rmsnorm(x, x, w, None),
                 lambda: api.post_pre_rmsnorm_backward(x, x, x, w, w),
                 lambda: api.post_pre_rmsnorm_backward(x, x, x, w, w, accumulate=w),
                 lambda: api.grouped_linear(x, torch.zeros(1, 8, 8), off),
                 lambda: api.grouped_linear(x, None, off),
                 lambda: api.grouped_linear_backward(x, x, torch.zeros(1, 8, 8), off)):
        with pytest.raises(ValueError):
            call()


def test_norms_without_rows_need_a_channels_gate(lib):
    """A channel's gate is [d] whatever the rows (the sums of the weights' gradients
    read it); only a token's, [0], may be missing."""
    f, b = lib.mok_post_pre_rmsnorm_forward, lib.mok_post_pre_rmsnorm_backward
    d = norms(rows=0, gate=1)
    assert f(d, None, None, A, A, None, None, None, None, None) == 1
    for grads in ((A, A, A), (A, None, None), (None, A, None), (None, None, A), (None,) * 3):
        assert b(d, None, None, None, A, A, None, None, None, None, *grads, None, 0, None,
                 None) == 1
    # those that are right end at the missing GPU, if at all
    if not torch.cuda.is_available():
        ok = f(norms(rows=0), None, None, A, A, None, None, None, None, None)
        assert ok != 1
        assert f(norms(rows=0, gate=2), None, None, A, A, None, None, None, None, None) == ok
        assert f(d, None, None, A, A, A, None, None, None, None) == ok
