"""PyTorch-facing wrappers of the C ABI in include/mok.h.

Tensors only provide device memory and the current stream; every step runs in
libmok.so.  Shapes and dtypes are checked here, everything else by the library.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib

BF16, MXFP8, NVFP4 = 0, 1, 2
FLAG_BF16_ACT_OUT = 0x1    # y and dx written as bf16 (default fp32)
FLAG_BF16_WGRAD_OUT = 0x2  # weight gradients written as bf16 (default fp32)
FLAG_ACCUMULATE_WGRAD = 0x4  # backward adds into the fp32 weight gradients
FLAG_RECOMPUTE_GATE_UP = 0x8  # g, u not kept by the forward; the backward recomputes them
FLAG_SINGLE_CTA_GEMM = 0x10  # one-CTA 128-row GEMM tiles instead of CTA pairs
FLAG_RECOMPUTE_DISPATCH = 0x20  # dispatched x rows not kept; the backward gathers them again
NOT_KEPT = (1 << 64) - 1  # saved-layout offset of a field the flags leave out


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_desc(T, d, E, I, k, dtype=BF16, flags=0, mb_tokens=0, ring_slots=0) -> _lib.MoeDesc:
    return _lib.MoeDesc(T=T, d=d, E=E, I=I, k=k, dtype=dtype, mb_tokens=mb_tokens,
                        ring_slots=ring_slots, flags=flags, reserved=0)


def workspace_sizes(desc):
    """(forward scratch, saved, backward scratch) bytes."""
    lib = _lib.load()
    f, s, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _lib.check(lib.mok_moe_workspace_size(ctypes.byref(desc), ctypes.byref(f), ctypes.byref(s),
                                          ctypes.byref(b)), "mok_moe_workspace_size")
    return f.value, s.value, b.value


def saved_layout(desc) -> _lib.SavedLayout:
    lib = _lib.load()
    L = _lib.SavedLayout()
    _lib.check(lib.mok_moe_saved_layout(ctypes.byref(desc), ctypes.byref(L)), "mok_moe_saved_layout")
    return L


def stage_workspace_size(desc) -> int:
    lib = _lib.load()
    n = ctypes.c_size_t()
    _lib.check(lib.mok_moe_stage_workspace_size(ctypes.byref(desc), ctypes.byref(n)),
               "mok_moe_stage_workspace_size")
    return n.value


def forward(desc, x, w_router, bias, w_gate_up, w_down, y, saved, workspace, stream=None):
    lib = _lib.load()
    _lib.check(lib.mok_moe_forward(ctypes.byref(desc), _ptr(x), _ptr(w_router), _ptr(bias),
                                   _ptr(w_gate_up), _ptr(w_down), _ptr(y), _ptr(saved),
                                   saved.numel(), _ptr(workspace), workspace.numel(),
                                   _stream(stream)), "mok_moe_forward")


def backward(desc, dy, x, w_router, bias, w_gate_up, w_down, saved, dx, dw_router, dw_gate_up,
             dw_down, workspace, stream=None):
    lib = _lib.load()
    _lib.check(lib.mok_moe_backward(ctypes.byref(desc), _ptr(dy), _ptr(x), _ptr(w_router),
                                    _ptr(bias), _ptr(w_gate_up), _ptr(w_down), _ptr(saved),
                                    saved.numel(), _ptr(dx), _ptr(dw_router), _ptr(dw_gate_up),
                                    _ptr(dw_down), _ptr(workspace), workspace.numel(),
                                    _stream(stream)), "mok_moe_backward")


def route(desc, x, w_router, bias, topk_idx, topk_w, workspace, stream=None):
    lib = _lib.load()
    _lib.check(lib.mok_moe_route(ctypes.byref(desc), _ptr(x), _ptr(w_router), _ptr(bias),
                                 _ptr(topk_idx), _ptr(topk_w), _ptr(workspace), workspace.numel(),
                                 _stream(stream)), "mok_moe_route")


def dispatch_plan(desc, topk_idx, counts, offsets, pos, token_of_row, workspace, stream=None):
    lib = _lib.load()
    _lib.check(lib.mok_moe_dispatch_plan(ctypes.byref(desc), _ptr(topk_idx), _ptr(counts),
                                         _ptr(offsets), _ptr(pos), _ptr(token_of_row),
                                         _ptr(workspace), workspace.numel(), _stream(stream)),
               "mok_moe_dispatch_plan")


def gemm_bf16(A, a_mn_major, B, b_mn_major, C, workspace, stream=None):
    """C = A @ B with A given as [M,K] (a_mn_major=False) or [K,M] (True) and
    B as [N,K] (b_mn_major=False) or [K,N] (True)."""
    lib = _lib.load()
    M, N = C.shape
    K = A.shape[0] if a_mn_major else A.shape[1]
    _lib.check(lib.mok_gemm_bf16(M, N, K, _ptr(A), int(a_mn_major), _ptr(B), int(b_mn_major),
                                 _ptr(C), _ptr(workspace), workspace.numel(), _stream(stream)),
               "mok_gemm_bf16")


def gemm_mxfp8(A, sa, B, sb, C, workspace, cta_pair=False, stream=None):
    """C[M,N] fp32 = dequant(A) dequant(B)^T for E4M3 codes A [M,K], B [N,K]
    and E8M0 scale bytes sa [M,K/32], sb [N,K/32] (see mok_gemm_mxfp8)."""
    lib = _lib.load()
    M, N = C.shape
    K = A.shape[1]
    _lib.check(lib.mok_gemm_mxfp8(M, N, K, _ptr(A), _ptr(sa), _ptr(B), _ptr(sb), _ptr(C),
                                  int(cta_pair), _ptr(workspace), workspace.numel(),
                                  _stream(stream)),
               "mok_gemm_mxfp8")


def mx_quantize(x, along_rows: bool, out=None, codes=None, scales=None, stream=None):
    """MXFP8 fake quantisation of a 2-D bf16 tensor (see mok_mx_quantize)."""
    lib = _lib.load()
    out = torch.empty_like(x) if out is None else out
    rows, cols = x.shape
    _lib.check(lib.mok_mx_quantize(_ptr(x), rows, cols, int(along_rows), _ptr(out), _ptr(codes),
                                   _ptr(scales), _stream(stream)), "mok_mx_quantize")
    return out


def nvfp4_tensor_scale(x, g=None, stream=None):
    """NVFP4 tensor scale of a bf16 tensor into the device fp32 `g` (see
    mok_nvfp4_tensor_scale)."""
    g = torch.empty(1, dtype=torch.float32, device=x.device) if g is None else g
    _lib.check(_lib.load().mok_nvfp4_tensor_scale(_ptr(x), x.numel(), _ptr(g), _stream(stream)),
               "mok_nvfp4_tensor_scale")
    return g


def nvfp4_quantize(x, g, codes=None, scales=None, stream=None):
    """NVFP4 codes [rows, cols/2] and E4M3 block scales [rows, cols/16] of a
    2-D bf16 tensor with tensor scale g (see mok_nvfp4_quantize)."""
    rows, cols = x.shape
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=x.device) if codes is None \
        else codes
    scales = torch.empty(rows, cols // 16, dtype=torch.uint8, device=x.device) if scales is None \
        else scales
    _lib.check(_lib.load().mok_nvfp4_quantize(_ptr(x), rows, cols, _ptr(g), _ptr(codes),
                                              _ptr(scales), _stream(stream)),
               "mok_nvfp4_quantize")
    return codes, scales


def nvfp4_quantize_cols(x, g, codes=None, scales=None, stream=None):
    """NVFP4 of the columns of a bf16 [ng, K, C] (or [K, C]) tensor, blocks of
    16 along K: codes [ng*C, K/2] and E4M3 scales [ng*C, K/16] (see
    mok_nvfp4_quantize_cols)."""
    x3 = x if x.dim() == 3 else x.unsqueeze(0)
    ng, K, C = x3.shape
    codes = torch.empty(ng * C, K // 2, dtype=torch.uint8, device=x.device) if codes is None \
        else codes
    scales = torch.empty(ng * C, K // 16, dtype=torch.uint8, device=x.device) if scales is None \
        else scales
    _lib.check(_lib.load().mok_nvfp4_quantize_cols(_ptr(x3), ng, K, C, _ptr(g), _ptr(codes),
                                                   _ptr(scales), _stream(stream)),
               "mok_nvfp4_quantize_cols")
    return codes, scales


def gemm_nvfp4(A, sa, ga, B, sb, gb, C, workspace, stream=None):
    """C[M,N] fp32 = ga gb dequant(A) dequant(B)^T for NVFP4 codes A [M,K/2],
    B [N,K/2], E4M3 block scales sa [M,K/16], sb [N,K/16] and device tensor
    scales ga, gb (see mok_gemm_nvfp4)."""
    M, N = C.shape
    K = 2 * A.shape[1]
    _lib.check(_lib.load().mok_gemm_nvfp4(M, N, K, _ptr(A), _ptr(sa), _ptr(ga), _ptr(B),
                                          _ptr(sb), _ptr(gb), _ptr(C), _ptr(workspace),
                                          workspace.numel(), _stream(stream)), "mok_gemm_nvfp4")


# -------------------------------------------- operators around the layer --
# One decode step makes several of these calls, so their host time counts: the
# checks of shapes, types, strides and devices run once for each combination of
# them and leave the C descriptor (nothing else is kept).

_ELEM = {torch.bfloat16: 0, torch.float32: 1}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
_BF, _F32, _I32, _U8 = (torch.bfloat16,), (torch.float32,), (torch.int32,), (torch.uint8,)
_MASK = (torch.uint8, torch.bool)
_plan = functools.lru_cache(maxsize=8192)
_status_words = {}


def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _addr(t):
    return None if t is None else t.data_ptr()


def _call_stream(t, stream):
    """The raw stream of a call on the GPU of `t`, which must be the current one."""
    index = t.get_device()
    if index < 0 or index != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors must be on the current GPU, not on {t.device}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream


def _alloc(shape, dtype, device, stream):
    """A tensor of the stream that the call runs on, so that its memory is not
    handed out again before that stream is done with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def operator_status(device=None):
    """The device int32 that the operators below report into (sticky: the
    first error stays; read it with `device_status`, zero it to go on)."""
    index = torch.cuda.current_device() if device is None else torch.device(device).index
    word = _status_words.get(index)
    if word is None:
        word = torch.zeros(64, dtype=torch.int32, device=torch.device("cuda", index))
        torch.cuda.synchronize(index)  # zero before a first call on any other stream
        _status_words[index] = word
    return word


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _matrix(m, name, shape=None, dtypes=_ELEM, device=None):
    """Checks the metadata of a matrix with consecutive columns; returns its row stride."""
    sh, st, dt, dev = m
    _need(len(sh) == 2, f"{name} must be a matrix, got {tuple(sh)}")
    _need(shape is None or sh == shape, f"{name} must be {shape}, got {tuple(sh)}")
    _need(dt in dtypes, f"{name} must not be {dt}")
    _need(dev.type == "cuda" and (device is None or dev == device),
          f"{name} must be on the GPU of the other tensors, not on {dev}")
    _need(sh[1] <= 1 or st[1] == 1, f"{name} must have consecutive columns")
    if sh[0] <= 1:
        return sh[1]
    _need(st[0] >= sh[1], f"{name} must have rows that do not overlap")
    return st[0]


def _dense(m, name, shape, dtypes, device):
    """Checks the metadata of a contiguous tensor of a given shape."""
    sh, st, dt, dev = m
    _need(sh == shape, f"{name} must be {shape}, got {tuple(sh)}")
    _need(dt in dtypes, f"{name} must not be {dt}")
    _need(dev == device, f"{name} must be on the GPU of the other tensors, not on {dev}")
    n = 1
    for size, step in zip(reversed(sh), reversed(st)):
        _need(size <= 1 or step == n, f"{name} must be contiguous")
        n *= size


@_plan
def _norm_plan(x, weight, res, s, y, eps, mx):
    ld_x = _matrix(x, "x")
    (rows, d), dev = x[0], x[3]
    _dense(weight, "weight", (d,), _ELEM, dev)
    ld_r = 0 if res is None else _matrix(res, "residual", (rows, d), device=dev)
    stream_dt = x[2] if res is None else res[2]
    ld_s = 0 if s is None else _matrix(s, "s", (rows, d), (stream_dt,), dev)
    ld_y = 0 if y is None else _matrix(y, "y", (rows, d), _BF, dev)
    _need(not mx or d % 32 == 0, "MXFP8 needs d a multiple of 32")
    return _lib.RmsnormDesc(rows, d, ld_x, ld_r, ld_s, ld_y, eps, _ELEM[x[2]], _ELEM[stream_dt],
                            _ELEM[weight[2]], 0, 0)


@_plan
def _mx_out_plan(x, codes, scales, values):
    (rows, d), dev = x[0], x[3]
    _dense(codes, "codes", (rows, d), _U8, dev)
    _dense(scales, "scales", (rows, d // 32), _U8, dev)
    if values is not None:
        _dense(values, "values", (rows, d), _BF, dev)


def add_rmsnorm(x, weight, residual=None, eps=1e-6, *, s=None, y=None, stream=None):
    """s = x + residual and y = RMSNorm(s) * weight (see
    mok_add_rmsnorm_forward): (s, y), s in the residual's type (x itself
    without a residual), y bf16.  x, residual bf16 or fp32 matrices, weight
    bf16 or fp32; rows may be strided."""
    st = _call_stream(x, stream)
    if residual is not None and s is None:
        s = _alloc(x.shape, residual.dtype, x.device, stream)
    if y is None:
        y = _alloc(x.shape, torch.bfloat16, x.device, stream)
    desc = _norm_plan(_meta(x), _meta(weight), _meta(residual), _meta(s), _meta(y), eps, False)
    _lib.check(_lib.load().mok_add_rmsnorm_forward(desc, _addr(x), _addr(residual), _addr(weight),
                                                   _addr(s), _addr(y), None, None, None, st),
               "mok_add_rmsnorm_forward")
    return (x if s is None else s), y


def add_rmsnorm_mx(x, weight, residual=None, eps=1e-6, *, s=None, y=None, values=None, codes=None,
                   scales=None, stream=None):
    """`add_rmsnorm` with the norm in MXFP8: (s, codes, scales), codes uint8
    [rows, d] (E4M3), scales uint8 [rows, d/32] (E8M0), as `gemm_mxfp8` takes
    them.  y (the bf16 norm) and values (the bf16 values of the codes) are
    written if given.  d a multiple of 32."""
    st = _call_stream(x, stream)
    if residual is not None and s is None:
        s = _alloc(x.shape, residual.dtype, x.device, stream)
    desc = _norm_plan(_meta(x), _meta(weight), _meta(residual), _meta(s), _meta(y), eps, True)
    rows, d = x.shape
    if codes is None:
        codes = _alloc((rows, d), torch.uint8, x.device, stream)
    if scales is None:
        scales = _alloc((rows, d // 32), torch.uint8, x.device, stream)
    _mx_out_plan(_meta(x), _meta(codes), _meta(scales), _meta(values))
    _lib.check(_lib.load().mok_add_rmsnorm_forward(desc, _addr(x), _addr(residual), _addr(weight),
                                                   _addr(s), _addr(y), _addr(values), _addr(codes),
                                                   _addr(scales), st), "mok_add_rmsnorm_forward")
    return (x if s is None else s), codes, scales


@_plan
def _norm_bwd_plan(dy, s, weight, ds, dx, dweight, eps, accumulate):
    ld_dy = _matrix(dy, "dy")
    (rows, d), dev = dy[0], dy[3]
    ld_s = _matrix(s, "s", (rows, d), device=dev)
    _dense(weight, "weight", (d,), _ELEM, dev)
    ld_ds = 0 if ds is None else _matrix(ds, "ds", (rows, d), (s[2],), dev)
    ld_dx = _matrix(dx, "dx", (rows, d), (s[2],), dev)
    _dense(dweight, "dweight", (d,), _F32, dev)
    desc = _lib.RmsnormDesc(rows, d, ld_dy, ld_ds, ld_s, ld_dx, eps, _ELEM[dy[2]], _ELEM[s[2]],
                            _ELEM[weight[2]], int(accumulate), 0)
    n = ctypes.c_size_t()
    _lib.check(_lib.load().mok_add_rmsnorm_workspace_size(desc, n),
               "mok_add_rmsnorm_workspace_size")
    return desc, n.value


def add_rmsnorm_backward(dy, s, weight, ds=None, eps=1e-6, *, dx=None, dweight=None,
                         accumulate=False, workspace=None, stream=None):
    """Gradients of `add_rmsnorm` from dy and the stored s (see
    mok_add_rmsnorm_backward): (dx, dweight).  dx, in the type of s, is the
    gradient of x and of residual alike, with ds (the gradient that reaches s by
    other ways) added; dweight fp32, added into with `accumulate`."""
    st = _call_stream(dy, stream)
    _need(dweight is not None or not accumulate, "accumulate needs dweight")
    if dx is None:
        dx = _alloc(dy.shape, s.dtype, dy.device, stream)
    if dweight is None:
        dweight = _alloc(dy.shape[1:], torch.float32, dy.device, stream)
    desc, n = _norm_bwd_plan(_meta(dy), _meta(s), _meta(weight), _meta(ds), _meta(dx),
                             _meta(dweight), eps, accumulate)
    if workspace is None:
        workspace = _alloc((n,), torch.uint8, dy.device, stream)
    _lib.check(_lib.load().mok_add_rmsnorm_backward(desc, _addr(dy), _addr(s), _addr(weight),
                                                    _addr(ds), _addr(dx), _addr(dweight),
                                                    _addr(workspace), workspace.nbytes,
                                                    _addr(operator_status(dy.device)), st),
               "mok_add_rmsnorm_backward")
    return dx, dweight


@_plan
def _balance_plan(logits, k, mask, lse, balance_coef, z_coef):
    ld = _matrix(logits, "logits", None, _F32)
    (T, E), dev = logits[0], logits[3]
    if mask is not None:
        _dense(mask, "mask", (T,), _MASK, dev)
    if lse is not None:
        _dense(lse, "lse", (T,), _F32, dev)
    desc = _lib.BalanceDesc(T, ld, E, k, balance_coef, z_coef)
    n = ctypes.c_size_t()
    _lib.check(_lib.load().mok_router_balance_workspace_size(desc, n),
               "mok_router_balance_workspace_size")
    return desc, n.value


@_plan
def _topk_plan(idx, T, dev):
    _need(len(idx[0]) == 2, "topk_idx must be a matrix")
    _dense(idx, "topk_idx", (T, idx[0][1]), _I32, dev)


def router_balance(logits, topk_idx, mask=None, *, balance_coef, z_coef=0.0, workspace=None,
                   stream=None):
    """The router's auxiliary losses over the tokens of `mask` (see
    mok_router_balance_forward): (loss [2] = balance and z loss, counts int32
    [E], prob [E] = mean probability, lse [T], n_valid int32 [1]).  logits fp32
    [T, E], topk_idx int32 [T, k], mask uint8 or bool [T].  The results share
    two allocations."""
    st = _call_stream(logits, stream)
    dev = logits.device
    _topk_plan(_meta(topk_idx), logits.shape[0], dev)
    desc, n = _balance_plan(_meta(logits), topk_idx.shape[1], _meta(mask), None, balance_coef,
                            z_coef)
    # the fp32 results (and the scratch) in one allocation, the integers in another
    T, E = desc.T, desc.E
    at_lse = (E + 2 + 3) // 4 * 4
    at_ws = (at_lse + T + 3) // 4 * 4
    buf = _alloc((at_ws + (n + 3) // 4 if workspace is None else at_ws,), torch.float32, dev, stream)
    ints = _alloc((E + 1,), torch.int32, dev, stream)
    prob = buf.as_strided((E,), (1,), 0)
    loss = buf.as_strided((2,), (1,), E)
    lse = buf.as_strided((T,), (1,), at_lse)
    counts = ints.as_strided((E,), (1,), 0)
    n_valid = ints.as_strided((1,), (1,), E)
    f, i = buf.data_ptr(), ints.data_ptr()
    ws = f + 4 * at_ws if workspace is None else workspace.data_ptr()
    _lib.check(_lib.load().mok_router_balance_forward(
        desc, _addr(logits), _addr(topk_idx), _addr(mask), f + 4 * E, i, f, f + 4 * at_lse,
        i + 4 * E, ws, n if workspace is None else workspace.nbytes, _addr(operator_status(dev)),
        st), "mok_router_balance_forward")
    return loss, counts, prob, lse, n_valid


@_plan
def _balance_bwd_plan(dloss, logits, counts, n_valid, dlogits):
    dev = logits[3]
    _dense(dloss, "dloss", (2,), _F32, dev)
    _dense(counts, "counts", (logits[0][1],), _I32, dev)
    _dense(n_valid, "n_valid", (1,), _I32, dev)
    _need(_matrix(dlogits, "dlogits", logits[0], _F32, dev) ==
          _matrix(logits, "logits", None, _F32), "dlogits must have the row stride of logits")


def router_balance_backward(dloss, logits, lse, counts, n_valid, k, mask=None, *, balance_coef,
                            z_coef=0.0, dlogits=None, stream=None):
    """dlogits [T, E] of dloss[0] * balance loss + dloss[1] * z loss, from the
    forward's lse, counts and n_valid (see mok_router_balance_backward)."""
    st = _call_stream(logits, stream)
    desc, _ = _balance_plan(_meta(logits), k, _meta(mask), _meta(lse), balance_coef, z_coef)
    if dlogits is None:
        dlogits = _alloc((desc.T, desc.ld_logits), torch.float32, logits.device, stream)
        if desc.ld_logits != desc.E:
            dlogits = dlogits[:, :desc.E]
    _balance_bwd_plan(_meta(dloss), _meta(logits), _meta(counts), _meta(n_valid), _meta(dlogits))
    _lib.check(_lib.load().mok_router_balance_backward(
        desc, _addr(dloss), _addr(logits), _addr(lse), _addr(counts), _addr(n_valid), _addr(mask),
        _addr(dlogits), st), "mok_router_balance_backward")
    return dlogits


@_plan
def _linear_plan(x, w, bias, residual, y, z, act):
    ld_x = _matrix(x, "x", None, _BF)
    (M, K), dev = x[0], x[3]
    _need(len(w[0]) == 2, "w must be a matrix")
    N = w[0][0]
    _dense(w, "w", (N, K), _BF, dev)
    _need(act in ACTIVATIONS, f"act must be one of {tuple(ACTIVATIONS)}")
    _need(y[2] in _ELEM, f"y must not be {y[2]}")
    if bias is not None:
        _dense(bias, "bias", (N,), _F32, dev)
    for t, name in ((y, "y"), (residual, "residual"), (z, "z")):
        if t is not None:
            _dense(t, name, (M, N), (y[2],), dev)
    return _lib.LinearDesc(M, N, K, ld_x, ACTIVATIONS[act], _ELEM[y[2]], 0, 0)


def linear(x, w, bias=None, *, act="none", residual=None, out_dtype=None, y=None, z=None,
           keep_z=False, stream=None):
    """y = act(x w^T + bias) + residual (see mok_linear_forward); with keep_z,
    (y, z) with the pre-activation z for `linear_backward`.  x [M, K] and w
    [N, K] bf16 (K a multiple of 8), bias fp32 [N]; y, z and residual [M, N] of
    out_dtype, bf16 (the default) or fp32."""
    st = _call_stream(x, stream)
    if y is None or (keep_z and z is None):
        shape = (x.shape[0], w.shape[0])
        dt = out_dtype if out_dtype is not None else (torch.bfloat16 if y is None else y.dtype)
        if y is None:
            y = _alloc(shape, dt, x.device, stream)
        if keep_z and z is None:
            z = _alloc(shape, dt, x.device, stream)
    _need(out_dtype is None or y.dtype == out_dtype, "y must have out_dtype")
    desc = _linear_plan(_meta(x), _meta(w), _meta(bias), _meta(residual), _meta(y), _meta(z), act)
    _lib.check(_lib.load().mok_linear_forward(desc, _addr(x), _addr(w), _addr(bias),
                                              _addr(residual), _addr(y), _addr(z),
                                              _addr(operator_status(x.device)), st),
               "mok_linear_forward")
    return (y, z) if keep_z else y


@_plan
def _linear_bwd_plan(dy, x, w, z, act, dx, dw, dbias, accumulate):
    ld_x = _matrix(x, "x", None, _BF)
    (M, K), dev = x[0], x[3]
    _need(len(w[0]) == 2, "w must be a matrix")
    N = w[0][0]
    _dense(w, "w", (N, K), _BF, dev)
    _dense(dy, "dy", (M, N), _ELEM, dev)
    _need(act in ACTIVATIONS, f"act must be one of {tuple(ACTIVATIONS)}")
    _need(act == "none" or z is not None, "the activation's gradient needs z")
    if z is not None:
        _dense(z, "z", (M, N), (dy[2],), dev)
    _dense(dx, "dx", (M, K), _ELEM, dev)
    _dense(dw, "dw", (N, K), _F32, dev)
    if dbias is not None:
        _dense(dbias, "dbias", (N,), _F32, dev)
    desc = _lib.LinearDesc(M, N, K, ld_x, ACTIVATIONS[act], _ELEM[dy[2]], _ELEM[dx[2]],
                           int(accumulate))
    n = ctypes.c_size_t()
    _lib.check(_lib.load().mok_linear_workspace_size(desc, n), "mok_linear_workspace_size")
    return desc, n.value


def linear_backward(dy, x, w, z=None, *, act="none", bias=False, dx_dtype=None, dx=None, dw=None,
                    dbias=None, accumulate=False, workspace=None, stream=None):
    """Gradients of `linear` (see mok_linear_backward): (dx, dw, dbias), dbias
    None unless `bias` is true or a tensor for it is given.  dy [M, N] bf16 or
    fp32, z of its type; dx bf16 (the default) or fp32; dw, dbias fp32.
    `accumulate` adds into the given dx (fp32), dw and dbias."""
    st = _call_stream(x, stream)
    _need(not accumulate or (dx is not None and dw is not None and not (bias and dbias is None)),
          "accumulate needs dx, dw and dbias to add into")
    if dx is None:
        dx = _alloc(x.shape, torch.bfloat16 if dx_dtype is None else dx_dtype, x.device, stream)
    _need(dx_dtype is None or dx.dtype == dx_dtype, "dx must have dx_dtype")
    if dw is None:
        dw = _alloc(w.shape, torch.float32, x.device, stream)
    if bias and dbias is None:
        dbias = _alloc(w.shape[:1], torch.float32, x.device, stream)
    if act == "none":
        z = None
    desc, n = _linear_bwd_plan(_meta(dy), _meta(x), _meta(w), _meta(z), act, _meta(dx), _meta(dw),
                               _meta(dbias), accumulate)
    if workspace is None:
        workspace = _alloc((n,), torch.uint8, x.device, stream)
    _lib.check(_lib.load().mok_linear_backward(desc, _addr(dy), _addr(x), _addr(w), _addr(z),
                                               _addr(dx), _addr(dw), _addr(dbias),
                                               _addr(workspace), workspace.nbytes,
                                               _addr(operator_status(x.device)), st),
               "mok_linear_backward")
    return dx, dw, dbias


def device_status(buf, stream=None) -> int:
    """Synchronises the stream and returns the device status word of `buf`."""
    lib = _lib.load()
    code = ctypes.c_int32()
    _lib.check(lib.mok_get_device_status(_ptr(buf), _stream(stream), ctypes.byref(code)),
               "mok_get_device_status")
    return code.value


def fill_zero(buf, stream=None):
    """Zeroes the contiguous device tensor `buf` with the library's bulk-store
    fill (its byte size a multiple of 16, its address 16-byte aligned)."""
    nbytes = buf.numel() * buf.element_size()
    _lib.check(_lib.load().mok_fill_zero(_ptr(buf), nbytes, _stream(stream)), "mok_fill_zero")
    return buf


def last_launch_count() -> int:
    return int(_lib.load().mok_last_launch_count())


def profile_enable(on: bool = True):
    _lib.check(_lib.load().mok_profile_enable(int(on)), "mok_profile_enable")


def profile_reset():
    _lib.check(_lib.load().mok_profile_reset(), "mok_profile_reset")


def profile_collect() -> dict:
    """{kernel name: (launches, total ms)} since the last reset (waits for the events)."""
    lib = _lib.load()
    buf = (_lib.KernelTime * 64)()
    n = ctypes.c_int32()
    _lib.check(lib.mok_profile_collect(buf, 64, ctypes.byref(n)), "mok_profile_collect")
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(n.value)}


class MoELayer:
    """Owns the three buffers of one layer shape and calls forward/backward."""

    def __init__(self, T, d, E, I, k, device="cuda", flags=0, dtype=BF16, mb_tokens=0,
                 ring_slots=0):
        self.desc = make_desc(T, d, E, I, k, dtype=dtype, flags=flags, mb_tokens=mb_tokens,
                              ring_slots=ring_slots)
        self.T, self.d, self.E, self.I, self.k = T, d, E, I, k
        self.act_dtype = torch.bfloat16 if flags & FLAG_BF16_ACT_OUT else torch.float32
        self.wgrad_dtype = torch.bfloat16 if flags & FLAG_BF16_WGRAD_OUT else torch.float32
        f, s, b = workspace_sizes(self.desc)
        self.fwd_ws = torch.empty(max(f, 256), dtype=torch.uint8, device=device)
        self.saved = torch.zeros(max(s, 256), dtype=torch.uint8, device=device)
        self.bwd_ws = torch.empty(max(b, 256), dtype=torch.uint8, device=device)
        self.layout = saved_layout(self.desc)

    def saved_tensor(self, field: str, dtype, shape, micro_batch: int = 0):
        off = getattr(self.layout, field)
        if off == NOT_KEPT:
            raise KeyError(f"{field} is not kept in saved with these flags")
        off += micro_batch * self.layout.mb_stride
        n = 1
        for v in shape:
            n *= v
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return self.saved[off:off + nbytes].view(dtype).view(*shape)

    def forward(self, x, w_router, bias, w_gate_up, w_down, y=None, stream=None):
        if y is None:
            y = torch.empty(x.shape, dtype=self.act_dtype, device=x.device)
        forward(self.desc, x, w_router, bias, w_gate_up, w_down, y, self.saved, self.fwd_ws,
                stream)
        return y

    def backward(self, dy, x, w_router, bias, w_gate_up, w_down, dx=None, dw_router=None,
                 dw_gate_up=None, dw_down=None, stream=None):
        def out(like, dt, given):
            return torch.empty(like.shape, dtype=dt, device=like.device) if given is None else given
        dx = out(x, self.act_dtype, dx)
        dw_router = out(w_router, self.wgrad_dtype, dw_router)
        dw_gate_up = out(w_gate_up, self.wgrad_dtype, dw_gate_up)
        dw_down = out(w_down, self.wgrad_dtype, dw_down)
        backward(self.desc, dy, x, w_router, bias, w_gate_up, w_down, self.saved, dx, dw_router,
                 dw_gate_up, dw_down, self.bwd_ws, stream)
        return dx, dw_router, dw_gate_up, dw_down

    def status(self, stream=None) -> int:
        return device_status(self.saved, stream)
