"""Python binding of the gated linear recurrence, the 8-bit activation
checkpoints and the RMS norm (include/kda.h): marshalling only, as in the
package's ``__init__``.  Every function runs asynchronously on the current stream
of its tensors' device."""
from __future__ import annotations

import ctypes
import sys

ACT8_BLOCK = 128   # values that share a scale

SYMBOLS = ("kda_glr_workspace_size", "kda_glr_fwd", "kda_glr_bwd", "kda_glr_bwd_act8", "kda_glr_step",
           "kda_act8_pack", "kda_act8_unpack", "kda_chunk_bwd_act8_workspace_size", "kda_chunk_bwd_act8",
           "kda_gdn_chunk_bwd_act8", "kda_rmsnorm_fwd", "kda_rmsnorm_fwd_act8", "kda_rmsnorm_bwd_workspace_size",
           "kda_rmsnorm_bwd", "kda_rmsnorm_bwd_act8")


def declare(lib):
    """Declares the C signatures of SYMBOLS on the loaded library."""
    vp, i32, i64, sz, f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "kda_glr_workspace_size": (sz, [i32] * 5),
        "kda_glr_fwd": (i32, [vp] * 4 + [i32] + [vp] * 2 + [i32] * 5 + [vp, sz, vp]),
        "kda_glr_bwd": (i32, [vp] * 4 + [i32] + [vp] * 5 + [i32] * 5 + [vp, sz, vp]),
        "kda_glr_bwd_act8": (i32, [vp] * 5 + [i32] + [vp] * 5 + [i32] * 5 + [vp, sz, vp]),
        "kda_glr_step": (i32, [vp] * 4 + [i32] * 4 + [vp]),
        "kda_act8_pack": (i32, [vp] * 3 + [i64, i32, i32, vp]),
        "kda_act8_unpack": (i32, [vp] * 3 + [i64, i32, i32, vp]),
        "kda_chunk_bwd_act8_workspace_size": (sz, [i32] * 7),
        "kda_chunk_bwd_act8": (i32, [vp] * 10 + [i32] + [vp] * 8 + [i32] * 7 + [vp, sz, vp]),
        "kda_gdn_chunk_bwd_act8": (i32, [vp] * 10 + [i32] + [vp] * 8 + [i32] * 7 + [vp, sz, vp]),
        "kda_rmsnorm_fwd": (i32, [vp] * 6 + [i64, i32, f, i32, i32, vp]),
        "kda_rmsnorm_fwd_act8": (i32, [vp] * 7 + [i64, i32, f, i32, i32, vp]),
        "kda_rmsnorm_bwd_workspace_size": (sz, [i64, i32]),
        "kda_rmsnorm_bwd": (i32, [vp] * 7 + [i64, i32, i32, i32, vp, sz, vp]),
        "kda_rmsnorm_bwd_act8": (i32, [vp] * 8 + [i64, i32, i32, i32, vp, sz, vp]),
    }
    assert set(sig) == set(SYMBOLS)
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args


kda = sys.modules[__package__]   # the package: its library handle, type codes and errors


class _LazyTorch:
    """torch, imported at its first use; from then on the module itself."""

    def __getattr__(self, name):
        global torch
        import torch
        return getattr(torch, name)


torch = _LazyTorch()


def _p(t):
    return None if t is None else t.data_ptr()


def _launch(dev, name, *args):
    """The library's call `name` on the current stream of dev, which is made the
    current device for it.  The device's index and the stream's handle are asked for
    directly: torch's wrappers around them take 2 us of a call of 6."""
    fn, index = getattr(kda.load_library(), name), dev.index
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != 0:
        raise kda.KDAError(rc, name, kda.kda_last_hip_error())


def _code(t):
    """The library's type code of a tensor (any other type is refused)."""
    d = t.dtype
    return 1 if d == torch.bfloat16 else 0 if d == torch.float32 else kda._dtype_code(t)


def _fits(t, dev, shape, dtype):
    """What _need asks of a tensor, all at once: the way of calls that are right."""
    return t.device == dev and t.shape == shape and t.dtype == dtype and t.is_contiguous()


def _need(name, t, dev, shape=None, dtype=None):
    if shape is not None and dtype is not None and _fits(t, dev, shape, dtype):
        return
    if t.device != dev:
        raise ValueError("%s must be on %s" % (name, dev))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, t.dtype))


def _device_of(name, t):
    if not t.is_cuda:
        raise ValueError("%s must be on a GPU, not on %s" % (name, t.device))
    return t.device


def _blocks(cols):
    return -(-cols // ACT8_BLOCK)


# ------------------------------------------------- gated linear recurrence
def kda_glr_workspace_size(B, T, D, num_seqs=0, io_dtype=1) -> int:
    return int(kda.load_library().kda_glr_workspace_size(B, T, D, num_seqs, io_dtype))


def _glr_sizes(like, cu_seqlens, dev):
    """(B, T, D, N, packed) of a [B, T, D] or, for one sequence or a packed batch, [T, D] tensor."""
    if like.dim() not in (2, 3):
        raise ValueError("expected [B, T, D] or [T, D], not %s" % (tuple(like.shape),))
    B, T, D = (1,) * (3 - like.dim()) + tuple(like.shape)
    if cu_seqlens is None:
        return B, T, D, B, 0
    _need("cu_seqlens", cu_seqlens, dev, dtype=torch.int32)
    return B, T, D, cu_seqlens.numel() - 1, cu_seqlens.numel() - 1


def _glr_workspace(B, T, D, nseq, io, workspace, dev):
    if workspace is None:
        need = kda.load_library().kda_glr_workspace_size(B, T, D, nseq, io)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    else:
        _need("workspace", workspace, dev)
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def kda_glr_fwd(x, log_alpha, h0=None, cu_seqlens=None, *, h=None, h_T=None, output_final_state=True,
                workspace=None):
    """Gated linear recurrence h_t = exp(log_alpha_t) h_{t-1} + x_t per channel.

    x, log_alpha: [B, T, D] (or [T, D] for B = 1); h0: [N, D] fp32 or None;
    cu_seqlens: int32 [N+1] on the device (B must be 1) or None.  log_alpha = -inf
    is a reset.  Returns (h, h_T), h_T [N, D] fp32 or None when
    output_final_state is False."""
    dev = _device_of("x", x)
    shape = x.shape
    _need("x", x, dev, shape, x.dtype)
    _need("log_alpha", log_alpha, dev, shape, log_alpha.dtype)
    B, T, D, N, nseq = _glr_sizes(x, cu_seqlens, dev)
    f32 = torch.float32
    if h0 is not None:
        _need("h0", h0, dev, (N, D), f32)
    io, gt = _code(x), _code(log_alpha)
    if h is None:
        h = torch.empty_like(x)
    else:
        _need("h", h, dev, x.shape, x.dtype)
    if h_T is not None:
        _need("h_T", h_T, dev, (N, D), f32)
    elif output_final_state:
        h_T = torch.empty((N, D), dtype=f32, device=dev)
    ws, wsb = _glr_workspace(B, T, D, nseq, io, workspace, dev)
    _launch(dev, "kda_glr_fwd", _p(x), _p(log_alpha), _p(h0), _p(cu_seqlens), nseq, _p(h), _p(h_T), B, T, D, io, gt,
            _p(ws), wsb)
    return h, h_T


def _glr_bwd(name, log_alpha, h, scales, grad_h, h0, grad_hT, cu_seqlens, want_grad_h0, workspace):
    dev = _device_of("grad_h", grad_h)
    f32 = torch.float32
    _need("grad_h", grad_h, dev, grad_h.shape, grad_h.dtype)
    _need("log_alpha", log_alpha, dev, grad_h.shape, log_alpha.dtype)
    B, T, D, N, nseq = _glr_sizes(grad_h, cu_seqlens, dev)
    if scales is None:
        _need("h", h, dev, grad_h.shape, grad_h.dtype)
    else:
        _need("h_codes", h, dev, grad_h.shape, torch.int8)
        _need("h_scales", scales, dev, tuple(grad_h.shape[:-1]) + (_blocks(D),), f32)
    for n, t in (("h0", h0), ("grad_hT", grad_hT)):
        if t is not None:
            _need(n, t, dev, (N, D), f32)
    io, gt = _code(grad_h), _code(log_alpha)
    dx, dla = torch.empty_like(grad_h), torch.empty_like(log_alpha)
    dh0 = torch.empty((N, D), dtype=f32, device=dev) if want_grad_h0 else None
    ws, wsb = _glr_workspace(B, T, D, nseq, io, workspace, dev)
    saved = (_p(h),) if scales is None else (_p(h), _p(scales))
    _launch(dev, name, _p(log_alpha), *saved, _p(h0), _p(cu_seqlens), nseq, _p(grad_h), _p(grad_hT), _p(dx), _p(dla),
            _p(dh0), B, T, D, io, gt, _p(ws), wsb)
    return dx, dla, dh0


def kda_glr_bwd(log_alpha, h, grad_h, h0=None, grad_hT=None, cu_seqlens=None, *, want_grad_h0=True, workspace=None):
    """Gradients of kda_glr_fwd from its output h: (dx, dlog_alpha, dh0), dh0
    None when want_grad_h0 is False."""
    return _glr_bwd("kda_glr_bwd", log_alpha, h, None, grad_h, h0, grad_hT, cu_seqlens, want_grad_h0, workspace)


def kda_glr_bwd_act8(log_alpha, h_codes, h_scales, grad_h, h0=None, grad_hT=None, cu_seqlens=None, *,
                     want_grad_h0=True, workspace=None):
    """kda_glr_bwd with h in 8 bits: codes and scales as kda_act8_pack(h) gives them."""
    return _glr_bwd("kda_glr_bwd_act8", log_alpha, h_codes, h_scales, grad_h, h0, grad_hT, cu_seqlens, want_grad_h0,
                    workspace)


def kda_glr_step(x, log_alpha, S, h=None):
    """One token of kda_glr_fwd: x, log_alpha [B, D]; S [B, D] fp32, updated in place.  Returns h."""
    dev = _device_of("x", x)
    if x.dim() != 2:
        raise ValueError("x must be [B, D], not %s" % (tuple(x.shape),))
    shape, io = x.shape, x.dtype
    _need("x", x, dev, shape, io)
    _need("log_alpha", log_alpha, dev, shape, log_alpha.dtype)
    _need("S", S, dev, shape, torch.float32)
    if h is None:
        h = torch.empty_like(x)
    else:
        _need("h", h, dev, shape, io)
    B, D = shape
    _launch(dev, "kda_glr_step", x.data_ptr(), log_alpha.data_ptr(), S.data_ptr(), h.data_ptr(), B, D, _code(x),
            _code(log_alpha))
    return h


# ---------------------------------------------- 8-bit activation checkpoints
def _rows_cols(name, t):
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError("%s must have a last axis of at least one value, not %s" % (name, tuple(t.shape)))
    cols = t.shape[-1]
    return t.numel() // cols, cols


def kda_act8_pack(x, *, codes=None, scales=None):
    """x [..., d] in 8 bits: (codes int8 [..., d], scales fp32 [..., ceil(d / 128)]),
    one scale for each 128 consecutive values of the last axis."""
    dev = _device_of("x", x)
    _need("x", x, dev, x.shape, x.dtype)
    rows, cols = _rows_cols("x", x)
    sshape = (*x.shape[:-1], _blocks(cols))
    if codes is None:
        codes = torch.empty_like(x, dtype=torch.int8)
    else:
        _need("codes", codes, dev, x.shape, torch.int8)
    if scales is None:
        scales = x.new_empty(sshape, dtype=torch.float32)
    else:
        _need("scales", scales, dev, sshape, torch.float32)
    _launch(dev, "kda_act8_pack", x.data_ptr(), codes.data_ptr(), scales.data_ptr(), rows, cols, _code(x))
    return codes, scales


def kda_act8_unpack(codes, scales, dtype=None, *, out=None):
    """The values that codes and scales (kda_act8_pack) stand for, in dtype
    (bfloat16 unless given)."""
    dev = _device_of("codes", codes)
    shape = codes.shape
    _need("codes", codes, dev, shape, torch.int8)
    rows, cols = _rows_cols("codes", codes)
    _need("scales", scales, dev, (*shape[:-1], _blocks(cols)), torch.float32)
    if out is None:
        out = torch.empty_like(codes, dtype=dtype or torch.bfloat16)
    else:
        _need("out", out, dev, shape, dtype)
    _launch(dev, "kda_act8_unpack", codes.data_ptr(), scales.data_ptr(), out.data_ptr(), rows, cols, _code(out))
    return out


def kda_chunk_bwd_act8_workspace_size(B, T, H, d_k, d_v, num_seqs=0, io_dtype=1) -> int:
    return int(kda.load_library().kda_chunk_bwd_act8_workspace_size(B, T, H, d_k, d_v, num_seqs, io_dtype))


def _chunk_bwd_act8(name, q8, k8, v8, log_alpha, beta, grad_o, h0, grad_hT, cu_seqlens, want_grad_h0, workspace):
    gdn = name == "kda_gdn_chunk_bwd_act8"
    dev = _device_of("grad_o", grad_o)
    f32, i8 = torch.float32, torch.int8
    _need("grad_o", grad_o, dev)
    if grad_o.dim() not in (3, 4):
        raise ValueError("grad_o must be [B, T, H, d_v] or [T, H, d_v], not %s" % (tuple(grad_o.shape),))
    lead = tuple(grad_o.shape[:-1])
    B, T, H = (1,) * (3 - len(lead)) + lead
    dv, dk = grad_o.shape[-1], q8[0].shape[-1]
    for n, (c, s), d in (("q", q8, dk), ("k", k8, dk), ("v", v8, dv)):
        _need(n + " codes", c, dev, lead + (d,), i8)
        _need(n + " scales", s, dev, lead + (_blocks(d),), f32)
    _need("beta", beta, dev, lead)
    if log_alpha is not None:
        _need("log_alpha", log_alpha, dev, lead if gdn else lead + (dk,), beta.dtype)
    elif not gdn:
        raise ValueError("log_alpha is required")
    if cu_seqlens is not None:
        _need("cu_seqlens", cu_seqlens, dev, dtype=torch.int32)
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    nseq = 0 if cu_seqlens is None else N
    for n, t in (("h0", h0), ("grad_hT", grad_hT)):
        if t is not None:
            _need(n, t, dev, (N, H, dk, dv), f32)
    io, gt = _code(grad_o), _code(beta)
    new = lambda d: torch.empty(lead + (d,), dtype=grad_o.dtype, device=dev)  # noqa: E731
    dq, dk_, dv_ = new(dk), new(dk), new(dv)
    dla = None if log_alpha is None else torch.empty_like(log_alpha)
    db = torch.empty_like(beta)
    dh0 = torch.empty((N, H, dk, dv), dtype=f32, device=dev) if want_grad_h0 else None
    if workspace is None:
        need = kda.load_library().kda_chunk_bwd_act8_workspace_size(B, T, H, dk, dv, nseq, io)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    else:
        _need("workspace", workspace, dev)
    _launch(dev, name, _p(q8[0]), _p(q8[1]), _p(k8[0]), _p(k8[1]), _p(v8[0]), _p(v8[1]), _p(log_alpha), _p(beta),
            _p(h0), _p(cu_seqlens), nseq, _p(grad_o), _p(grad_hT), _p(dq), _p(dk_), _p(dv_), _p(dla), _p(db), _p(dh0),
            B, T, H, dk, dv, io, gt, _p(workspace), workspace.numel() * workspace.element_size())
    return dq, dk_, dv_, dla, db, dh0


def kda_chunk_bwd_act8(q8, k8, v8, log_alpha, beta, grad_o, h0=None, grad_hT=None, cu_seqlens=None, *,
                       want_grad_h0=True, workspace=None):
    """kda_chunk_bwd with q, k and v in 8 bits: q8, k8, v8 are the (codes, scales)
    that kda_act8_pack gives for them.  Returns what kda_chunk_bwd does."""
    return _chunk_bwd_act8("kda_chunk_bwd_act8", q8, k8, v8, log_alpha, beta, grad_o, h0, grad_hT, cu_seqlens,
                           want_grad_h0, workspace)


def kda_gdn_chunk_bwd_act8(q8, k8, v8, log_alpha, beta, grad_o, h0=None, grad_hT=None, cu_seqlens=None, *,
                           want_grad_h0=True, workspace=None):
    """kda_gdn_chunk_bwd (log_alpha [B, T, H] or None) with q, k and v in 8 bits."""
    return _chunk_bwd_act8("kda_gdn_chunk_bwd_act8", q8, k8, v8, log_alpha, beta, grad_o, h0, grad_hT, cu_seqlens,
                           want_grad_h0, workspace)


# ------------------------------------------------------------------- RMS norm
def _norm_fwd(name, x, weight, residual, eps, y, codes, scales, r, want_rstd):
    dev = _device_of("x", x)
    f32 = torch.float32
    _need("x", x, dev, x.shape, x.dtype)
    rows, cols = _rows_cols("x", x)
    if weight is not None:
        _need("weight", weight, dev, (cols,), weight.dtype)
    io, wt = _code(x), _code(x if weight is None else weight)
    if residual is None:
        if r is not None:
            raise ValueError("r is the sum with a residual: there is none")
    else:
        _need("residual", residual, dev, x.shape, x.dtype)
        if r is None:
            r = torch.empty_like(x)
        else:
            _need("r", r, dev, x.shape, x.dtype)
    rstd = x.new_empty(x.shape[:-1], dtype=f32) if want_rstd else None
    if name == "kda_rmsnorm_fwd":
        if y is None:
            y = torch.empty_like(x)
        else:
            _need("y", y, dev, x.shape, x.dtype)
        out = (_p(y),)
    else:
        sshape = (*x.shape[:-1], _blocks(cols))
        if codes is None:
            codes = torch.empty_like(x, dtype=torch.int8)
        else:
            _need("codes", codes, dev, x.shape, torch.int8)
        if scales is None:
            scales = x.new_empty(sshape, dtype=f32)
        else:
            _need("scales", scales, dev, sshape, f32)
        out = (_p(codes), _p(scales))
    _launch(dev, name, _p(x), _p(residual), _p(weight), *out, _p(r), _p(rstd), rows, cols, eps, io, wt)
    r = x if residual is None else r
    return (y, r, rstd) if name == "kda_rmsnorm_fwd" else (codes, scales, r, rstd)


def kda_rmsnorm_fwd(x, weight=None, residual=None, eps=1e-6, *, y=None, r=None, want_rstd=True):
    """RMS norm over the last axis of r = x + residual (x itself without one):
    y = r / sqrt(mean(r^2) + eps) * weight.  x, residual: [..., d]; weight: [d] or
    None.  Returns (y, r, rstd); r may be given, also as x or residual itself (in
    place); rstd [...] fp32 is for the backward (None when want_rstd is False)."""
    return _norm_fwd("kda_rmsnorm_fwd", x, weight, residual, eps, y, None, None, r, want_rstd)


def kda_rmsnorm_fwd_act8(x, weight=None, residual=None, eps=1e-6, *, codes=None, scales=None, r=None,
                         want_rstd=True):
    """kda_rmsnorm_fwd with y in 8 bits (the format of kda_act8_pack).  Returns
    (codes, scales, r, rstd)."""
    return _norm_fwd("kda_rmsnorm_fwd_act8", x, weight, residual, eps, None, codes, scales, r, want_rstd)


def kda_rmsnorm_bwd_workspace_size(rows, cols) -> int:
    return int(kda.load_library().kda_rmsnorm_bwd_workspace_size(rows, cols))


def _norm_bwd(name, r, scales, weight, rstd, grad_y, grad_r, want_grad_weight, grad_x, workspace):
    dev = _device_of("grad_y", grad_y)
    f32 = torch.float32
    _need("grad_y", grad_y, dev, grad_y.shape, grad_y.dtype)
    rows, cols = _rows_cols("grad_y", grad_y)
    if scales is None:
        _need("r", r, dev, grad_y.shape, grad_y.dtype)
        saved = (_p(r),)
    else:
        _need("r_codes", r, dev, grad_y.shape, torch.int8)
        _need("r_scales", scales, dev, tuple(grad_y.shape[:-1]) + (_blocks(cols),), f32)
        saved = (_p(r), _p(scales))
    _need("rstd", rstd, dev, grad_y.shape[:-1], f32)
    if weight is not None:
        _need("weight", weight, dev, (cols,), weight.dtype)
    if grad_r is not None:
        _need("grad_r", grad_r, dev, grad_y.shape, grad_y.dtype)
    io, wt = _code(grad_y), _code(grad_y if weight is None else weight)
    if grad_x is None:
        grad_x = torch.empty_like(grad_y)
    else:
        _need("grad_x", grad_x, dev, grad_y.shape, grad_y.dtype)
    gw = None
    if want_grad_weight:
        gw = grad_y.new_empty((cols,)) if weight is None else torch.empty_like(weight)
        if workspace is None:
            need = kda.load_library().kda_rmsnorm_bwd_workspace_size(rows, cols)
            workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    if workspace is not None:
        _need("workspace", workspace, dev)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _launch(dev, name, *saved, _p(weight), _p(rstd), _p(grad_y), _p(grad_r), _p(grad_x), _p(gw), rows, cols, io, wt,
            _p(workspace), wsb)
    return grad_x, gw


def kda_rmsnorm_bwd(r, weight, rstd, grad_y, grad_r=None, *, want_grad_weight=True, grad_x=None, workspace=None):
    """Gradients of kda_rmsnorm_fwd: (grad_x, grad_weight).  grad_x is the gradient
    of x and of residual alike; grad_r (or None) is the gradient that reaches r by
    its other uses; grad_weight is None when want_grad_weight is False."""
    return _norm_bwd("kda_rmsnorm_bwd", r, None, weight, rstd, grad_y, grad_r, want_grad_weight, grad_x, workspace)


def kda_rmsnorm_bwd_act8(r_codes, r_scales, weight, rstd, grad_y, grad_r=None, *, want_grad_weight=True, grad_x=None,
                         workspace=None):
    """kda_rmsnorm_bwd with r in 8 bits: codes and scales as kda_act8_pack(r) gives them."""
    return _norm_bwd("kda_rmsnorm_bwd_act8", r_codes, r_scales, weight, rstd, grad_y, grad_r, want_grad_weight,
                     grad_x, workspace)


# ------------------------------------------------------------------- autograd
# To capture a training step into a graph, capture the kda_* calls: torch's own
# bookkeeping of leaf gradients belongs to the stream on which an eager graph of the
# same leaves was built, and its backward may not run under another stream's capture.
_FUNCTIONS = {}


def _function(name):
    """The autograd functions, made on first use (torch is imported lazily)."""
    if not _FUNCTIONS:
        class _GLR(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, log_alpha, h0, cu_seqlens, act8):
                h, h_T = kda_glr_fwd(x, log_alpha, h0=h0, cu_seqlens=cu_seqlens)
                saved = kda_act8_pack(h) if act8 else (h, None)
                ctx.save_for_backward(log_alpha, h0, cu_seqlens, *saved)
                ctx.io_dtype = x.dtype
                ctx.set_materialize_grads(False)
                return h, h_T

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, grad_h, grad_hT):
                log_alpha, h0, cu_seqlens, h, scales = ctx.saved_tensors
                if grad_h is None and grad_hT is None:
                    return None, None, None, None, None
                if grad_h is None:
                    grad_h = torch.zeros(log_alpha.shape, dtype=ctx.io_dtype, device=log_alpha.device)
                name = "kda_glr_bwd" if scales is None else "kda_glr_bwd_act8"
                dx, dla, dh0 = _glr_bwd(name, log_alpha, h, scales, grad_h.contiguous(), h0,
                                        None if grad_hT is None else grad_hT.contiguous(), cu_seqlens,
                                        h0 is not None and ctx.needs_input_grad[2], None)
                return dx, dla, dh0, None, None

        class _Norm(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, weight, residual, eps, act8):
                y, r, rstd = kda_rmsnorm_fwd(x, weight, residual, eps)
                saved = kda_act8_pack(r) if act8 else (r, None)
                ctx.save_for_backward(weight, rstd, *saved)
                ctx.set_materialize_grads(False)
                ctx.with_residual = residual is not None
                return (y, r) if ctx.with_residual else y

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, grad_y, grad_r=None):
                weight, rstd, r, scales = ctx.saved_tensors
                if grad_y is None:   # only the stream's sum was used
                    return grad_r, None, grad_r, None, None
                want_w = weight is not None and ctx.needs_input_grad[1]
                name = "kda_rmsnorm_bwd" if scales is None else "kda_rmsnorm_bwd_act8"
                dx, dw = _norm_bwd(name, r, scales, weight, rstd, grad_y.contiguous(),
                                   None if grad_r is None else grad_r.contiguous(), want_w, None, None)
                return dx, dw, dx if ctx.with_residual else None, None, None

        _FUNCTIONS.update(glr=_GLR, norm=_Norm)
    return _FUNCTIONS[name]


def gated_linear_recurrence(x, log_alpha, h0=None, cu_seqlens=None, *, act8=False):
    """kda_glr_fwd with autograd: returns (h, h_T), and gradients flow to x,
    log_alpha and h0 through kda_glr_bwd.  With act8 the forward keeps h for the
    backward in 8 bits (about half of bf16's memory); dlog_alpha is then taken at
    those values, dx and dh0 do not depend on them.  Under graph capture call
    kda_glr_fwd and kda_glr_bwd instead: torch may not run a captured backward while
    an eager graph of the same leaves lives."""
    return _function("glr").apply(x, log_alpha, h0, cu_seqlens, act8)


def rms_norm(x, weight=None, residual=None, eps=1e-6, *, act8=False):
    """kda_rmsnorm_fwd with autograd: returns y, or (y, r) with a residual, r = x +
    residual being the new stream.  Gradients flow to x, weight and residual.  With
    act8 the forward keeps r for the backward in 8 bits.  Under graph capture call
    kda_rmsnorm_fwd and kda_rmsnorm_bwd instead, as for gated_linear_recurrence."""
    return _function("norm").apply(x, weight, residual, eps, act8)
