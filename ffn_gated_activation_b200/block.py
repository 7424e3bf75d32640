"""Tensor-level binding of the operators around the activation in an expert
block: the residual RMS norm in front of it, the whole expert layer of a
decoding step, and NVFP4 storage and products.

As in functional.py, PyTorch supplies device memory and the stream, and every
step of the computation runs in the library's kernels.  Each call runs on the
device of its tensors, whichever is current; with ``stream`` given, what it
allocates belongs to that stream.
"""
from __future__ import annotations

import contextlib
import math

import torch

from . import abi
from .functional import (DEFAULT_BETA, DEFAULT_LINEAR_BETA, _check_beta, _dtype_code, _given, _mx_rule, aligned_rows)

DEFAULT_EPSILON = 1e-6


_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream  # (device index) -> cudaStream_t


class _Scope:
    """The device (and, if given, the stream) a call runs on; yields the stream's handle."""

    __slots__ = ("device", "stream", "entered")

    def __init__(self, device, stream):
        self.device, self.stream, self.entered = device, stream, None

    def __enter__(self) -> int:
        device, stream = self.device, self.stream
        if stream is None and device.index == _current_device():
            return _current_stream(device.index)
        if stream is not None and stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        self.entered = contextlib.ExitStack()
        self.entered.enter_context(torch.cuda.device(device))
        if stream is not None:
            self.entered.enter_context(torch.cuda.stream(stream))
        return _current_stream(device.index)

    def __exit__(self, *exc):
        if self.entered is not None:
            self.entered.close()
        return False


def _cuda(t: torch.Tensor, what: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return t.device


def _on(t: torch.Tensor, device, what: str) -> None:
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")


def _all_on(device, *named) -> None:
    for i in range(0, len(named), 2):
        if named[i].device != device:
            _on(named[i], device, named[i + 1])


def _matrix(t: torch.Tensor, cols: int):
    """[..., cols] as rows of `cols` adjacent elements that do not overlap (copied
    where they do), and its row pitch.  What is contiguous comes back as it is,
    of whatever shape."""
    if t.is_contiguous():
        return t, cols
    if t.dim() != 2:
        t = t.reshape(-1, cols)
        if t.is_contiguous():
            return t, cols
    rows = t.shape[0]
    if t.numel() and (t.stride(1) != 1 or (rows > 1 and t.stride(0) < cols)):
        return t.contiguous(), cols
    return t, t.stride(0) if rows > 1 else cols


def _rows(t: torch.Tensor, cols: int) -> int:
    return t.numel() // cols if cols else 0


def _check_eps(eps):
    if type(eps) is float and 0.0 <= eps < math.inf:
        return
    if not (isinstance(eps, (int, float)) and math.isfinite(eps) and eps >= 0):
        raise ValueError(f"eps must be a finite number >= 0, got {eps!r}")


def _empty(shape, dtype, device):
    """torch.empty; with its strides given it takes half the host time."""
    if len(shape) == 2:
        return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def _out(out, shape, dtype, device, what):
    """A matrix output, allocated when not given: (tensor, its 2-D view, row pitch)."""
    cols = shape[-1]
    if out is None:
        out = _empty(shape, dtype, device)
        return out, out, cols  # contiguous: its rows follow from the pointer and the pitch
    o2 = _given(out, tuple(shape), device, what, dtype)
    return out, o2, o2.stride(0) if o2.shape[0] > 1 else cols


def _out_like(out, x, cols, what):
    """_out for an output of x's shape and dtype."""
    if out is None and x.is_contiguous():
        out = torch.empty_like(x)
        return out, out, cols
    return _out(out, x.shape, x.dtype, x.device, what)


# ---- residual addition + RMS norm -------------------------------------------------

def _norm_args(x, weight, eps, residual):
    """Checks of a norm's inputs; returns (device, dtype code, weight dtype code, hidden)."""
    device = _cuda(x, "x")
    _check_eps(eps)
    shape = x.shape
    if not shape:
        raise ValueError("x must be [..., hidden]")
    hidden = shape[-1]
    dtype, wdtype = _dtype_code(x, "x"), _dtype_code(weight, "weight")
    if weight.dim() != 1 or weight.shape[0] != hidden:
        raise ValueError(f"weight must be [{hidden}], got {tuple(weight.shape)}")
    _on(weight, device, "weight")
    if residual is not None:
        if residual.shape != shape or residual.dtype != x.dtype:
            raise ValueError(f"residual must have x's shape {tuple(shape)} and dtype {x.dtype}, got "
                             f"{tuple(residual.shape)} {residual.dtype}")
        _on(residual, device, "residual")
    return device, dtype, wdtype, hidden


def situ_glu_rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, eps: float = DEFAULT_EPSILON,
                          residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                          h_out: torch.Tensor | None = None, stream=None):
    """h = x + residual (rounded to x's dtype), y = h / sqrt(mean h^2 + eps) * weight
    over the last axis of x [..., hidden].  Returns (y, h); h is None without a
    residual.  ``weight`` [hidden] in bf16 or fp32; y and h in x's dtype."""
    args = _norm_args(x, weight, eps, residual)
    if residual is None and h_out is not None:
        raise ValueError("h_out needs a residual")
    return _norm_fwd(args, x, weight, eps, residual, out, h_out, stream)


def _norm_fwd(args, x, weight, eps, residual, out, h_out, stream):
    """situ_glu_rms_norm_fwd after its checks; ``args`` as _norm_args returns them."""
    device, dtype, wdtype, hidden = args
    with _Scope(device, stream) as handle:
        x2, xp = _matrix(x, hidden)
        w = weight.contiguous()
        y, y2, yp = _out_like(out, x, hidden, "out")
        h, r_ptr, rp, h_ptr, hp = None, None, 0, None, 0
        if residual is not None:
            r2, rp = _matrix(residual, hidden)
            h, h2, hp = _out_like(h_out, x, hidden, "h_out")
            r_ptr, h_ptr = r2.data_ptr(), h2.data_ptr()
        st = abi.situ_glu_rms_norm_fwd(x2.data_ptr(), dtype, _rows(x2, hidden), hidden, xp, r_ptr, rp, w.data_ptr(), wdtype, eps,
                                       h_ptr, hp, y2.data_ptr(), yp, handle)
    if st:
        abi.check(st, "situ_glu_rms_norm_fwd")
    return y, h


def situ_glu_rms_norm_fwd_mxfp8(x: torch.Tensor, weight: torch.Tensor, eps: float = DEFAULT_EPSILON,
                                residual: torch.Tensor | None = None, rule="ocp", data=None, scale=None,
                                h_out: torch.Tensor | None = None, stream=None):
    """The forward with MXFP8 rows (format and rules of situ_glu_fwd_mxfp8),
    quantised from the fp32 values: returns (E4M3 codes [..., hidden], scale
    bytes [..., hidden / 32], h or None).  hidden must be a multiple of 32."""
    device, dtype, wdtype, hidden = _norm_args(x, weight, eps, residual)
    if residual is None and h_out is not None:
        raise ValueError("h_out needs a residual")
    if hidden % 32:
        raise ValueError(f"hidden must be a multiple of 32, got {hidden}")
    with _Scope(device, stream) as handle:
        x2, xp = _matrix(x, hidden)
        w = weight.contiguous()
        lead = tuple(x.shape[:-1])
        data, d2, dp = _bytes(data, lead + (hidden,), torch.float8_e4m3fn, device, "MXFP8 data")
        scale, s2, sp = _bytes(scale, lead + (hidden // 32,), torch.uint8, device, "MXFP8 scale")
        h, r_ptr, rp, h_ptr, hp = None, None, 0, None, 0
        if residual is not None:
            r2, rp = _matrix(residual, hidden)
            h, h2, hp = _out_like(h_out, x, hidden, "h_out")
            r_ptr, h_ptr = r2.data_ptr(), h2.data_ptr()
        st = abi.situ_glu_rms_norm_fwd_mxfp8(x2.data_ptr(), dtype, _rows(x2, hidden), hidden, xp, r_ptr, rp, w.data_ptr(),
                                             wdtype, eps, h_ptr, hp, d2.data_ptr(), dp, s2.data_ptr(), sp, _mx_rule(rule),
                                             handle)
    if st:
        abi.check(st, "situ_glu_rms_norm_fwd_mxfp8")
    return data, scale, h


def situ_glu_rms_norm_bwd(grad_y: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = DEFAULT_EPSILON,
                          grad_h: torch.Tensor | None = None, want_dw: bool = True,
                          d_x: torch.Tensor | None = None, d_weight: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None):
    """Gradients of the forward from its h (x where there was no residual):
    returns (d_x, d_weight or None).  d_x is the gradient of x and of the
    residual; ``grad_h`` is the gradient that reaches h by itself (the residual
    stream's).  d_weight is summed in an order that the shape fixes.
    Calls that overlap on the GPU need a ``workspace`` each
    (situ_glu_rms_norm_bwd_workspace_bytes; allocated when not given)."""
    args = _norm_args(h, weight, eps, None)
    device = args[0]
    for name, g in (("grad_y", grad_y), ("grad_h", grad_h)):
        if g is not None:
            if g.shape != h.shape or g.dtype != h.dtype:
                raise ValueError(f"{name} must have h's shape {tuple(h.shape)} and dtype {h.dtype}, got "
                                 f"{tuple(g.shape)} {g.dtype}")
            _on(g, device, name)
    return _norm_bwd(args, grad_y, h, weight, eps, grad_h, want_dw, d_x, d_weight, workspace, stream)


def _norm_bwd(args, grad_y, h, weight, eps, grad_h, want_dw, d_x=None, d_weight=None, workspace=None, stream=None):
    """situ_glu_rms_norm_bwd after its checks."""
    device, dtype, wdtype, hidden = args
    with _Scope(device, stream) as handle:
        h2, hp = _matrix(h, hidden)
        g2, gp = _matrix(grad_y, hidden)
        w = weight.contiguous()
        gh_ptr, ghp = None, 0
        if grad_h is not None:
            gh2, ghp = _matrix(grad_h, hidden)
            gh_ptr = gh2.data_ptr()
        d_x, dx2, dxp = _out_like(d_x, h, hidden, "d_x")
        dw_ptr = None
        if not want_dw:
            d_weight = None
        else:
            if d_weight is None:
                d_weight = torch.empty_strided((hidden,), (1,), dtype=weight.dtype, device=device)
            elif tuple(d_weight.shape) != (hidden,) or d_weight.dtype != weight.dtype or d_weight.device != device or \
                    not d_weight.is_contiguous():
                raise ValueError(f"d_weight must be a contiguous {weight.dtype} [{hidden}] on {device}")
            dw_ptr = d_weight.data_ptr()
        tokens = _rows(h2, hidden)
        ws = abi.situ_glu_rms_norm_bwd_workspace_bytes(tokens, hidden, 1) if want_dw else 0
        ws_ptr = None
        if ws:
            workspace = _workspace(workspace, ws, device)
            ws_ptr = workspace.data_ptr()
        st = abi.situ_glu_rms_norm_bwd(g2.data_ptr(), gp, gh_ptr, ghp, h2.data_ptr(), dtype, tokens, hidden, hp,
                                       w.data_ptr(), wdtype, eps, dx2.data_ptr(), dxp, dw_ptr, ws_ptr, ws, handle)
    if st:
        abi.check(st, "situ_glu_rms_norm_bwd")
    return d_x, d_weight


def _workspace(given, nbytes: int, device) -> torch.Tensor:
    """The caller's scratch, or one allocated for this call."""
    if given is None:
        return torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=device)
    if given.device != device or not given.is_contiguous() or given.numel() * given.element_size() < nbytes:
        raise ValueError(f"workspace must be contiguous, on {device}, of at least {nbytes} bytes")
    return given


class AddRMSNormFunction(torch.autograd.Function):
    """Residual addition + RMS norm; saves h and weight only (h is an output)."""

    @staticmethod
    def forward(ctx, x, weight, eps, residual):
        ctx.set_materialize_grads(False)
        args = _norm_args(x, weight, eps, residual)
        y, h = _norm_fwd(args, x, weight, eps, residual, None, None, None)
        ctx.args, ctx.eps = args, eps
        if residual is None:
            ctx.save_for_backward(x, weight)
            return y
        ctx.save_for_backward(h, weight)
        return y, h

    @staticmethod
    def backward(ctx, grad_y, grad_h=None):
        saved = ctx.saved_tensors  # once: hooks that recompute them unpack once
        if not torch.is_grad_enabled():
            return _norm_grads(ctx, saved, grad_y, grad_h)
        with torch.no_grad():  # create_graph: a second derivative may follow
            grads = _norm_grads(ctx, saved, grad_y, grad_h)
        anchor = next(t for t in saved if t.requires_grad)
        given = [g for g in grads if g is not None]
        guarded = iter(_OnceDifferentiable.apply(anchor, *given))
        return tuple(g if g is None else next(guarded) for g in grads)


class _OnceDifferentiable(torch.autograd.Function):
    """Gradients as they are, whose own derivative is an error.  They depend on the
    norm's inputs (``anchor`` stands for these) even where the gradients that came
    in are constants, so that nothing else would tell that it is missing."""

    @staticmethod
    def forward(ctx, anchor, *grads):
        return tuple(g.view_as(g) for g in grads)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("add_rms_norm is once_differentiable: it has no second derivative")


def _norm_grads(ctx, saved, grad_y, grad_h):
    needs_x, want_dw, _, needs_residual = ctx.needs_input_grad
    h, weight = saved
    if grad_y is None:  # nothing reached y: the stream's gradient passes through
        d_x, d_w = grad_h, torch.zeros_like(weight) if want_dw else None
    else:  # the engine has checked the gradients' shapes, types and devices, not their alignment
        grad_y = aligned_rows(grad_y)
        if grad_h is not None:
            grad_h = aligned_rows(grad_h)
        d_x, d_w = _norm_bwd(ctx.args, grad_y, h, weight, ctx.eps, grad_h, want_dw)
    return d_x if needs_x else None, d_w, None, d_x if needs_residual else None


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = DEFAULT_EPSILON,
                 residual: torch.Tensor | None = None):
    """Differentiable residual addition + RMS norm over the last axis: y, or
    (y, h) with a residual (h = x + residual, the residual stream from here on).
    Gradients whose rows do not start on 16 bytes are copied; a second derivative
    is an error.
    As with any PyTorch function, a step captured into a CUDA graph whose
    backward() accumulates into leaves' .grad must not share these leaves with an
    eager graph that is still alive: drop that one first, or use
    torch.autograd.grad."""
    return AddRMSNormFunction.apply(x, weight, eps, residual)


# ---- the expert layer of a decoding step ------------------------------------------

def situ_glu_moe_fwd(x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor | None, w1: torch.Tensor,
                     w2: torch.Tensor, beta: float = DEFAULT_BETA, linear_beta: float | None = DEFAULT_LINEAR_BETA,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """y[t] = sum over t's experts of W2_e (SiTU-GLU(W1_e x[t]) w[t, e]) for up to
    64 tokens.  x: bf16 [T, H]; topk_ids: int64 [T, k], an id outside
    [0, E) is skipped (-1: an empty slot); topk_weights: [T, k] or None (1);
    w1: bf16 [E, 2I, H] (I gate rows, then I up rows); w2: bf16 [E, H, I].
    Returns bf16 [T, H].  w1 and w2 are read where they lie if their last axis is
    contiguous and the others step as one (a padded row pitch will do); anything
    else, a transposed weight say, is copied whole in every call: lay it out once.
    Calls that overlap on the GPU need a ``workspace`` each
    (situ_glu_moe_workspace_bytes; allocated when not given)."""
    _check_beta(beta, linear_beta)
    device = _cuda(x, "x")
    if not (x.dtype is w1.dtype is w2.dtype is torch.bfloat16):
        raise TypeError(f"x, w1 and w2 must be bfloat16, got {x.dtype}, {w1.dtype} and {w2.dtype}")
    if x.dim() != 2 or topk_ids.dim() != 2 or topk_ids.shape[0] != x.shape[0]:
        raise ValueError(f"x must be [T, H] and topk_ids [T, k], got {tuple(x.shape)} and {tuple(topk_ids.shape)}")
    if topk_ids.dtype != torch.int64:
        raise TypeError(f"topk_ids must be int64, got {topk_ids.dtype}")
    tokens, hidden = x.shape
    topk = topk_ids.shape[1]
    if w1.dim() != 3 or w2.dim() != 3 or w1.shape[2] != hidden or w2.shape[1] != hidden or \
            w1.shape[0] != w2.shape[0] or w1.shape[1] != 2 * w2.shape[2]:
        raise ValueError(f"w1 {tuple(w1.shape)} and w2 {tuple(w2.shape)} must be [E, 2I, {hidden}] and [E, {hidden}, I]")
    experts, inter = w2.shape[0], w2.shape[2]
    if topk_weights is not None and topk_weights.shape != topk_ids.shape:
        raise ValueError(f"topk_weights must be {tuple(topk_ids.shape)}, got {tuple(topk_weights.shape)}")
    _all_on(device, topk_ids, "topk_ids", w1, "w1", w2, "w2")
    wdtype = abi.SITU_DTYPE_F32
    if topk_weights is not None:
        _on(topk_weights, device, "topk_weights")
        wdtype = _dtype_code(topk_weights, "topk_weights")
    with _Scope(device, stream) as handle:
        x2, xp = _matrix(x, hidden)
        ids, idp = _matrix(topk_ids, topk)
        tw_ptr, twp = None, topk
        if topk_weights is not None:
            tw, twp = _matrix(topk_weights, topk)
            tw_ptr = tw.data_ptr()
        w1f, w1p = _matrix(w1, hidden)
        w2f, w2p = _matrix(w2, inter)
        out, o2, op = _out(out, (tokens, hidden), torch.bfloat16, device, "out")
        ws = abi.situ_glu_moe_workspace_bytes(tokens, topk, hidden, inter)
        ws_ptr = None
        if ws:
            workspace = _workspace(workspace, ws, device)
            ws_ptr = workspace.data_ptr()
        st = abi.situ_glu_moe_fwd(x2.data_ptr(), tokens, hidden, xp, ids.data_ptr(), topk, idp, tw_ptr, wdtype, twp,
                                  w1f.data_ptr(), experts, inter, w1p, w2f.data_ptr(), w2p, beta,
                                  int(linear_beta is not None), linear_beta if linear_beta is not None else 0.0,
                                  o2.data_ptr(), op, ws_ptr, ws, handle)
    if st:
        abi.check(st, "situ_glu_moe_fwd")
    return out


# ---- NVFP4 storage and product ----------------------------------------------------

def _amax_word(amax, device, what="amax"):
    if amax.dtype != torch.float32 or amax.numel() != 1 or amax.device != device:
        raise ValueError(f"{what} must be one float32 element on {device}")
    return amax


def situ_glu_nvfp4_quantize(x: torch.Tensor, amax: torch.Tensor | None = None, data=None, scale=None,
                            amax_out: torch.Tensor | None = None, amax_only: bool = False, stream=None):
    """NVFP4 of x [..., C] (bf16 or fp32, C a multiple of 16), in the format of
    situ_glu_fwd_nvfp4: returns (packed E2M1 codes [..., C / 2] uint8, E4M3
    block scales [..., C / 16], amax [1]).  Every code and scale is the
    correctly rounded one.  ``amax``: a known tensor maximum; otherwise it is
    computed into ``amax_out``.  ``amax_only``: (None, None, amax)."""
    device = _cuda(x, "x")
    dtype = _dtype_code(x, "x")
    if x.dim() < 1 or x.shape[-1] % 16 or x.shape[-1] == 0:
        raise ValueError(f"the last axis of x must be a positive multiple of 16, got {tuple(x.shape)}")
    cols, lead = x.shape[-1], tuple(x.shape[:-1])
    if amax_only and amax is not None:
        raise ValueError("amax_only computes the tensor maximum: do not pass one")
    with _Scope(device, stream) as handle:
        x2, xp = _matrix(x, cols)
        d_ptr, dp, s_ptr, sp = None, cols // 2, None, cols // 16
        if not amax_only:
            data, d2, dp = _bytes(data, lead + (cols // 2,), torch.uint8, device, "NVFP4 data")
            scale, s2, sp = _bytes(scale, lead + (cols // 16,), torch.float8_e4m3fn, device, "NVFP4 scale")
            d_ptr, s_ptr = d2.data_ptr(), s2.data_ptr()
        given = 2 if amax_only else int(amax is not None)
        if amax is None:
            amax = amax_out if amax_out is not None else torch.empty_strided((1,), (1,), dtype=torch.float32, device=device)
        _amax_word(amax, device)
        st = abi.situ_glu_nvfp4_quantize(x2.data_ptr(), dtype, _rows(x2, cols), cols, xp, d_ptr, dp, s_ptr, sp, amax.data_ptr(),
                                         given, handle)
    if st:
        abi.check(st, "situ_glu_nvfp4_quantize")
    return (None, None, amax) if amax_only else (data, scale, amax)


def _bytes(given, shape, dtype, device, what):
    """As _out for codes or scales: one byte an element, of any dtype where given."""
    if given is None:
        return _out(None, shape, dtype, device, what)
    return (given,) + _out(given, shape, given.dtype if given.element_size() == 1 else None, device, what)[1:]


def _codes(data, scale, what):
    """Checks of NVFP4 codes and scales [..., C / 2] and [..., C / 16]; returns C."""
    if data.element_size() != 1 or scale.element_size() != 1:
        raise TypeError(f"{what}: codes and scales are one byte an element")
    if data.dim() < 1 or scale.shape[:-1] != data.shape[:-1] or data.shape[-1] != 8 * scale.shape[-1]:
        raise ValueError(f"{what}: codes {tuple(data.shape)} and scales {tuple(scale.shape)} must be "
                         "[..., C / 2] and [..., C / 16]")
    return 2 * data.shape[-1]


def situ_glu_nvfp4_dequantize(data: torch.Tensor, scale: torch.Tensor, amax: torch.Tensor,
                              dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
    """The values q * scale * amax / 2688 that NVFP4 codes stand for, [..., C] in ``dtype``."""
    device = _cuda(data, "data")
    cols = _codes(data, scale, "situ_glu_nvfp4_dequantize")
    _on(scale, device, "scale")
    _amax_word(amax, device)
    with _Scope(device, stream) as handle:
        d2, dp = _matrix(data, cols // 2)
        s2, sp = _matrix(scale, cols // 16)
        out, o2, op = _out(out, tuple(data.shape[:-1]) + (cols,), dtype, device, "out")
        st = abi.situ_glu_nvfp4_dequantize(d2.data_ptr(), dp, s2.data_ptr(), sp, amax.data_ptr(), _rows(o2, cols), cols,
                                           o2.data_ptr(), _dtype_code(out, "out"), op, handle)
    if st:
        abi.check(st, "situ_glu_nvfp4_dequantize")
    return out


def situ_glu_nvfp4_gemm(a, w, offsets: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Grouped NVFP4 product on the fp4 tensor cores: rows [offsets[e],
    offsets[e + 1]) of a times expert e's weight transposed.

    a, w: (codes, scales, amax) as situ_glu_nvfp4_quantize and
    situ_glu_fwd_nvfp4 return them; a of [T, K], w of [E, N, K] (or [N, K]: one
    expert), its amax one element or [E].  offsets: int64 [E + 1], or None with
    one expert (every row).  Returns [T, N] in out_dtype (bf16 or fp32); rows
    outside every expert are left as they are in ``out`` (uninitialised when
    out is None)."""
    (ad, asc, aa), (wd, wsc, wa) = a, w
    device = _cuda(ad, "a")
    k = _codes(ad, asc, "a")
    if _codes(wd, wsc, "w") != k or ad.dim() != 2 or wd.dim() not in (2, 3):
        raise ValueError(f"a must hold [T, K] and w [E, N, K] or [N, K], got codes {tuple(ad.shape)} and {tuple(wd.shape)}")
    experts, n = (wd.shape[0], wd.shape[1]) if wd.dim() == 3 else (1, wd.shape[0])
    _all_on(device, asc, "a's scales", wd, "w's codes", wsc, "w's scales", wa, "w's amax")
    _amax_word(aa, device, "a's amax")
    if wa.dtype != torch.float32 or wa.numel() not in (1, experts):
        raise ValueError(f"w's amax must be 1 or {experts} float32 elements")
    if offsets is None:
        if experts != 1:
            raise ValueError(f"offsets are needed with {experts} experts")
    elif offsets.device != device or offsets.dtype != torch.int64 or offsets.dim() != 1 or offsets.numel() != experts + 1:
        raise ValueError(f"offsets must be int64 [{experts + 1}] on {device}")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    tokens = ad.shape[0]
    with _Scope(device, stream) as handle:
        (ad, adp), (asc, asp) = _matrix(ad, k // 2), _matrix(asc, k // 16)
        (wd, wdp), (wsc, wsp) = _matrix(wd, k // 2), _matrix(wsc, k // 16)
        if not wa.is_contiguous():
            wa = wa.contiguous()
        off = offsets.contiguous() if offsets is not None else None
        out, o2, op = _out(out, (tokens, n), out_dtype, device, "out")
        st = abi.situ_glu_nvfp4_gemm(ad.data_ptr(), adp, asc.data_ptr(), asp, aa.data_ptr(), tokens, k, wd.data_ptr(), wdp,
                                     wsc.data_ptr(), wsp, wa.data_ptr(), 0 if wa.numel() == 1 else 1, experts, n,
                                     off.data_ptr() if off is not None else None, o2.data_ptr(), _dtype_code(out, "out"),
                                     op, handle)
    if st:
        abi.check(st, "situ_glu_nvfp4_gemm")
    return out
