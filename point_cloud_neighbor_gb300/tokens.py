"""Operators over point tokens: layer norm, rotary positions with several
axes, and attention with a bias by squared distance.

``pc_*`` marshal arguments to the C ABI (include/pointcloud.h), forward and
backward; :func:`layer_norm`, :func:`rotary` and :func:`attention` are the
differentiable forms.  Tensors are float32 or bfloat16 on a CUDA device;
there is no CPU path.
"""
from __future__ import annotations

import ctypes
import math

import torch
from torch.autograd.function import once_differentiable

from .binding import _check_lengths, _ptr_or_none, _raise_on, lib

PC_F32, PC_BF16 = 0, 1
PC_ROTARY_HALF_SPLIT, PC_ROTARY_INVERSE = 1, 2

_DTYPES = {torch.float32: PC_F32, torch.bfloat16: PC_BF16}
_Strides = ctypes.c_int64 * 3


# The current device and stream by their raw getters: torch.cuda's wrappers
# cost more than a small kernel takes.
_current = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _run(what: str, fn, index: int, *args):
    """Call a library function with the current stream of device `index` as its
    last argument; raise on a status that is not PC_OK."""
    if _current() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st:
        _raise_on(st, what)


def _code(t, name: str) -> int:
    """The dtype code of a CUDA tensor of float32 or bfloat16."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device}); "
                         "this library has no CPU path")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16 (got {t.dtype})")
    return code


def _same(t, name: str, shape, dtype, index: int):
    """A packed tensor of a given shape, type and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.get_device() != index or t.dtype is not dtype or t.shape != shape \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape "
                         f"{tuple(shape)} on cuda:{index}")
    return t


# --- layer norm -------------------------------------------------------------------

def _norm_args(x, weight, bias):
    code = _code(x, "x")
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError("x must be contiguous with at least one axis")
    C, index, pt = x.shape[-1], x.get_device(), None
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != index \
                or t.shape != (C,) or not t.is_contiguous() \
                or t.dtype not in (torch.float32, x.dtype):
            raise ValueError(f"{name} must be a contiguous float32 or {x.dtype} tensor "
                             f"[{C}] on {x.device}")
        if pt is not None and t.dtype is not pt:
            raise ValueError("weight and bias must have the same dtype")
        pt = t.dtype
    return (code, index, C, x.numel() // C if C else 0,
            PC_F32 if pt is None else _DTYPES[pt])


def pc_layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
                  bias: torch.Tensor | None = None, eps: float = 1e-5, *,
                  return_stats: bool = False, out: torch.Tensor | None = None):
    """Layer norm over the last axis: y, or with ``return_stats`` (y, mean,
    rstd), the statistics float32 of shape ``x.shape[:-1]``."""
    code, index, C, rows, pcode = _norm_args(x, weight, bias)
    if out is None:
        out = torch.empty_like(x)
    else:
        _same(out, "out", x.shape, x.dtype, index)
    mean = rstd = None
    if return_stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    _run("pc_layer_norm", lib().pc_layer_norm, index, x.data_ptr(), code, rows, C,
         _ptr_or_none(weight), _ptr_or_none(bias), pcode, float(eps), out.data_ptr(),
         _ptr_or_none(mean), _ptr_or_none(rstd))
    return (out, mean, rstd) if return_stats else out


def pc_layer_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                           rstd: torch.Tensor, weight: torch.Tensor | None = None,
                           bias: torch.Tensor | None = None, *, need_weight: bool = True,
                           need_bias: bool = True):
    """Gradients of :func:`pc_layer_norm`: (grad_x, grad_weight, grad_bias),
    None for a parameter that is None or not needed.  ``mean`` and ``rstd``
    are the forward call's statistics."""
    code, index, C, rows, pcode = _norm_args(x, weight, bias)
    _same(grad_out, "grad_out", x.shape, x.dtype, index)
    _same(mean, "mean", x.shape[:-1], torch.float32, index)
    _same(rstd, "rstd", x.shape[:-1], torch.float32, index)
    dx = torch.empty_like(x)
    dw = torch.empty_like(weight) if weight is not None and need_weight else None
    db = torch.empty_like(bias) if bias is not None and need_bias else None
    _run("pc_layer_norm_backward", lib().pc_layer_norm_backward, index, grad_out.data_ptr(),
         x.data_ptr(), code, rows, C, mean.data_ptr(), rstd.data_ptr(), _ptr_or_none(weight),
         pcode, dx.data_ptr(), _ptr_or_none(dw), _ptr_or_none(db))
    return dx, dw, db


# --- rotary -----------------------------------------------------------------------

def _heads(t, name: str, B: int, L: int, D: int, dtype, index: int):
    """A [B, L, heads, D] tensor with a contiguous last axis: its heads and
    strides (None if packed)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != L or shape[3] != D:
        raise ValueError(f"{name} must have shape [{B}, {L}, heads, {D}] "
                         f"(got {tuple(shape)})")
    if t.dtype is not dtype or not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name} must be {dtype} on cuda:{index} (got {t.dtype} on {t.device})")
    if t.is_contiguous():
        return shape[2], None
    sb, sl, sh, sd = t.stride()
    if sd != 1 and D > 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    return shape[2], _Strides(sb, sl, sh)


def pc_rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor,
              freqs: torch.Tensor, *, interleaved: bool = True, inverse: bool = False):
    """Rotary positions with several axes: (q', k'), k' None if k is.

    q [B, L, H, D] and k [B, L, Hkv, D] (last axis contiguous, others of any
    stride); positions [B, L, A] float32, A = 1..4; freqs [A, F] float32.
    Pair a F + f of every head turns by positions[..., a] * freqs[a, f]; a
    pair is channels (2p, 2p + 1), or with ``interleaved=False`` (p, A F + p).
    Channels from 2 A F on are copied.  ``inverse`` turns back: the gradient.
    """
    code = _code(q, "q")
    if q.dim() != 4:
        raise ValueError(f"q must have shape [B, L, H, D] (got {tuple(q.shape)})")
    B, L, H, D = q.shape
    index, dtype = q.get_device(), q.dtype
    qs = _heads(q, "q", B, L, D, dtype, index)[1]
    Hkv, ks = (0, None) if k is None else _heads(k, "k", B, L, D, dtype, index)
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 2:
        raise ValueError("freqs must be a float32 CUDA tensor [A, F]")
    A, F = freqs.shape
    _same(freqs, "freqs", (A, F), torch.float32, index)
    _same(positions, "positions", (B, L, A), torch.float32, index)
    flags = (0 if interleaved else PC_ROTARY_HALF_SPLIT) | (PC_ROTARY_INVERSE if inverse else 0)
    oq = torch.empty((B, L, H, D), dtype=dtype, device=q.device)
    ok = None if k is None else torch.empty((B, L, Hkv, D), dtype=dtype, device=q.device)
    _run("pc_rotary", lib().pc_rotary, index, q.data_ptr(), _ptr_or_none(k), code, B, L, H, Hkv,
         D, qs, ks, positions.data_ptr(), freqs.data_ptr(), A, F, flags, oq.data_ptr(),
         _ptr_or_none(ok))
    return oq, ok


# --- attention --------------------------------------------------------------------

def _attention_args(q, k, v, scale, query_xyz, ref_xyz, slopes, query_lengths, ref_lengths):
    code = _code(q, "q")
    if q.dim() != 4:
        raise ValueError(f"q must have shape [B, Lq, H, D] (got {tuple(q.shape)})")
    B, Lq, H, D = q.shape
    index, dtype = q.get_device(), q.dtype
    qs = _heads(q, "q", B, Lq, D, dtype, index)[1]
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a CUDA tensor [B, Lk, Hkv, D]")
    Lk = k.shape[1]
    Hkv, ks = _heads(k, "k", B, Lk, D, dtype, index)
    Hv, vs = _heads(v, "v", B, Lk, D, dtype, index)
    if Hv != Hkv:
        raise ValueError("k and v must have the same number of heads")
    if H and (Hkv < 1 or H % Hkv):
        raise ValueError(f"the {Hkv} key heads must divide the {H} query heads")
    px = py = ps = None
    if slopes is not None and query_xyz is not None and ref_xyz is not None:
        ps = _same(slopes, "slopes", (H,), torch.float32, index).data_ptr()
        px = _same(query_xyz, "query_xyz", (B, Lq, 3), torch.float32, index).data_ptr()
        py = _same(ref_xyz, "ref_xyz", (B, Lk, 3), torch.float32, index).data_ptr()
    elif not (slopes is None and query_xyz is None and ref_xyz is None):
        raise ValueError("slopes, query_xyz and ref_xyz go together")
    ql = None if query_lengths is None else \
        _check_lengths(query_lengths, B, q.device, "query_lengths").data_ptr()
    rl = None if ref_lengths is None else \
        _check_lengths(ref_lengths, B, q.device, "ref_lengths").data_ptr()
    if scale is None:
        scale = 1.0 / math.sqrt(max(D, 1))
    return index, (q.data_ptr(), k.data_ptr(), v.data_ptr()), \
        (code, B, Lq, Lk, H, Hkv, D, qs, ks, vs, float(scale), px, py, ps, ql, rl)


def pc_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                 scale: float | None = None, query_xyz: torch.Tensor | None = None,
                 ref_xyz: torch.Tensor | None = None, slopes: torch.Tensor | None = None,
                 query_lengths: torch.Tensor | None = None,
                 ref_lengths: torch.Tensor | None = None, return_lse: bool = False,
                 return_low: bool = False):
    """Attention over point tokens: out [B, Lq, H, D], or (out, lse [B, H, Lq]),
    or (out, lse, low).

    z_ij = scale q_i.k_j - slopes[h] |query_xyz_i - ref_xyz_j|^2 over the
    first ``ref_lengths[b]`` keys; ``scale`` is 1 / sqrt(D) by default.  q
    [B, Lq, H, D], k and v [B, Lk, Hkv, D] (last axis contiguous, others of
    any stride), Hkv divides H.  slopes [H], query_xyz [B, Lq, 3] and ref_xyz
    [B, Lk, 3] are float32, all given or none.  Rows past
    ``query_lengths[b]`` and rows without keys are 0 (lse -inf); a NaN in a
    valid row or key gives NaN in the rows it enters.

    ``return_low`` (with ``return_lse``): what rounding the output to bfloat16
    left, [B, Lq, H, D] bfloat16, for the backward call; None in float32.
    """
    index, qkv, args = _attention_args(q, k, v, scale, query_xyz, ref_xyz, slopes,
                                       query_lengths, ref_lengths)
    B, Lq, H, D = q.shape
    if return_low and not return_lse:
        raise ValueError("return_low goes with return_lse")
    out = torch.empty((B, Lq, H, D), dtype=q.dtype, device=q.device)
    lse = low = None
    if return_lse:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=q.device)
    if return_low and q.dtype is torch.bfloat16:
        low = torch.empty((B, Lq, H, D), dtype=q.dtype, device=q.device)
    _run("pc_attention", lib().pc_attention_ex, index, *qkv, *args, out.data_ptr(),
         _ptr_or_none(low), _ptr_or_none(lse))
    if return_low:
        return out, lse, low
    return (out, lse) if return_lse else out


def pc_attention_backward(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                          v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, *,
                          scale: float | None = None,
                          query_xyz: torch.Tensor | None = None,
                          ref_xyz: torch.Tensor | None = None,
                          slopes: torch.Tensor | None = None,
                          query_lengths: torch.Tensor | None = None,
                          ref_lengths: torch.Tensor | None = None,
                          need_slopes: bool = True, need_q: bool = True, need_kv: bool = True,
                          out_low: torch.Tensor | None = None):
    """Gradients of :func:`pc_attention` from its ``out`` and ``lse``: (grad_q,
    grad_k, grad_v, grad_slopes), the last None without slopes or with
    ``need_slopes=False``.  The positions get no gradient.  With
    ``need_q=False`` or ``need_kv=False`` the pass that forms grad_q (and the
    slopes' gradient, for which it runs all the same), or grad_k and grad_v, is
    left out and they are None.

    A bfloat16 call needs the output before its rounding: from ``out_low``, the
    forward call's ``low``, or it runs the forward pass again.  The results are
    the same.
    """
    index, qkv, args = _attention_args(q, k, v, scale, query_xyz, ref_xyz, slopes,
                                       query_lengths, ref_lengths)
    B, Lq, H, D = shape = q.shape
    dtype, dev = q.dtype, q.device
    _same(grad_out, "grad_out", shape, dtype, index)
    _same(out, "out", shape, dtype, index)
    _same(lse, "lse", (B, H, Lq), torch.float32, index)
    if out_low is not None:
        if dtype is not torch.bfloat16:
            raise ValueError("out_low belongs to bfloat16 outputs")
        _same(out_low, "out_low", shape, dtype, index)
    ds = torch.empty_like(slopes) if slopes is not None and need_slopes else None
    dq = dk = dv = None
    if need_q or ds is not None:
        dq = torch.empty(shape, dtype=dtype, device=dev)
    if need_kv:
        dk = torch.empty(k.shape, dtype=dtype, device=dev)
        dv = torch.empty(v.shape, dtype=dtype, device=dev)
    _run("pc_attention_backward", lib().pc_attention_backward_ex, index, grad_out.data_ptr(),
         *qkv, out.data_ptr(), _ptr_or_none(out_low), lse.data_ptr(), *args, _ptr_or_none(dq),
         _ptr_or_none(dk), _ptr_or_none(dv), _ptr_or_none(ds))
    return dq if need_q else None, dk, dv, ds


# --- differentiable forms -----------------------------------------------------------

def _no_gradient(**tensors):
    """Raise for a tensor that asks for a gradient these operators do not form."""
    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{name} gets no gradient from this operator: pass "
                                 f"{name}.detach()")


# Layer norm and attention are differentiable once: their gradients come from
# library calls that autograd does not see, so a second derivative has to raise.

class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = pc_layer_norm(x, weight, bias, eps, return_stats=True)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        _, need_weight, need_bias, _ = ctx.needs_input_grad
        dx, dw, db = pc_layer_norm_backward(g.contiguous(), x, mean, rstd, weight, bias,
                                            need_weight=need_weight, need_bias=need_bias)
        return dx, dw, db, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable :func:`pc_layer_norm` (x, weight and bias; once)."""
    return _LayerNorm.apply(x.contiguous(), weight, bias, eps)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, freqs, interleaved, inverse):
        ctx.save_for_backward(positions, freqs)
        ctx.interleaved, ctx.inverse = interleaved, inverse
        return pc_rotary(q, k, positions, freqs, interleaved=interleaved, inverse=inverse)

    @staticmethod
    def backward(ctx, gq, gk):
        # the turn back, itself differentiable, of what is asked for
        gs = [g.contiguous() for g, need in zip((gq, gk), ctx.needs_input_grad) if need]
        turned = _Rotary.apply(gs[0], gs[1] if len(gs) > 1 else None, *ctx.saved_tensors,
                               ctx.interleaved, not ctx.inverse)
        dq, dk = turned if ctx.needs_input_grad[0] else (None, turned[0])
        return dq, dk, None, None, None, None


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor,
           freqs: torch.Tensor, interleaved: bool = True):
    """Differentiable :func:`pc_rotary` (q and k, any number of times; positions
    and freqs get no gradient and must not ask for one)."""
    _no_gradient(positions=positions, freqs=freqs)
    return _Rotary.apply(q, k, positions, freqs, interleaved, False)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, slopes, scale, query_xyz, ref_xyz, query_lengths, ref_lengths):
        out, lse, low = pc_attention(q, k, v, scale=scale, query_xyz=query_xyz,
                                     ref_xyz=ref_xyz, slopes=slopes,
                                     query_lengths=query_lengths, ref_lengths=ref_lengths,
                                     return_lse=True, return_low=True)
        ctx.save_for_backward(q, k, v, out, lse, low, slopes, query_xyz, ref_xyz, query_lengths,
                              ref_lengths)
        ctx.scale = scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        q, k, v, out, lse, low, slopes, qx, rx, ql, rl = ctx.saved_tensors
        dq, dk, dv, ds = pc_attention_backward(
            g.contiguous(), q, k, v, out, lse, scale=ctx.scale, query_xyz=qx, ref_xyz=rx,
            slopes=slopes, query_lengths=ql, ref_lengths=rl,
            need_slopes=ctx.needs_input_grad[3], need_q=ctx.needs_input_grad[0],
            need_kv=ctx.needs_input_grad[1] or ctx.needs_input_grad[2], out_low=low)
        return dq, dk, dv, ds, None, None, None, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
              scale: float | None = None, query_xyz: torch.Tensor | None = None,
              ref_xyz: torch.Tensor | None = None, slopes: torch.Tensor | None = None,
              query_lengths: torch.Tensor | None = None,
              ref_lengths: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable :func:`pc_attention` (q, k, v and slopes, once; the
    positions get no gradient and must not ask for one)."""
    _no_gradient(query_xyz=query_xyz, ref_xyz=ref_xyz)
    if not torch.is_grad_enabled() or not any(
            isinstance(t, torch.Tensor) and t.requires_grad for t in (q, k, v, slopes)):
        # nothing to keep for a backward pass
        return pc_attention(q, k, v, scale=scale, query_xyz=query_xyz, ref_xyz=ref_xyz,
                            slopes=slopes, query_lengths=query_lengths, ref_lengths=ref_lengths)
    return _Attention.apply(q, k, v, slopes, scale, query_xyz, ref_xyz, query_lengths,
                            ref_lengths)
