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

from .binding import _check_lengths, _ptr_or_none, _raise_on, lib

PC_F32, PC_BF16 = 0, 1
PC_ROTARY_HALF_SPLIT, PC_ROTARY_INVERSE = 1, 2

_DTYPES = {torch.float32: PC_F32, torch.bfloat16: PC_BF16}
_Strides = ctypes.c_int64 * 3


class _NoSwitch:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_HERE = _NoSwitch()


def _on(device: torch.device):
    """The device's context, without the cost of a switch where it is current."""
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _tensor(t, name: str, dtypes=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device}); "
                         "this library has no CPU path")
    if t.dtype not in (_DTYPES if dtypes is None else dtypes):
        raise ValueError(f"{name} must be float32 or bfloat16 (got {t.dtype})"
                         if dtypes is None else f"{name} must be {dtypes[0]} (got {t.dtype})")
    return t


def _same(t, name: str, shape, dtype, device, what: str = ""):
    """A packed tensor of a given shape, type and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape "
                         f"{tuple(shape)} on {device}{what}")
    return t


# --- layer norm -------------------------------------------------------------------

def _norm_args(x, weight, bias):
    _tensor(x, "x")
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError("x must be contiguous with at least one axis")
    C = x.shape[-1]
    pt = None
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.device != x.device or t.shape != (C,) \
                or not t.is_contiguous() or t.dtype not in (torch.float32, x.dtype):
            raise ValueError(f"{name} must be a contiguous float32 or {x.dtype} tensor "
                             f"[{C}] on {x.device}")
        if pt is not None and t.dtype != pt:
            raise ValueError("weight and bias must have the same dtype")
        pt = t.dtype
    return C, (x.numel() // C if C else 0), torch.float32 if pt is None else pt


def pc_layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
                  bias: torch.Tensor | None = None, eps: float = 1e-5, *,
                  return_stats: bool = False, out: torch.Tensor | None = None):
    """Layer norm over the last axis: y, or with ``return_stats`` (y, mean,
    rstd), the statistics float32 of shape ``x.shape[:-1]``."""
    C, rows, pt = _norm_args(x, weight, bias)
    dev = x.device
    with _on(dev):
        if out is None:
            out = torch.empty_like(x)
        else:
            _same(out, "out", x.shape, x.dtype, dev)
        mean = rstd = None
        if return_stats:
            mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
            rstd = torch.empty_like(mean)
        st = lib().pc_layer_norm(x.data_ptr(), _DTYPES[x.dtype], rows, C,
                                 _ptr_or_none(weight), _ptr_or_none(bias), _DTYPES[pt],
                                 float(eps), out.data_ptr(), _ptr_or_none(mean),
                                 _ptr_or_none(rstd), _stream(dev))
    _raise_on(st, "pc_layer_norm")
    return (out, mean, rstd) if return_stats else out


def pc_layer_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                           rstd: torch.Tensor, weight: torch.Tensor | None = None,
                           bias: torch.Tensor | None = None):
    """Gradients of :func:`pc_layer_norm`: (grad_x, grad_weight, grad_bias),
    None for a parameter that is None.  ``mean`` and ``rstd`` are the forward
    call's statistics."""
    C, rows, pt = _norm_args(x, weight, bias)
    dev = x.device
    _same(grad_out, "grad_out", x.shape, x.dtype, dev)
    _same(mean, "mean", x.shape[:-1], torch.float32, dev)
    _same(rstd, "rstd", x.shape[:-1], torch.float32, dev)
    with _on(dev):
        dx = torch.empty_like(x)
        dw = None if weight is None else torch.empty_like(weight)
        db = None if bias is None else torch.empty_like(bias)
        st = lib().pc_layer_norm_backward(
            grad_out.data_ptr(), x.data_ptr(), _DTYPES[x.dtype], rows, C, mean.data_ptr(),
            rstd.data_ptr(), _ptr_or_none(weight), _DTYPES[pt], dx.data_ptr(),
            _ptr_or_none(dw), _ptr_or_none(db), _stream(dev))
    _raise_on(st, "pc_layer_norm_backward")
    return dx, dw, db


# --- rotary -----------------------------------------------------------------------

def _heads(t, name: str, B: int, L: int, D: int, dtype, device):
    """A [B, L, heads, D] tensor with a contiguous last axis."""
    _tensor(t, name)
    if t.dim() != 4 or t.shape[0] != B or t.shape[1] != L or t.shape[3] != D:
        raise ValueError(f"{name} must have shape [{B}, {L}, heads, {D}] "
                         f"(got {tuple(t.shape)})")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} on {device} (got {t.dtype} on {t.device})")
    if t.stride(3) != 1 and D > 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    return t


def _strides_of(t):
    return None if t.is_contiguous() else _Strides(t.stride(0), t.stride(1), t.stride(2))


def pc_rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor,
              freqs: torch.Tensor, *, interleaved: bool = True, inverse: bool = False):
    """Rotary positions with several axes: (q', k'), k' None if k is.

    q [B, L, H, D] and k [B, L, Hkv, D] (last axis contiguous, others of any
    stride); positions [B, L, A] float32, A = 1..4; freqs [A, F] float32.
    Pair a F + f of every head turns by positions[..., a] * freqs[a, f]; a
    pair is channels (2p, 2p + 1), or with ``interleaved=False`` (p, A F + p).
    Channels from 2 A F on are copied.  ``inverse`` turns back: the gradient.
    """
    _tensor(q, "q")
    if q.dim() != 4:
        raise ValueError(f"q must have shape [B, L, H, D] (got {tuple(q.shape)})")
    B, L, H, D = q.shape
    dev = q.device
    _heads(q, "q", B, L, D, q.dtype, dev)
    if k is not None:
        _heads(k, "k", B, L, D, q.dtype, dev)
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 2:
        raise ValueError("freqs must be a float32 CUDA tensor [A, F]")
    A, F = freqs.shape
    _same(freqs, "freqs", (A, F), torch.float32, dev)
    _same(positions, "positions", (B, L, A), torch.float32, dev)
    flags = (0 if interleaved else PC_ROTARY_HALF_SPLIT) | (PC_ROTARY_INVERSE if inverse else 0)
    with _on(dev):
        oq = torch.empty(q.shape, dtype=q.dtype, device=dev)
        ok = None if k is None else torch.empty(k.shape, dtype=q.dtype, device=dev)
        st = lib().pc_rotary(q.data_ptr(), _ptr_or_none(k), _DTYPES[q.dtype], B, L, H,
                             0 if k is None else k.shape[2], D, _strides_of(q),
                             None if k is None else _strides_of(k), positions.data_ptr(),
                             freqs.data_ptr(), A, F, flags, oq.data_ptr(),
                             _ptr_or_none(ok), _stream(dev))
    _raise_on(st, "pc_rotary")
    return oq, ok


# --- attention --------------------------------------------------------------------

def _attention_args(q, k, v, scale, query_xyz, ref_xyz, slopes, query_lengths, ref_lengths):
    _tensor(q, "q")
    if q.dim() != 4:
        raise ValueError(f"q must have shape [B, Lq, H, D] (got {tuple(q.shape)})")
    B, Lq, H, D = q.shape
    dev = q.device
    _heads(q, "q", B, Lq, D, q.dtype, dev)
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a CUDA tensor [B, Lk, Hkv, D]")
    Lk, Hkv = k.shape[1], k.shape[2]
    _heads(k, "k", B, Lk, D, q.dtype, dev)
    _heads(v, "v", B, Lk, D, q.dtype, dev)
    if v.shape[2] != Hkv:
        raise ValueError("k and v must have the same number of heads")
    if H and (Hkv < 1 or H % Hkv):
        raise ValueError(f"the {Hkv} key heads must divide the {H} query heads")
    if (slopes is None) != (query_xyz is None) or (slopes is None) != (ref_xyz is None):
        raise ValueError("slopes, query_xyz and ref_xyz go together")
    if slopes is not None:
        _same(slopes, "slopes", (H,), torch.float32, dev)
        _same(query_xyz, "query_xyz", (B, Lq, 3), torch.float32, dev)
        _same(ref_xyz, "ref_xyz", (B, Lk, 3), torch.float32, dev)
    ql = _check_lengths(query_lengths, B, dev, "query_lengths")
    rl = _check_lengths(ref_lengths, B, dev, "ref_lengths")
    if scale is None:
        scale = 1.0 / math.sqrt(max(D, 1))
    return (_DTYPES[q.dtype], B, Lq, Lk, H, Hkv, D, _strides_of(q), _strides_of(k),
            _strides_of(v), float(scale), _ptr_or_none(query_xyz), _ptr_or_none(ref_xyz),
            _ptr_or_none(slopes), _ptr_or_none(ql), _ptr_or_none(rl))


def pc_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                 scale: float | None = None, query_xyz: torch.Tensor | None = None,
                 ref_xyz: torch.Tensor | None = None, slopes: torch.Tensor | None = None,
                 query_lengths: torch.Tensor | None = None,
                 ref_lengths: torch.Tensor | None = None, return_lse: bool = False):
    """Attention over point tokens: out [B, Lq, H, D], or (out, lse [B, H, Lq]).

    z_ij = scale q_i.k_j - slopes[h] |query_xyz_i - ref_xyz_j|^2 over the
    first ``ref_lengths[b]`` keys; ``scale`` is 1 / sqrt(D) by default.  q
    [B, Lq, H, D], k and v [B, Lk, Hkv, D] (last axis contiguous, others of
    any stride), Hkv divides H.  slopes [H], query_xyz [B, Lq, 3] and ref_xyz
    [B, Lk, 3] are float32, all given or none.  Rows past
    ``query_lengths[b]`` and rows without keys are 0 (lse -inf).
    """
    args = _attention_args(q, k, v, scale, query_xyz, ref_xyz, slopes, query_lengths,
                           ref_lengths)
    dev = q.device
    with _on(dev):
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        lse = None
        if return_lse:
            lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32,
                              device=dev)
        st = lib().pc_attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), *args,
                                out.data_ptr(), _ptr_or_none(lse), _stream(dev))
    _raise_on(st, "pc_attention")
    return (out, lse) if return_lse else out


def pc_attention_backward(grad_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                          v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, *,
                          scale: float | None = None,
                          query_xyz: torch.Tensor | None = None,
                          ref_xyz: torch.Tensor | None = None,
                          slopes: torch.Tensor | None = None,
                          query_lengths: torch.Tensor | None = None,
                          ref_lengths: torch.Tensor | None = None,
                          need_slopes: bool = True):
    """Gradients of :func:`pc_attention` from its ``out`` and ``lse``: (grad_q,
    grad_k, grad_v, grad_slopes), the last None without slopes or with
    ``need_slopes=False``.  The positions get no gradient."""
    args = _attention_args(q, k, v, scale, query_xyz, ref_xyz, slopes, query_lengths,
                           ref_lengths)
    dev = q.device
    B, Lq, H, _ = q.shape
    _same(grad_out, "grad_out", q.shape, q.dtype, dev)
    _same(out, "out", q.shape, q.dtype, dev)
    _same(lse, "lse", (B, H, Lq), torch.float32, dev)
    with _on(dev):
        dq = torch.empty(q.shape, dtype=q.dtype, device=dev)
        dk = torch.empty(k.shape, dtype=q.dtype, device=dev)
        dv = torch.empty(v.shape, dtype=q.dtype, device=dev)
        ds = torch.empty_like(slopes) if slopes is not None and need_slopes else None
        st = lib().pc_attention_backward(
            grad_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
            lse.data_ptr(), *args, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
            _ptr_or_none(ds), _stream(dev))
    _raise_on(st, "pc_attention_backward")
    return dq, dk, dv, ds


# --- differentiable forms -----------------------------------------------------------

class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = pc_layer_norm(x, weight, bias, eps, return_stats=True)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, g):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        dx, dw, db = pc_layer_norm_backward(g.contiguous(), x, mean, rstd, weight, bias)
        return dx, dw, db, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable :func:`pc_layer_norm` (x, weight and bias)."""
    return _LayerNorm.apply(x.contiguous(), weight, bias, eps)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, freqs, interleaved):
        ctx.save_for_backward(positions, freqs)
        ctx.interleaved = interleaved
        return pc_rotary(q, k, positions, freqs, interleaved=interleaved)

    @staticmethod
    def backward(ctx, gq, gk):
        positions, freqs = ctx.saved_tensors
        dq, dk = pc_rotary(gq.contiguous(), None if gk is None else gk.contiguous(),
                           positions, freqs, interleaved=ctx.interleaved, inverse=True)
        return dq, dk, None, None, None


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor,
           freqs: torch.Tensor, interleaved: bool = True):
    """Differentiable :func:`pc_rotary` (q and k; not positions, not freqs)."""
    return _Rotary.apply(q, k, positions, freqs, interleaved)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, slopes, scale, query_xyz, ref_xyz, query_lengths, ref_lengths):
        out, lse = pc_attention(q, k, v, scale=scale, query_xyz=query_xyz, ref_xyz=ref_xyz,
                                slopes=slopes, query_lengths=query_lengths,
                                ref_lengths=ref_lengths, return_lse=True)
        ctx.save_for_backward(q, k, v, out, lse, slopes, query_xyz, ref_xyz, query_lengths,
                              ref_lengths)
        ctx.scale = scale
        return out

    @staticmethod
    def backward(ctx, g):
        q, k, v, out, lse, slopes, qx, rx, ql, rl = ctx.saved_tensors
        dq, dk, dv, ds = pc_attention_backward(
            g.contiguous(), q, k, v, out, lse, scale=ctx.scale, query_xyz=qx, ref_xyz=rx,
            slopes=slopes, query_lengths=ql, ref_lengths=rl,
            need_slopes=ctx.needs_input_grad[3])
        return dq, dk, dv, ds, None, None, None, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
              scale: float | None = None, query_xyz: torch.Tensor | None = None,
              ref_xyz: torch.Tensor | None = None, slopes: torch.Tensor | None = None,
              query_lengths: torch.Tensor | None = None,
              ref_lengths: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable :func:`pc_attention` (q, k, v and slopes; not the
    positions)."""
    return _Attention.apply(q, k, v, slopes, scale, query_xyz, ref_xyz, query_lengths,
                            ref_lengths)
