"""Operators over the features of points: group norm with an activation, gated
projections, and the lookup of feature rows.

``pc_*`` marshal arguments to the C ABI (include/pointcloud.h), forward and
backward; :func:`group_norm`, :func:`gated_linear` and :func:`embedding` are
the differentiable forms.  Tensors are float32 or bfloat16 on a CUDA device;
there is no CPU path.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from .binding import _check_lengths, _ptr_or_none, lib
from .tokens import PC_F32, _DTYPES, _code, _run, _same

PC_ACT_NONE, PC_ACT_SILU, PC_ACT_GELU, PC_ACT_RELU, PC_ACT_SIGMOID = range(5)

_ACTIVATIONS = {"none": PC_ACT_NONE, None: PC_ACT_NONE, "silu": PC_ACT_SILU,
                "gelu": PC_ACT_GELU, "relu": PC_ACT_RELU, "sigmoid": PC_ACT_SIGMOID}


def _activation(name) -> int:
    try:
        return _ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError("activation must be one of 'none', 'silu', 'gelu', 'relu', 'sigmoid' "
                         f"(got {name!r})") from None


def _packed(t, name: str, shape, dtype, index: int):
    """The address of a packed tensor of a given shape, type and device (the short way for
    what is right; _same says what is wrong)."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape \
            and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    return _same(t, name, shape, dtype, index).data_ptr()


def _count(shape) -> int:
    n = 1
    for k in shape:
        n *= k
    return n


# --- group norm -------------------------------------------------------------------

def _group_param(t, name: str, x, C: int, index: int):
    if not isinstance(t, torch.Tensor) or t.shape != (C,) or t.get_device() != index \
            or not t.is_contiguous() or t.dtype not in (torch.float32, x.dtype):
        raise ValueError(f"{name} must be a contiguous float32 or {x.dtype} tensor "
                         f"[{C}] on {x.device}")
    return t.data_ptr(), t.dtype


def _group_args(x, groups, weight, bias, activation, lengths):
    code = _code(x, "x")
    shape = x.shape
    if len(shape) != 3 or not x.is_contiguous():
        raise ValueError(f"x must be contiguous [B, L, C] (got {tuple(shape)})")
    B, L, C = shape
    index = x.get_device()
    groups = int(groups)
    if groups < 1 or C % groups:
        raise ValueError(f"groups={groups} must divide the {C} channels")
    pw = pb = wt = bt = None
    if weight is not None:
        pw, wt = _group_param(weight, "weight", x, C, index)
    if bias is not None:
        pb, bt = _group_param(bias, "bias", x, C, index)
        if wt is not None and bt is not wt:
            raise ValueError("weight and bias must have the same dtype")
    pt = wt or bt
    pl = None if lengths is None else _check_lengths(lengths, B, x.device, "lengths").data_ptr()
    return (code, index, B, L, C, groups, pw, pb, PC_F32 if pt is None else _DTYPES[pt],
            _activation(activation), pl)


def pc_group_norm(x: torch.Tensor, groups: int, weight: torch.Tensor | None = None,
                  bias: torch.Tensor | None = None, eps: float = 1e-5, *,
                  activation: str | None = None, lengths: torch.Tensor | None = None,
                  return_stats: bool = False, out: torch.Tensor | None = None):
    """Group norm of x [B, L, C] over each cloud's points and C / groups
    neighbouring channels, then an activation ('none', 'silu', 'gelu', 'relu',
    'sigmoid'): y, or with ``return_stats`` (y, mean, rstd), the statistics
    float32 [B, groups].

    Only the first ``lengths[b]`` points count ([B] int64); what lies past them
    is not read into any result, and y is 0 there.
    """
    code, index, B, L, C, groups, pw, pb, pcode, act, pl = _group_args(
        x, groups, weight, bias, activation, lengths)
    if out is None:
        out = torch.empty_like(x)
    else:
        _same(out, "out", x.shape, x.dtype, index)
    if not return_stats:
        _run("pc_group_norm", lib().pc_group_norm, index, x.data_ptr(), code, B, L, C, groups,
             pw, pb, pcode, float(eps), act, pl, out.data_ptr(), None, None)
        return out
    mean = torch.empty((B, groups), dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    _run("pc_group_norm", lib().pc_group_norm, index, x.data_ptr(), code, B, L, C, groups, pw,
         pb, pcode, float(eps), act, pl, out.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    return out, mean, rstd


def pc_group_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                           rstd: torch.Tensor, groups: int,
                           weight: torch.Tensor | None = None,
                           bias: torch.Tensor | None = None, *,
                           activation: str | None = None,
                           lengths: torch.Tensor | None = None, need_x: bool = True,
                           need_weight: bool = True, need_bias: bool = True):
    """Gradients of :func:`pc_group_norm`: (grad_x, grad_weight, grad_bias), None
    for what is not needed or for a parameter that is None.  ``mean`` and
    ``rstd`` are the forward call's statistics; ``bias`` enters the
    activation's derivative."""
    code, index, B, L, C, groups, pw, pb, pcode, act, pl = _group_args(
        x, groups, weight, bias, activation, lengths)
    pg = _packed(grad_out, "grad_out", x.shape, x.dtype, index)
    pm = _packed(mean, "mean", (B, groups), torch.float32, index)
    pr = _packed(rstd, "rstd", (B, groups), torch.float32, index)
    dx = torch.empty_like(x) if need_x else None
    dw = torch.empty_like(weight) if weight is not None and need_weight else None
    db = torch.empty_like(bias) if bias is not None and need_bias else None
    _run("pc_group_norm_backward", lib().pc_group_norm_backward, index, pg, x.data_ptr(), code,
         B, L, C, groups, pm, pr, pw, pb, pcode, act, pl, _ptr_or_none(dx), _ptr_or_none(dw),
         _ptr_or_none(db))
    return dx, dw, db


# --- gated projection ---------------------------------------------------------------

def _gated_args(x, w_gate, w_up, b_gate, b_up, activation):
    code = _code(x, "x")
    shape = x.shape
    if not shape or not x.is_contiguous():
        raise ValueError("x must be contiguous with at least one axis")
    C, index, dtype = shape[-1], x.get_device(), x.dtype
    if not isinstance(w_gate, torch.Tensor) or w_gate.dim() != 2 or w_gate.shape[1] != C:
        raise ValueError(f"w_gate must be a {dtype} CUDA tensor [F, {C}]")
    ws = w_gate.shape
    F = ws[0]
    pg, pu = _packed(w_gate, "w_gate", ws, dtype, index), _packed(w_up, "w_up", ws, dtype, index)
    bg = bu = None
    if b_gate is not None and b_up is not None:
        bg = _packed(b_gate, "b_gate", (F,), dtype, index)
        bu = _packed(b_up, "b_up", (F,), dtype, index)
    elif not (b_gate is None and b_up is None):
        raise ValueError("b_gate and b_up go together")
    rows = shape[0] if len(shape) == 2 else _count(shape[:-1])
    return index, (x.data_ptr(), code, rows, C, F, pg, pu, bg, bu, _activation(activation)), F


PC_GATED_GRAD_X, PC_GATED_GRAD_WEIGHT, PC_GATED_GRAD_BIAS = 1, 2, 4
PC_GATED_UNALIGNED = 8


# Calls of as many elements take their scratch from torch's allocator, which keeps it
# (the library's pool does for smaller ones).
LARGE = 1 << 24


def _workspace(x, args, gradients: int, index: int):
    px, code, rows, C, F, pg, pu = args[:7]
    if (px | pg | pu) % 16:
        gradients |= PC_GATED_UNALIGNED
    with torch.cuda.device(index):
        n = lib().pc_gated_linear_workspace_bytes(code, rows, C, F, gradients)
    return (torch.empty(n, dtype=torch.uint8, device=x.device), n) if n else (None, 0)


def pc_gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                    b_gate: torch.Tensor | None = None, b_up: torch.Tensor | None = None, *,
                    activation: str | None = "silu",
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """act(x w_gate^T + b_gate) * (x w_up^T + b_up): the first half of a gated
    feed-forward block.  x [..., C]; w_gate and w_up [F, C], as in a linear
    layer; b_gate and b_up [F], both or neither; all of one dtype.  Returns
    [..., F].  In float32 an infinity in x or the weights (or a value beyond
    3.389e38) makes what it enters NaN, whatever the definition gives there."""
    index, args, F = _gated_args(x, w_gate, w_up, b_gate, b_up, activation)
    shape = (*x.shape[:-1], F)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    else:
        _same(out, "out", shape, x.dtype, index)
    work, n = None, 0
    if args[2] * (args[3] + 2 * F) >= LARGE:
        work, n = _workspace(x, args, 0, index)
    _run("pc_gated_linear", lib().pc_gated_linear, index, *args, out.data_ptr(),
         _ptr_or_none(work), n)
    return out


def pc_gated_linear_backward(grad_out: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor,
                             w_up: torch.Tensor, b_gate: torch.Tensor | None = None,
                             b_up: torch.Tensor | None = None, *,
                             activation: str | None = "silu", need_x: bool = True,
                             need_weight: bool = True, need_bias: bool = True):
    """Gradients of :func:`pc_gated_linear`: (grad_x, grad_w_gate, grad_w_up,
    grad_b_gate, grad_b_up), None for what is not needed or was None.  Nothing
    of the forward call is needed but its arguments.  Only the results are rounded
    to the type: in bfloat16 the gradients of the two projections enter their
    products in two parts."""
    index, args, F = _gated_args(x, w_gate, w_up, b_gate, b_up, activation)
    _same(grad_out, "grad_out", (*x.shape[:-1], F), x.dtype, index)
    dx = torch.empty_like(x) if need_x else None
    dwg = dwu = dbg = dbu = None
    if need_weight:
        dwg, dwu = torch.empty_like(w_gate), torch.empty_like(w_up)
    if need_bias and b_gate is not None:
        dbg, dbu = torch.empty_like(b_gate), torch.empty_like(b_up)
    which = (PC_GATED_GRAD_X if need_x else 0) | (PC_GATED_GRAD_WEIGHT if need_weight else 0) \
        | (PC_GATED_GRAD_BIAS if dbg is not None else 0)
    work, n = None, 0
    if which and args[2] * (args[3] + 2 * F) >= LARGE:
        work, n = _workspace(x, args, which, index)
    _run("pc_gated_linear_backward", lib().pc_gated_linear_backward, index,
         grad_out.data_ptr(), *args, _ptr_or_none(dx), _ptr_or_none(dwg), _ptr_or_none(dwu),
         _ptr_or_none(dbg), _ptr_or_none(dbu), _ptr_or_none(work), n)
    return dx, dwg, dwu, dbg, dbu


# --- lookup -----------------------------------------------------------------------

def _lookup(idx, index: int):
    """The address of indices."""
    if isinstance(idx, torch.Tensor) and idx.dtype is torch.int64 \
            and idx.get_device() == index and idx.is_contiguous():
        return idx.data_ptr()
    raise ValueError(f"idx must be a contiguous int64 tensor on cuda:{index}")


def _lookup_sizes(idx, ts):
    """Tables, rows, channels, indices into each; the shape of the rows looked up."""
    s = idx.shape
    if len(ts) == 2:
        return 1, ts[0], ts[1], idx.numel(), (*s, ts[1])
    B = ts[0]
    if not s or s[0] != B:
        raise ValueError(f"idx must have shape [{B}, ...] (got {tuple(s)})")
    return B, ts[1], ts[2], _count(s[1:]), (*s, ts[2])


def pc_embedding(table: torch.Tensor, idx: torch.Tensor, scale: float = 1.0, *,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """scale * table[idx], zeros where idx = -1.

    table [V, C] with idx of any shape, or a table for each cloud [B, V, C]
    with idx [B, ...] (the neighbours that kNN or Ball Query found).  Returns
    [*idx.shape, C].  Other out-of-range indices give zeros and set
    PC_ERR_INVALID_ARGUMENT in the device status word.
    """
    code = _code(table, "table")
    ts = table.shape
    if len(ts) not in (2, 3) or not table.is_contiguous():
        raise ValueError(f"table must be contiguous [V, C] or [B, V, C] (got {tuple(ts)})")
    index = table.get_device()
    pi = _lookup(idx, index)
    B, V, C, T, shape = _lookup_sizes(idx, ts)
    if out is None:
        out = torch.empty(shape, dtype=table.dtype, device=table.device)
    else:
        _same(out, "out", shape, table.dtype, index)
    _run("pc_embedding", lib().pc_embedding, index, table.data_ptr(), code, B, V, C, pi, T,
         float(scale), out.data_ptr())
    return out


def pc_embedding_backward(grad_out: torch.Tensor, idx: torch.Tensor, shape,
                          scale: float = 1.0) -> torch.Tensor:
    """Gradient of :func:`pc_embedding` with respect to the table, whose shape is
    ``shape`` ((V, C) or (B, V, C)): scale times the sum of the rows of grad_out
    [*idx.shape, C] that each row of the table went to, in the order of the
    tokens."""
    code = _code(grad_out, "grad_out")
    index = grad_out.get_device()
    shape = tuple(int(n) for n in shape)
    if len(shape) not in (2, 3):
        raise ValueError(f"shape must be (V, C) or (B, V, C) (got {shape})")
    pi = _lookup(idx, index)
    B, V, C, T, rows = _lookup_sizes(idx, shape)
    pg = _packed(grad_out, "grad_out", rows, grad_out.dtype, index)
    grad = torch.empty(shape, dtype=grad_out.dtype, device=grad_out.device)
    _run("pc_embedding_backward", lib().pc_embedding_backward, index, pg, code, B, V, C, pi, T,
         float(scale), grad.data_ptr())
    return grad


# --- differentiable forms -----------------------------------------------------------

# Group norm and the gated projection are differentiable once (as layer norm and
# attention): a second derivative raises.  The lookup's gradient is linear, and
# its own gradient is the lookup.

class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, groups, eps, activation, lengths):
        y, mean, rstd = pc_group_norm(x, groups, weight, bias, eps, activation=activation,
                                      lengths=lengths, return_stats=True)
        ctx.save_for_backward(x, weight, bias, mean, rstd, lengths)
        ctx.groups, ctx.activation = groups, activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, weight, bias, mean, rstd, lengths = ctx.saved_tensors
        need_x, need_weight, need_bias = ctx.needs_input_grad[:3]
        dx, dw, db = pc_group_norm_backward(g.contiguous(), x, mean, rstd, ctx.groups, weight,
                                            bias, activation=ctx.activation, lengths=lengths,
                                            need_x=need_x, need_weight=need_weight,
                                            need_bias=need_bias)
        return dx, dw, db, None, None, None, None


def group_norm(x: torch.Tensor, groups: int, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, eps: float = 1e-5, *,
               activation: str | None = None,
               lengths: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable :func:`pc_group_norm` (x, weight and bias; once)."""
    return _GroupNorm.apply(x.contiguous(), weight, bias, groups, eps, activation, lengths)


class _GatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, b_gate, b_up, activation):
        ctx.save_for_backward(x, w_gate, w_up, b_gate, b_up)
        ctx.activation = activation
        return pc_gated_linear(x, w_gate, w_up, b_gate, b_up, activation=activation)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, w_gate, w_up, b_gate, b_up = ctx.saved_tensors
        need = ctx.needs_input_grad
        grads = pc_gated_linear_backward(g.contiguous(), x, w_gate, w_up, b_gate, b_up,
                                         activation=ctx.activation, need_x=need[0],
                                         need_weight=need[1] or need[2],
                                         need_bias=need[3] or need[4])
        return (*grads, None)


def gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                 b_gate: torch.Tensor | None = None, b_up: torch.Tensor | None = None, *,
                 activation: str | None = "silu") -> torch.Tensor:
    """Differentiable :func:`pc_gated_linear` (x, weights and biases; once).  The
    weights may be halves of one array (``w.chunk(2)``)."""
    return _GatedLinear.apply(x.contiguous(), w_gate.contiguous(), w_up.contiguous(), b_gate,
                              b_up, activation)


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, idx, scale):
        ctx.save_for_backward(idx)
        ctx.shape, ctx.scale = tuple(table.shape), scale
        return pc_embedding(table, idx, scale)

    @staticmethod
    def backward(ctx, g):
        idx, = ctx.saved_tensors
        return _EmbeddingGrad.apply(g.contiguous(), idx, ctx.shape, ctx.scale), None, None


class _EmbeddingGrad(torch.autograd.Function):
    @staticmethod
    def forward(ctx, g, idx, shape, scale):
        ctx.save_for_backward(idx)
        ctx.scale = scale
        return pc_embedding_backward(g, idx, shape, scale)

    @staticmethod
    def backward(ctx, gg):
        idx, = ctx.saved_tensors
        return _Embedding.apply(gg.contiguous(), idx, ctx.scale), None, None, None


def embedding(table: torch.Tensor, idx: torch.Tensor, scale: float = 1.0) -> torch.Tensor:
    """Differentiable :func:`pc_embedding` (the table; any number of times)."""
    return _Embedding.apply(table.contiguous(), idx.contiguous(), scale)
