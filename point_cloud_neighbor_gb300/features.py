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
    code = _ACTIVATIONS.get(name) if name is None or isinstance(name, str) else None
    if code is None:
        raise ValueError("activation must be one of 'none', 'silu', 'gelu', 'relu', 'sigmoid' "
                         f"(got {name!r})")
    return code


# --- group norm -------------------------------------------------------------------

def _group_args(x, groups, weight, bias, activation, lengths):
    code = _code(x, "x")
    if x.dim() != 3 or not x.is_contiguous():
        raise ValueError(f"x must be contiguous [B, L, C] (got {tuple(x.shape)})")
    B, L, C = x.shape
    index, pt = x.get_device(), None
    groups = int(groups)
    if groups < 1 or C % groups:
        raise ValueError(f"groups={groups} must divide the {C} channels")
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
    if lengths is not None:
        _check_lengths(lengths, B, x.device, "lengths")
    return (code, index, B, L, C, groups, PC_F32 if pt is None else _DTYPES[pt],
            _activation(activation))


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
    code, index, B, L, C, groups, pcode, act = _group_args(x, groups, weight, bias, activation,
                                                           lengths)
    if out is None:
        out = torch.empty_like(x)
    else:
        _same(out, "out", x.shape, x.dtype, index)
    mean = rstd = None
    if return_stats:
        mean = torch.empty((B, groups), dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    _run("pc_group_norm", lib().pc_group_norm, index, x.data_ptr(), code, B, L, C, groups,
         _ptr_or_none(weight), _ptr_or_none(bias), pcode, float(eps), act,
         _ptr_or_none(lengths), out.data_ptr(), _ptr_or_none(mean), _ptr_or_none(rstd))
    return (out, mean, rstd) if return_stats else out


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
    code, index, B, L, C, groups, pcode, act = _group_args(x, groups, weight, bias, activation,
                                                           lengths)
    _same(grad_out, "grad_out", x.shape, x.dtype, index)
    _same(mean, "mean", (B, groups), torch.float32, index)
    _same(rstd, "rstd", (B, groups), torch.float32, index)
    dx = torch.empty_like(x) if need_x else None
    dw = torch.empty_like(weight) if weight is not None and need_weight else None
    db = torch.empty_like(bias) if bias is not None and need_bias else None
    _run("pc_group_norm_backward", lib().pc_group_norm_backward, index, grad_out.data_ptr(),
         x.data_ptr(), code, B, L, C, groups, mean.data_ptr(), rstd.data_ptr(),
         _ptr_or_none(weight), _ptr_or_none(bias), pcode, act, _ptr_or_none(lengths),
         _ptr_or_none(dx), _ptr_or_none(dw), _ptr_or_none(db))
    return dx, dw, db


# --- gated projection ---------------------------------------------------------------

def _gated_args(x, w_gate, w_up, b_gate, b_up, activation):
    code = _code(x, "x")
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError("x must be contiguous with at least one axis")
    C, index, dtype = x.shape[-1], x.get_device(), x.dtype
    if not isinstance(w_gate, torch.Tensor) or w_gate.dim() != 2 or w_gate.shape[1] != C:
        raise ValueError(f"w_gate must be a {dtype} CUDA tensor [F, {C}]")
    F = w_gate.shape[0]
    _same(w_gate, "w_gate", (F, C), dtype, index)
    _same(w_up, "w_up", (F, C), dtype, index)
    if (b_gate is None) != (b_up is None):
        raise ValueError("b_gate and b_up go together")
    if b_gate is not None:
        _same(b_gate, "b_gate", (F,), dtype, index)
        _same(b_up, "b_up", (F,), dtype, index)
    rows = 1
    for n in x.shape[:-1]:
        rows *= n
    return index, (x.data_ptr(), code, rows, C, F, w_gate.data_ptr(), w_up.data_ptr(),
                   _ptr_or_none(b_gate), _ptr_or_none(b_up), _activation(activation)), F


PC_GATED_GRAD_X, PC_GATED_GRAD_WEIGHT, PC_GATED_GRAD_BIAS = 1, 2, 4


def _workspace(x, rows: int, C: int, F: int, gradients: int, index: int):
    """Scratch of a large call from torch's allocator, which keeps it (the library's
    pool does for smaller ones)."""
    if rows * (C + 2 * F) < 1 << 24:
        return None, 0
    with torch.cuda.device(index):
        n = lib().pc_gated_linear_workspace_bytes(_DTYPES[x.dtype], rows, C, F, gradients)
    return (torch.empty(n, dtype=torch.uint8, device=x.device), n) if n else (None, 0)


def pc_gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                    b_gate: torch.Tensor | None = None, b_up: torch.Tensor | None = None, *,
                    activation: str | None = "silu",
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """act(x w_gate^T + b_gate) * (x w_up^T + b_up): the first half of a gated
    feed-forward block.  x [..., C]; w_gate and w_up [F, C], as in a linear
    layer; b_gate and b_up [F], both or neither; all of one dtype.  Returns
    [..., F]."""
    index, args, F = _gated_args(x, w_gate, w_up, b_gate, b_up, activation)
    shape = (*x.shape[:-1], F)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    else:
        _same(out, "out", shape, x.dtype, index)
    work, n = _workspace(x, *args[2:5], 0, index)
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
    of the forward call is needed but its arguments."""
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
    work, n = _workspace(x, *args[2:5], which, index) if which else (None, 0)
    _run("pc_gated_linear_backward", lib().pc_gated_linear_backward, index,
         grad_out.data_ptr(), *args, _ptr_or_none(dx), _ptr_or_none(dwg), _ptr_or_none(dwu),
         _ptr_or_none(dbg), _ptr_or_none(dbu), _ptr_or_none(work), n)
    return dx, dwg, dwu, dbg, dbu


# --- lookup -----------------------------------------------------------------------

def _lookup(idx, name: str, index: int):
    if not isinstance(idx, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if idx.dtype is not torch.int64 or not idx.is_cuda or idx.get_device() != index \
            or not idx.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int64 tensor on cuda:{index}")
    return idx


def _count(shape) -> int:
    n = 1
    for k in shape:
        n *= k
    return n


def pc_embedding(table: torch.Tensor, idx: torch.Tensor, scale: float = 1.0, *,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """scale * table[idx], zeros where idx = -1.

    table [V, C] with idx of any shape, or a table for each cloud [B, V, C]
    with idx [B, ...] (the neighbours that kNN or Ball Query found).  Returns
    [*idx.shape, C].  Other out-of-range indices give zeros and set
    PC_ERR_INVALID_ARGUMENT in the device status word.
    """
    code = _code(table, "table")
    if table.dim() not in (2, 3) or not table.is_contiguous():
        raise ValueError(f"table must be contiguous [V, C] or [B, V, C] "
                         f"(got {tuple(table.shape)})")
    index = table.get_device()
    _lookup(idx, "idx", index)
    B, T = 1, _count(idx.shape)
    if table.dim() == 3:
        B = table.shape[0]
        if idx.dim() < 1 or idx.shape[0] != B:
            raise ValueError(f"idx must have shape [{B}, ...] (got {tuple(idx.shape)})")
        T = _count(idx.shape[1:])
    V, C = table.shape[-2:]
    shape = (*idx.shape, C)
    if out is None:
        out = torch.empty(shape, dtype=table.dtype, device=table.device)
    else:
        _same(out, "out", shape, table.dtype, index)
    _run("pc_embedding", lib().pc_embedding, index, table.data_ptr(), code, B, V, C,
         idx.data_ptr(), T, float(scale), out.data_ptr())
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
    _lookup(idx, "idx", index)
    _same(grad_out, "grad_out", (*idx.shape, shape[-1]), grad_out.dtype, index)
    B, T = 1, _count(idx.shape)
    if len(shape) == 3:
        B = shape[0]
        if idx.dim() < 1 or idx.shape[0] != B:
            raise ValueError(f"idx must have shape [{B}, ...] (got {tuple(idx.shape)})")
        T = _count(idx.shape[1:])
    grad = torch.empty(shape, dtype=grad_out.dtype, device=grad_out.device)
    _run("pc_embedding_backward", lib().pc_embedding_backward, index, grad_out.data_ptr(), code,
         B, shape[-2], shape[-1], idx.data_ptr(), T, float(scale), grad.data_ptr())
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
