"""GPU checks of the operators over point features (group norm with an
activation, gated projection, lookup of rows) against plain implementations in
float64.

Tolerances are first-order error bounds of the float32 arithmetic, element by
element: u = 2^-24 a rounding (2 u where a sum is cut off instead of rounded), the
number of roundings of the longest chain times the sum of the magnitudes that
enter it, plus half a unit of the result's type.  In bfloat16 the gated
projection may round the gradients of its two projections to bfloat16 before
the products that take them: half a unit of each term.
"""
import math

import pytest
import torch

import point_cloud_neighbor_gb300 as pc

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a unit, at most
DTYPES = [torch.float32, torch.bfloat16]
ACTS = ["none", "silu", "gelu", "relu", "sigmoid"]
DEV = "cuda"


@pytest.fixture(autouse=True)
def clean_status():
    yield
    assert pc.pc_device_status(reset=True) == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def close(got, want, tol, what):
    """|got - want| <= tol element by element, and no NaN or infinity in got."""
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}"
    if got.numel() == 0:
        return
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    err = (got - want).abs()
    bad = err > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {got.numel()} off, worst "
                           f"{float((err / tol.clamp_min(1e-300)).max()):.3g} of the bound")


def act64(z, name):
    """act(z), act'(z) in float64."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp_min(0), (z > 0).double()
    if name == "gelu":
        c = torch.special.ndtr(z)
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    s = torch.special.expit(z)
    if name == "sigmoid":
        return s, s * (1 - s)
    return z * s, s * (1 + z * (1 - s))


def act_error(z, name, dtype):
    """The rounding of act(z) and of act'(z) themselves, absolute.  The functions' values are
    at most max(|z|, 1) and their derivatives at most 1.13; float32 takes functions of a few
    units each, bfloat16 the approximate ones: 2^-21 (|z| + 2) of the logistic function and
    2^-24 of the normal distribution's."""
    k = 16 * U if dtype is torch.float32 else 2.0 ** -21 * (z.abs() + 8)
    f, _ = act64(z, name)
    value = k * f.abs() + (2 * U * z.abs() if name == "gelu" else 0)
    return value + 1e-37, k * (1 + z.abs()) * (0 if name in ("none", "relu") else 1) + 1e-37


# --- gated projection -------------------------------------------------------------

def gated_reference(x, wg, wu, bg, bu, dy, act):
    """Results in float64 and their bounds for this dtype."""
    t = x.dtype
    x, wg, wu, dy = (v.double() for v in (x, wg, wu, dy))
    rows, C = x.shape
    F = wg.shape[0]
    a, u = x @ wg.T, x @ wu.T
    ax = x.abs()
    ea, eu = ax @ wg.abs().T, ax @ wu.abs().T
    if bg is not None:
        a, u = a + bg.double(), u + bu.double()
        ea, eu = ea + bg.double().abs(), eu + bu.double().abs()
    # a chain of C products and a few joins, each addition cut off; three-part products
    n = 2 * U * (C + 32)
    ea, eu = n * ea, n * eu
    f, df = act64(a, act)
    vf, vd = act_error(a, act, t)
    bend = 0.0 if act in ("none", "relu") else 1.2   # at least the second derivatives
    ef, ed = df.abs() * ea + bend * ea * ea + vf, bend * ea + vd
    H = HALF[t]
    y = f * u
    out = {"y": (y, ef * u.abs() + f.abs() * eu + ef * eu + (H + 2 * U) * y.abs())}
    da, du = dy * u * df, dy * f
    eda = dy.abs() * (u.abs() * ed + df.abs() * eu + ed * eu) + 4 * U * da.abs()
    edu = dy.abs() * ef + 4 * U * du.abs()
    part = H if t is torch.bfloat16 else 2 * U       # the gradients as operands of products
    eda, edu = eda + part * (da.abs() + eda), edu + part * (du.abs() + edu)
    dx = da @ wg + du @ wu
    mag = da.abs() @ wg.abs() + du.abs() @ wu.abs()
    out["dx"] = (dx, eda @ wg.abs() + edu @ wu.abs() + 2 * U * (2 * F + 64) * mag + H * dx.abs())
    for name, d, e in (("g", da, eda), ("u", du, edu)):
        w = d.T @ x
        out["dw" + name] = (w, e.T @ ax + 2 * U * (rows + 64) * (d.abs().T @ ax) + H * w.abs())
        s = d.sum(0)
        out["db" + name] = (s, e.sum(0) + 2 * U * (rows + 64) * d.abs().sum(0) + H * s.abs())
    return {k: (v, e + 1e-30) for k, (v, e) in out.items()}


def gated_inputs(g, rows, C, F, dtype, bias=True, s=1.2):
    x, dy = randn(g, rows, C, dtype=dtype), randn(g, rows, F, dtype=dtype)
    wg, wu = ((randn(g, F, C) * s / math.sqrt(C)).to(dtype) for _ in range(2))
    bg, bu = ((randn(g, F) * 0.3).to(dtype) if bias else None for _ in range(2))
    return x, wg, wu, bg, bu, dy


def gated_all(x, wg, wu, bg, bu, dy, act):
    y = pc.pc_gated_linear(x, wg, wu, bg, bu, activation=act)
    dx, dwg, dwu, dbg, dbu = pc.pc_gated_linear_backward(dy, x, wg, wu, bg, bu, activation=act)
    return {"y": y, "dx": dx, "dwg": dwg, "dwu": dwu, "dbg": dbg, "dbu": dbu}


SHAPES = [(1, 1, 1), (1, 16, 8), (2, 96, 40), (3, 7, 5), (4, 384, 1024), (5, 33, 65), (8, 64, 256),
          (9, 520, 72), (17, 40, 24), (32, 384, 1024), (33, 100, 36), (64, 2048, 512),
          (65, 64, 64), (127, 48, 200), (128, 64, 64), (129, 72, 130), (200, 384, 1024),
          (257, 515, 333), (1000, 40, 96), (1021, 129, 63), (2500, 64, 16), (4100, 16, 24),
          # sums over more than 16,384 rows and hidden units; the most channels
          (40000, 16, 24), (3, 40, 9000), (5, 16384, 8), (300, 33, 65536)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_gated_linear(shape, dtype):
    rows, C, F = shape
    act = ("silu", "gelu", "sigmoid", "none")[(rows + C) % 4]
    ins = gated_inputs(gen(rows * 7 + C), rows, C, F, dtype, bias=(rows + F) % 3 != 0)
    got = gated_all(*ins, act)
    for name, (want, tol) in gated_reference(*ins, act).items():
        if got[name] is not None:
            close(got[name], want, tol, f"{name} {act}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [3, 70, 300])
def test_gated_linear_activations(rows, act, dtype):
    ins = list(gated_inputs(gen(5), rows, 80, 96, dtype))
    if act == "relu":
        # whole numbers, so that a is exact and relu's step falls where the definition has it
        ins[:5] = [t.mul(2).round().clamp(-2, 2) if t is ins[0] else t.sign() for t in ins[:5]]
    else:
        ins[0] = ins[0] * 4   # the functions' far ends
    got = gated_all(*ins, act)
    for name, (want, tol) in gated_reference(*ins, act).items():
        close(got[name], want, tol, f"{name} {act}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(300, 384, 512), (4099, 64, 80), (40, 777, 1000), (6, 500, 900)])
def test_gated_linear_error_in_norm(shape, dtype):
    """The error against float64, in norm, is at most 1.5 times that of the same formula in
    float32 torch, rounded once (the rounding of the two gradients to bfloat16 alone: 1.42)."""
    rows, C, F = shape
    ins = gated_inputs(gen(11), rows, C, F, dtype)
    got = gated_all(*ins, "silu")
    want = gated_reference(*ins, "silu")
    x, wg, wu, bg, bu, dy = (t.float() for t in ins)
    a, u = x @ wg.T + bg, x @ wu.T + bu
    s = torch.sigmoid(a)
    da, du = dy * u * s * (1 + a * (1 - s)), dy * a * s
    plain = {"y": a * s * u, "dx": da @ wg + du @ wu, "dwg": da.T @ x, "dwu": du.T @ x,
             "dbg": da.sum(0), "dbu": du.sum(0)}
    for name, p in plain.items():
        w = want[name][0]
        e = float((got[name].double() - w).norm() / w.norm())
        r = float((p.to(dtype).double() - w).norm() / w.norm())
        assert e <= max(1.5 * r, 1e-6), f"{name}: {e:.3g} against {r:.3g}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [2, 150])
def test_gated_linear_at_odd_addresses_is_the_same(rows, dtype):
    g = gen(3)

    def moved(t):
        if t is None:
            return None
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:]
        return flat.copy_(t.reshape(-1)).view(t.shape)
    ins = gated_inputs(g, rows, 64, 88, dtype)
    want, got = gated_all(*ins, "silu"), gated_all(*(moved(t) for t in ins), "silu")
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_linear_gradients_of_some(dtype):
    ins = gated_inputs(gen(4), 140, 72, 56, dtype)
    x, wg, wu, bg, bu, dy = ins
    full = pc.pc_gated_linear_backward(dy, x, wg, wu, bg, bu)
    for need in ({"need_x": False}, {"need_weight": False}, {"need_bias": False},
                 {"need_x": False, "need_bias": False}, {"need_x": False, "need_weight": False},
                 {"need_weight": False, "need_bias": False},
                 {"need_x": False, "need_weight": False, "need_bias": False}):
        some = pc.pc_gated_linear_backward(dy, x, wg, wu, bg, bu, **need)
        kept = [need.get(n, True) for n in ("need_x", "need_weight", "need_weight", "need_bias",
                                            "need_bias")]
        for f, s, k in zip(full, some, kept):
            assert (s is not None) == k
            assert s is None or torch.equal(f, s)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_linear_in_a_caller_s_workspace(dtype):
    """The C ABI with and without a workspace, and the sizes it asks for."""
    from point_cloud_neighbor_gb300.binding import lib
    L = lib()
    for shape in ((300, 128, 200), (70, 33, 41)):
        ins = x, wg, wu, bg, bu, dy = gated_inputs(gen(8), *shape, dtype)
        want = gated_all(*ins, "silu")
        code = 0 if dtype is torch.float32 else 1
        outs = {k: torch.full_like(v, math.nan) for k, v in want.items()}
        n = L.pc_gated_linear_workspace_bytes(code, *shape, 7)
        assert n > 4 * shape[0] * shape[2]
        work = torch.empty(n + 256, dtype=torch.uint8, device=DEV)
        work[n:] = 77
        s = torch.cuda.current_stream().cuda_stream
        args = [x.data_ptr(), code, *shape, wg.data_ptr(), wu.data_ptr(), bg.data_ptr(),
                bu.data_ptr(), 1]
        m = L.pc_gated_linear_workspace_bytes(code, *shape, 0)
        assert (m == 0) == (dtype is torch.bfloat16 and shape[1] % 8 == 0)
        assert L.pc_gated_linear(*args, outs["y"].data_ptr(), work.data_ptr() if m else None, m,
                                 s) == 0
        grads = [outs[k].data_ptr() for k in ("dx", "dwg", "dwu", "dbg", "dbu")]
        for bytes_ in (n, n - 1, 0):   # too small: the library's own
            assert L.pc_gated_linear_backward(dy.data_ptr(), *args, *grads, work.data_ptr(),
                                              bytes_, s) == 0
            for k in want:
                assert torch.equal(outs[k], want[k]), k
                if k != "y":
                    outs[k].fill_(math.nan)
        assert (work[n:] == 77).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_linear_empty(dtype):
    g = gen(1)
    x, wg, wu, bg, bu, dy = gated_inputs(g, 0, 24, 40, dtype)
    assert pc.pc_gated_linear(x, wg, wu, bg, bu).shape == (0, 40)
    for t in pc.pc_gated_linear_backward(dy, x, wg, wu, bg, bu):
        assert not t.any()
    x, wg, wu, bg, bu, dy = gated_inputs(g, 5, 24, 0, dtype, s=0.0)
    assert pc.pc_gated_linear(x, wg, wu, bg, bu).shape == (5, 0)
    assert not pc.pc_gated_linear_backward(dy, x, wg, wu, bg, bu)[0].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_gated_linear_keeps_bad_rows_apart(rows, bad, dtype):
    ins = gated_inputs(gen(2), rows, 64, 72, dtype)
    x, wg, wu, bg, bu, dy = ins
    good = gated_all(*ins, "silu")
    xb = x.clone()
    xb[1, 5] = bad
    got = gated_all(xb, wg, wu, bg, bu, dy, "silu")
    keep = torch.arange(rows, device=DEV) != 1
    for name in ("y", "dx"):
        assert torch.equal(got[name][keep], good[name][keep])
        assert not torch.isfinite(got[name][1]).all()
    if math.isnan(bad):
        assert got["y"][1].isnan().all() and got["dwg"].isnan().all()
        assert got["dbg"].isnan().all()


# --- group norm -----------------------------------------------------------------

def gn_reference(x, G, w, b, eps, act, lengths, dy):
    t = x.dtype
    B, L, C = x.shape
    cg = C // G
    n = torch.full((B,), L, device=DEV) if lengths is None else lengths.clamp(0, L)
    keep = (torch.arange(L, device=DEV) < n[:, None])[:, :, None, None]
    x = torch.where(keep, x.double().view(B, L, G, cg), 0.0)
    w = (torch.ones(C, device=DEV) if w is None else w).double().view(G, cg)
    b = (torch.zeros(C, device=DEV) if b is None else b).double().view(G, cg)
    N = (n * cg).clamp_min(1).double()[:, None, None, None]

    def mean(v):
        return torch.where(keep, v, 0.0).sum((1, 3), keepdim=True) / N
    m = mean(x)
    rs = torch.where(n[:, None, None, None] > 0, 1 / (mean((x - m) ** 2) + eps).sqrt(), 0.0)
    xh = torch.where(keep, (x - m) * rs, 0.0)
    z = xh * w + b
    f, df = act64(z, act)
    # as for layer norm: the statistics' own roundings (a chain of 256 at most: the rows of a
    # thread, joins of threads, warps and blocks), and those of x around them
    K = 256 * U
    a = mean(x.abs())
    rel = 2 * K + 8 * U * a * rs + (K * a * rs) ** 2
    exh = rel * xh.abs() + 2 * K * a * rs + 4 * U * x.abs() * rs
    ez = w.abs() * exh + 4 * U * (w * xh).abs() + 2 * U * b.abs()
    vf, vd = act_error(z, act, t)
    bend = 0.0 if act in ("none", "relu") else 1.2
    ef, ed = df.abs() * ez + bend * ez * ez + vf, bend * ez + vd
    H = HALF[t]
    out = {"mean": (m.view(B, G), (K * a).view(B, G)), "rstd": (rs.view(B, G), (rel * rs).view(B, G)),
           "y": (torch.where(keep, f, 0.0).view(B, L, C), torch.where(keep, ef + H * f.abs(), 0.0).view(B, L, C))}
    d = torch.where(keep, dy.double().view(B, L, G, cg) * df, 0.0)
    e_d = torch.where(keep, dy.double().view(B, L, G, cg).abs() * ed, 0.0) + 2 * U * d.abs()
    g, eg = d * w, e_d * w.abs() + 2 * U * (d * w).abs()
    m1, m2 = mean(g), mean(g * xh)
    k1 = 64 * U + 2 * U * (n.max() * B)   # sums over rows and clouds: at most as many roundings
    k1 = torch.minimum(k1.double(), torch.tensor(4096 * U, device=DEV, dtype=torch.float64))
    em1 = mean(eg) + k1 * mean(g.abs())
    em2 = mean(eg * xh.abs() + g.abs() * exh) + k1 * mean((g * xh).abs())
    dx = rs * (g - m1 - xh * m2)
    edx = rs * (eg + em1 + xh.abs() * em2 + exh * m2.abs()
                + 4 * U * (g.abs() + m1.abs() + (xh * m2).abs())) + rel * dx.abs() + H * dx.abs()
    out["dx"] = (torch.where(keep, dx, 0.0).view(B, L, C), torch.where(keep, edx, 0.0).view(B, L, C))
    out["dw"] = ((d * xh).sum((0, 1)).view(C),
                 (e_d * xh.abs() + d.abs() * exh + k1 * (d * xh).abs()).sum((0, 1)).view(C))
    out["db"] = (d.sum((0, 1)).view(C), (e_d + k1 * d.abs()).sum((0, 1)).view(C))
    return {k: (v, e + 1e-30) for k, (v, e) in out.items()}


def gn_all(x, G, w, b, act, lengths, dy, eps=1e-5):
    y, mean, rstd = pc.pc_group_norm(x, G, w, b, eps, activation=act, lengths=lengths,
                                     return_stats=True)
    assert torch.equal(y, pc.pc_group_norm(x, G, w, b, eps, activation=act, lengths=lengths))
    dx, dw, db = pc.pc_group_norm_backward(dy, x, mean, rstd, G, w, b, activation=act,
                                           lengths=lengths)
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dw": dw, "db": db}


GN_SHAPES = [(1, 1, 2, 1), (1, 1, 64, 2), (2, 3, 6, 3), (1, 64, 384, 32), (3, 17, 96, 32),
             (5, 100, 48, 4), (2, 333, 195, 13), (2, 50, 515, 5), (1, 1000, 2048, 1),
             (2, 40, 2048, 32), (1, 30, 4104, 3), (1, 9, 16384, 1), (1, 20, 2310, 2),
             (2, 11, 1021, 1), (40, 7, 32, 8), (1, 5000, 64, 8), (1, 20000, 24, 2),
             (300, 2, 16, 4), (7, 257, 12, 4), (16, 1024, 128, 32), (1, 60000, 40, 4),
             (2, 30011, 35, 7), (3, 4093, 195, 13), (1, 2048, 384, 32), (2, 9000, 64, 1)]


@pytest.mark.parametrize("dtype,pdtype", [(torch.float32, torch.float32),
                                          (torch.bfloat16, torch.float32),
                                          (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("shape", GN_SHAPES)
def test_group_norm(shape, dtype, pdtype):
    B, L, C, G = shape
    g = gen(B + L + C)
    act = ("silu", "gelu", "sigmoid", "none")[(L + C) % 4]
    x = (randn(g, B, L, C) * 2 + randn(g, C)).to(dtype)
    w, b, dy = (randn(g, C) + 1).to(pdtype), randn(g, C).to(pdtype), randn(g, B, L, C, dtype=dtype)
    got = gn_all(x, G, w, b, act, None, dy)
    for name, (want, tol) in gn_reference(x, G, w, b, 1e-5, act, None, dy).items():
        if name in ("dw", "db"):
            tol = tol + HALF[pdtype] * want.abs()
        close(got[name], want, tol, f"{name} {act}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
def test_group_norm_ragged_with_bad_padding(act, dtype):
    """Lengths of all kinds; what lies past them is NaN or infinite and enters nothing."""
    g = gen(9)
    B, L, C, G = 7, 150, 40, 5
    x, dy = randn(g, B, L, C, dtype=dtype), randn(g, B, L, C, dtype=dtype)
    w, b = randn(g, C) + 1, randn(g, C)
    n = torch.tensor([150, 0, 1, 149, 64, -3, 999], device=DEV)
    if act == "relu":
        b = b.abs() + 20   # away from the step
    r = gn_reference(x, G, w, b, 1e-5, act, n, dy)
    past = (torch.arange(L, device=DEV) >= n[:, None])[..., None]
    x = torch.where(past, math.nan, x)
    dy = torch.where(past, math.inf, dy)
    got = gn_all(x, G, w, b, act, n, dy)
    for name, (want, tol) in r.items():
        close(got[name], want, tol, f"{name} {act}")
    assert not got["y"].masked_select(past).any() and not got["dx"].masked_select(past).any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_group_norm_without_parameters_and_gradients_of_some(dtype):
    g = gen(2)
    x, dy = randn(g, 3, 70, 48, dtype=dtype), randn(g, 3, 70, 48, dtype=dtype)
    y, m, r = pc.pc_group_norm(x, 6, activation="silu", return_stats=True)
    one, zero = torch.ones(48, device=DEV), torch.zeros(48, device=DEV)
    assert torch.equal(y, pc.pc_group_norm(x, 6, one, zero, activation="silu"))
    dx, dw, db = pc.pc_group_norm_backward(dy, x, m, r, 6, activation="silu")
    assert dw is None and db is None
    full = pc.pc_group_norm_backward(dy, x, m, r, 6, one, zero, activation="silu")
    assert torch.equal(dx, full[0])
    for need in ({"need_x": False}, {"need_weight": False}, {"need_bias": False},
                 {"need_weight": False, "need_bias": False},
                 {"need_x": False, "need_weight": False}):
        some = pc.pc_group_norm_backward(dy, x, m, r, 6, one, zero, activation="silu", **need)
        for f, s, k in zip(full, some, ("need_x", "need_weight", "need_bias")):
            assert (s is not None) == need.get(k, True)
            assert s is None or torch.equal(f, s)


def test_group_norm_of_large_means_outliers_and_constants():
    g = gen(4)
    # a mean of 1e4 deviations; a first point far off; constant groups
    x = randn(g, 2, 3000, 32) + 1e4
    x[1] = randn(g, 3000, 32)
    x[1, 0] = 1e4
    dy = randn(g, 2, 3000, 32)
    one, zero = torch.ones(32, device=DEV), torch.zeros(32, device=DEV)
    got = gn_all(x, 4, one, zero, "none", None, dy)
    for name, (want, tol) in gn_reference(x, 4, one, zero, 1e-5, "none", None, dy).items():
        close(got[name], want, tol, name)
    c = torch.full((1, 100, 8), 3.0, device=DEV)
    y, m, r = pc.pc_group_norm(c, 2, return_stats=True)
    assert not y.any() and (m == 3).all()
    close(r, torch.full_like(r, 1e-5).double() ** -0.5, torch.full_like(r, 1e-4).double(), "rstd")


@pytest.mark.parametrize("dtype", DTYPES)
def test_group_norm_at_odd_addresses(dtype):
    g = gen(6)
    x, dy = randn(g, 3, 90, 64, dtype=dtype), randn(g, 3, 90, 64, dtype=dtype)
    w, b = randn(g, 64), randn(g, 64)

    def moved(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].copy_(
            t.reshape(-1)).view(t.shape)
    got = gn_all(moved(x), 8, w, b, "silu", None, moved(dy))
    for name, (want, tol) in gn_reference(x, 8, w, b, 1e-5, "silu", None, dy).items():
        close(got[name], want, tol, name)


def test_group_norm_empty():
    w = torch.ones(8, device=DEV)
    for shape in ((0, 5, 8), (2, 0, 8)):
        x = torch.zeros(shape, device=DEV)
        y, m, r = pc.pc_group_norm(x, 2, w, w, return_stats=True)
        assert y.shape == shape and not m.any() and not r.any()
        dx, dw, db = pc.pc_group_norm_backward(y, x, m, r, 2, w, w)
        assert dx.shape == shape and not dw.any() and not db.any()


def test_group_norm_nan_stays_in_its_group():
    x = randn(gen(8), 2, 300, 16)
    good = pc.pc_group_norm(x, 4)
    x[0, 7, 5] = math.nan
    y = pc.pc_group_norm(x, 4)
    assert y[0, :, 4:8].isnan().all()
    y[0, :, 4:8] = good[0, :, 4:8]
    assert torch.equal(y, good)


# --- lookup -----------------------------------------------------------------------

def emb_reference(dy, idx, shape, scale):
    """Sums in float64, sums of magnitudes, counts."""
    B, V, C = shape if len(shape) == 3 else (1, *shape)
    idx = idx.reshape(B, -1)
    at = (idx + V * torch.arange(B, device=DEV)[:, None]).reshape(-1)
    ok = ((idx >= 0) & (idx < V)).reshape(-1)
    d = dy.double().reshape(-1, C)
    s, m = (torch.zeros(B * V, C, dtype=torch.float64, device=DEV) for _ in range(2))
    s.index_add_(0, at[ok], d[ok])
    m.index_add_(0, at[ok], d[ok].abs())
    return (s * scale).view(shape), (m * abs(scale)).view(shape)


EMB = [((1, 1), (1,)), ((7, 3), (5,)), ((40, 384), (512,)), ((100, 33), (1000,)),
       ((1000, 8), (4097,)), ((3, 16), (20000,)), ((1, 72), (9001,)), ((300, 515), (64, 3)),
       ((70000, 4), (3000,)), ((5, 24), (0,)), ((4, 64, 40), (4, 30, 9)), ((3, 1000, 64), (3, 2000)),
       ((33, 5, 7), (33, 1)), ((2, 1, 130), (2, 4200)), ((65535, 16), (300,)), ((65536, 2), (5000,)),
       ((511, 8), (700,)), ((512, 8), (700,)), ((300000, 4), (5000,)), ((9, 24), (200000,)),
       ((50, 2050), (900,))]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,tokens", EMB)
def test_embedding(shape, tokens, dtype):
    g = gen(sum(shape))
    V, C = shape[-2:]
    table = randn(g, *shape, dtype=dtype)
    u = torch.rand(tokens, generator=g, device=DEV)
    idx = (u * u * V).long().clamp_max(V - 1)      # low rows are frequent
    idx[torch.rand(tokens, generator=g, device=DEV) < 0.1] = -1
    scale = 1.7
    y = pc.pc_embedding(table, idx, scale)
    flat = table.reshape(-1, C)
    at = idx.clamp_min(0)
    if len(shape) == 3:
        at = at + (V * torch.arange(shape[0], device=DEV)).view(-1, *[1] * (len(tokens) - 1))
    want = (flat[at].float() * scale).to(dtype)
    assert torch.equal(y, torch.where(idx[..., None] >= 0, want, torch.zeros_like(want)))
    dy = randn(g, *tokens, C, dtype=dtype)
    d = pc.pc_embedding_backward(dy, idx, shape, scale)
    s, m = emb_reference(dy, idx, shape, scale)
    # a run of at most 64 tokens, up to 64 runs, sums of 64 runs, the ends: each at most 64 + 5
    close(d, s, (5 * 70 * U) * m + HALF[dtype] * s.abs() + 1e-30, "grad_table")
    assert torch.equal(d, pc.pc_embedding_backward(dy, idx, shape, scale))


def test_embedding_adds_in_the_order_of_the_tokens():
    """The float32 sums of a row's tokens one after the other, in runs that end at every 16th
    of the sorted tokens (a small call), and the runs one after the other."""
    g = gen(12)
    idx = torch.randint(0, 300, (5000,), generator=g, device=DEV)
    dy = randn(g, 5000, 6)
    d = pc.pc_embedding_backward(dy, idx, (300, 6))
    order = torch.sort(idx, stable=True)[1].cpu()
    rows, dy = idx.cpu(), dy.cpu()
    runs = {}
    for at, i in enumerate(order.tolist()):
        runs.setdefault(int(rows[i]), {}).setdefault(at // 16, []).append(dy[i])
    want = torch.zeros(300, 6)
    for row, parts in runs.items():
        sums = []
        for part in parts.values():
            s = torch.zeros(6)
            for v in part:
                s = s + v
            sums.append(s)
        want[row] = sums[0]
        for s in sums[1:]:
            want[row] += s
    assert torch.equal(d.cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_embedding_of_out_of_range_indices(dtype):
    table = randn(gen(1), 10, 24, dtype=dtype)
    idx = torch.tensor([3, -1, 10, -2, 2 ** 40, 9], device=DEV)
    y = pc.pc_embedding(table, idx)
    assert pc.pc_device_status(reset=True) == 1
    assert not y[1:5].any() and torch.equal(y[0], table[3]) and torch.equal(y[5], table[9])
    d = pc.pc_embedding_backward(torch.ones_like(y), idx, (10, 24))
    assert pc.pc_device_status(reset=True) == 1
    assert d.sum() == 48 and (d[3] == 1).all() and (d[9] == 1).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_embedding_keeps_bad_values_in_their_rows(dtype):
    g = gen(3)
    idx = torch.randint(0, 5, (2000,), generator=g, device=DEV)
    idx[:10] = -1
    dy = randn(g, 2000, 16, dtype=dtype)
    want = pc.pc_embedding_backward(dy, idx, (5, 16))
    dy[:10] = math.nan                                   # of absent tokens
    assert torch.equal(pc.pc_embedding_backward(dy, idx, (5, 16)), want)
    dy[int((idx == 2).nonzero()[0])] = math.inf
    d = pc.pc_embedding_backward(dy, idx, (5, 16))
    assert (d[2] == math.inf).all()
    d[2] = want[2]
    assert torch.equal(d, want)


def test_embedding_long_sum_of_one_row():
    T = 600_000
    dy = 1.0 + 0.25 * torch.rand(T, 4, generator=gen(5), device=DEV)
    d = pc.pc_embedding_backward(dy, torch.zeros(T, dtype=torch.int64, device=DEV), (3, 4))
    s, m = emb_reference(dy, torch.zeros(T, dtype=torch.int64, device=DEV), (3, 4), 1.0)
    close(d, s, (5 * 70 + 600) * U * m + 1e-30, "grad_table")   # 586 sums of 64 runs of 16
    assert not d[1:].any()


# --- beyond 32 bits ------------------------------------------------------------------

def test_embedding_beyond_32_bits():
    """Rows whose offset in the table is beyond 2^31 elements; keys of 28 bits."""
    V, C = (1 << 21) + 3, 1024
    table = torch.zeros(V, C, dtype=torch.bfloat16, device=DEV)
    idx = torch.tensor([V - 1, 5, V - 2, V - 1, -1], device=DEV)
    table[V - 1], table[V - 2], table[5] = 3.0, 2.0, 1.0
    y = pc.pc_embedding(table, idx)
    assert y[:, 0].tolist() == [3, 1, 2, 3, 0] and torch.equal(y, y[:, :1].expand_as(y))
    d = pc.pc_embedding_backward(y, idx, (V, C))
    assert (d[V - 1] == 6).all() and (d[V - 2] == 2).all() and (d[5] == 1).all()
    d[V - 1], d[V - 2], d[5] = 0, 0, 0
    assert not d.any()
    del table, d
    V = (1 << 27) + 9
    idx = torch.tensor([V - 1, 0, 1 << 27, V - 1], device=DEV)
    d = pc.pc_embedding_backward(torch.ones(4, 1, device=DEV), idx, (V, 1))
    assert d[V - 1] == 2 and d[0] == 1 and d[1 << 27] == 1 and d.sum() == 4


def test_group_norm_beyond_32_bits():
    B, L, C = 3, 700_000, 1024
    x = torch.empty(B, L, C, dtype=torch.bfloat16, device=DEV)
    g = gen(1)
    x[2] = torch.randn(L, C, generator=g, device=DEV, dtype=torch.bfloat16)
    x[:2] = 1
    w = randn(g, C)
    y, m, r = pc.pc_group_norm(x, 32, w, w, activation="silu", return_stats=True)
    y1, m1, r1 = pc.pc_group_norm(x[2:], 32, w, w, activation="silu", return_stats=True)
    # (other shares of the rows: statistics off by a few roundings, results by one of bfloat16's)
    assert (r[2] / r1[0] - 1).abs().max() < 1e-5 and (m[2] - m1[0]).abs().max() < 1e-5
    for i in (0, L // 2, L - 100):
        a, b = y[2, i:i + 100].float(), y1[0, i:i + 100].float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-4).all()
    del y, y1
    dx, dw, _ = pc.pc_group_norm_backward(x, x, m, r, 32, w, w, activation="silu")
    dx1, dw1, _ = pc.pc_group_norm_backward(x[2:], x[2:], m[2:], r[2:], 32, w, w,
                                            activation="silu")
    for i in (0, L // 2, L - 100):
        a, b = dx[2, i:i + 100].float(), dx1[0, i:i + 100].float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-4).all()


def test_gated_linear_beyond_32_bits():
    rows, C, F = 2_200_000, 8, 1024
    g = gen(2)
    x = torch.randn(rows, C, generator=g, device=DEV, dtype=torch.bfloat16)
    wg, wu = (torch.randn(F, C, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    y = pc.pc_gated_linear(x, wg, wu)
    dx, dwg, dwu, _, _ = pc.pc_gated_linear_backward(y, x, wg, wu)
    ref = gated_reference(x[-1000:], wg, wu, None, None, y[-1000:], "silu")
    for name, got in (("y", y), ("dx", dx)):
        close(got[-1000:], *ref[name], name)
    a, u = x.double() @ wg.double()[:8].T, x.double() @ wu.double()[:8].T
    s = torch.sigmoid(a)
    want = (y[:, :8].double() * u * s * (1 + a * (1 - s))).T @ x.double()
    # one rounding of da and one of the result, 2^-9 each; the error of 2.2e6 terms of random sign
    assert float((dwg[:8].double() - want).norm() / want.norm()) < 2.0 ** -8


# --- autograd, streams, graphs, all together ------------------------------------------

def chain(idx, lengths, dtype):
    """Rows looked up, normalised over each cloud, projected: as a block runs them."""
    def f(table, w, b, wg, wu, bg, bu):
        t = pc.embedding(table, idx, 0.5)
        t = pc.group_norm(t, 4, w, b, activation="gelu", lengths=lengths)
        return pc.gated_linear(t, wg, wu, bg, bu)
    return f


def chain64(idx, lengths):
    def f(table, w, b, wg, wu, bg, bu):
        B, L = idx.shape
        t = torch.where(idx[..., None] >= 0, table[idx.clamp_min(0)] * 0.5, 0.0)
        keep = (torch.arange(L, device=DEV) < lengths[:, None])[..., None]
        C = t.shape[-1]
        v = torch.where(keep, t, 0.0).view(B, L, 4, C // 4)
        n = (lengths * (C // 4)).clamp_min(1).view(B, 1, 1, 1)
        m = v.sum((1, 3), keepdim=True) / n
        k4 = keep[..., None]
        c = torch.where(k4, v - m, 0.0)
        z = c / ((c * c).sum((1, 3), keepdim=True) / n + 1e-5).sqrt()
        z = (z.view(B, L, C) * w + b)
        h = torch.where(keep, torch.nn.functional.gelu(z), 0.0)
        return torch.nn.functional.silu(h @ wg.T + bg) * (h @ wu.T + bu)
    return f


def chain_inputs(dtype, seed=0):
    g = gen(seed)
    B, L, V, C, F = 3, 130, 50, 48, 72
    idx = torch.randint(-1, V, (B, L), generator=g, device=DEV)
    lengths = torch.tensor([130, 77, 0], device=DEV)
    wg, wu = ((randn(g, F, C) / 6).to(dtype) for _ in range(2))
    leaves = [randn(g, V, C, dtype=dtype), 1 + 0.2 * randn(g, C), 0.2 * randn(g, C), wg, wu,
              randn(g, F, dtype=dtype), randn(g, F, dtype=dtype)]
    return idx, lengths, leaves, randn(g, B, L, F, dtype=dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_chain_against_float64(dtype):
    """Forward and gradients through all three; in norm, each operator's result rounded once:
    three roundings forward and three back of at most half a unit each, which the products mix."""
    idx, lengths, leaves, dy = chain_inputs(dtype)
    a = [t.clone().requires_grad_() for t in leaves]
    y = chain(idx, lengths, dtype)(*a)
    y.backward(dy)
    b = [t.double().requires_grad_() for t in leaves]
    want = chain64(idx, lengths)(*b)
    want.backward(dy.double())
    tol = 1e-5 if dtype is torch.float32 else 8 * HALF[dtype]
    for name, got, ref in [("y", y, want)] + [(f"grad {i}", p.grad, q.grad)
                                              for i, (p, q) in enumerate(zip(a, b))]:
        e = float((got.detach().double() - ref.detach()).norm() / ref.detach().norm())
        assert e <= tol, f"{name}: {e:.3g}"


def test_gradients_against_differences():
    idx, lengths, leaves, dy = chain_inputs(torch.float32, 7)
    f, g = chain(idx, lengths, torch.float32), gen(70)
    a = [t.clone().requires_grad_() for t in leaves]
    (f(*a) * dy).sum().backward()
    for i, leaf in enumerate(leaves):
        v = randn(g, *leaf.shape)
        h = 1e-2 / float(v.norm() / math.sqrt(v.numel()))
        ends = []
        for s in (h, -h):
            moved = list(leaves)
            moved[i] = leaf + s * v
            ends.append(float((f(*moved).double() * dy).sum()))
        got, want = float((a[i].grad.double() * v).sum()), (ends[0] - ends[1]) / (2 * h)
        size = float((a[i].grad.double().norm() * v.double().norm()))
        # (third derivatives times h^2 / 6, and float32 in the two sums)
        assert abs(got - want) <= 2e-3 * size, f"leaf {i}: {got} against {want}"


def test_second_derivatives():
    g = gen(1)
    table = randn(g, 9, 4).requires_grad_()
    idx = torch.tensor([1, 1, 3, -1], device=DEV)
    y = pc.embedding(table, idx, 2.0)
    d, = torch.autograd.grad((y ** 2).sum(), table, create_graph=True)   # 2 * 2 * 2 table
    dd, = torch.autograd.grad((d ** 2).sum(), table)
    k = torch.zeros(9, 1, device=DEV)
    k[1], k[3] = 2, 1
    assert torch.equal(d.detach(), 8 * k * table.detach())
    assert torch.equal(dd, 128 * k * k * table.detach())
    x = randn(g, 2, 6, 8).requires_grad_()
    w = randn(g, 5, 8)
    for out in (pc.group_norm(x, 2), pc.gated_linear(x, w, w)):
        d, = torch.autograd.grad((out ** 2).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            d.sum().backward()


@pytest.mark.parametrize("dtype", DTYPES)
def test_views_strides_and_partial_gradients(dtype):
    g = gen(2)
    x = randn(g, 16, 3, 40, dtype=dtype).transpose(0, 1).requires_grad_()
    w = randn(g, 2 * 24, 40, dtype=dtype).requires_grad_()
    y = pc.gated_linear(x, *w.chunk(2))
    y.sum().backward()
    ref = pc.pc_gated_linear_backward(torch.ones_like(y).contiguous(),
                                      x.detach().contiguous(), *w.detach().chunk(2))
    assert torch.equal(x.grad, ref[0])
    assert torch.equal(w.grad, torch.cat([ref[1], ref[2]]))
    wu = w.detach()[24:].clone().requires_grad_()
    y = pc.gated_linear(x.detach(), w.detach()[:24], wu)
    y.sum().backward()
    assert torch.equal(wu.grad, ref[2])


@pytest.mark.parametrize("dtype", DTYPES)
def test_other_streams_and_graphs(dtype):
    idx, lengths, leaves, dy = chain_inputs(dtype, 3)
    table, w, b, wg, wu, bg, bu = leaves

    def step():
        t = pc.pc_embedding(table, idx, 0.5)
        h, m, r = pc.pc_group_norm(t, 4, w, b, activation="gelu", lengths=lengths,
                                   return_stats=True)
        y = pc.pc_gated_linear(h, wg, wu, bg, bu)
        dh, *dws = pc.pc_gated_linear_backward(dy, h, wg, wu, bg, bu)
        dt, dw, db = pc.pc_group_norm_backward(dh, t, m, r, 4, w, b, activation="gelu",
                                               lengths=lengths)
        return [y, dt, dw, db, *dws, pc.pc_embedding_backward(dt, idx, table.shape, 0.5)]
    want = step()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:   # several at once
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(step())
    torch.cuda.synchronize()
    for out in outs:
        for a, e in zip(out, want):
            assert torch.equal(a, e)
    graphs = []
    for _ in range(2):  # two graphs, replayed in turn and at once
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step()
        graphs.append((graph, res))
    old = table.clone()
    for k in range(3):
        table.copy_(old * (k + 1))
        fresh = step()
        for i, (graph, _) in enumerate(graphs):
            streams[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(streams[i]):
                graph.replay()
        torch.cuda.synchronize()
        for _, res in graphs:
            for a, e in zip(res, fresh):
                assert torch.equal(a, e)


@pytest.mark.parametrize("dtype", DTYPES)
def test_forms_captured_with_their_gradients(dtype):
    """A training step of the differentiable forms in a graph, captured without a run of
    these sizes before it; replayed on other values it gives what an eager step does."""
    idx, lengths, leaves, dy = chain_inputs(dtype, 11)
    leaves = [t.requires_grad_() for t in leaves]
    f = chain(idx, lengths, dtype)

    def step():
        y = f(*leaves)
        return [y.detach(), *torch.autograd.grad(y, leaves, dy)]
    pc.pc_embedding(leaves[0].detach(), idx)  # (the library knows the device)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in (1.0, -0.5, 2.0):
        with torch.no_grad():
            for t in (leaves[0], leaves[3], dy):
                t.mul_(k)
            idx.copy_(idx.roll(1, 0))
            lengths.copy_(lengths.roll(1))
        graph.replay()
        for a, e in zip(got, step()):
            assert torch.equal(a, e)


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_calls_at_once_on_streams(dtype):
    """Calls whose scratch comes from torch's allocator, in several streams at once."""
    rows, C, F = 33000, 64, 512
    assert rows * (C + 2 * F) >= pc.features.LARGE
    ins = [gated_inputs(gen(20 + i), rows, C, F, dtype) for i in range(2)]
    want = [gated_all(*x, "silu") for x in ins]
    streams, got = [torch.cuda.Stream() for _ in ins], []
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, x in zip(streams, ins):
            with torch.cuda.stream(s):
                got.append(gated_all(*x, "silu"))
    torch.cuda.synchronize()
    for a, e in zip(got, want):
        for k in e:
            assert torch.equal(a[k], e[k]), k


def test_results_do_not_change_from_run_to_run():
    for dtype in DTYPES:
        ins = gated_inputs(gen(1), 3000, 128, 256, dtype)
        first = gated_all(*ins, "silu")
        for _ in range(3):
            again = gated_all(*ins, "silu")
            for k in first:
                assert torch.equal(first[k], again[k]), k


def test_a_withheld_copy_ends_with_the_status_word():
    for dtype in DTYPES:
        ins = gated_inputs(gen(6), 700, 256, 320, dtype)
        want = gated_all(*ins, "silu")
        x, wg, wu, bg, bu, dy = ins
        torch.cuda.synchronize()
        try:
            pc.pc_set_wait_timeout_ns(50_000_000)
            pc.pc_debug_set_stall(pc.PC_STALL_GATED)
            pc.pc_gated_linear(x, wg, wu, bg, bu)
            assert pc.pc_device_status(reset=True) == 4
            pc.pc_gated_linear_backward(dy, x, wg, wu, bg, bu)
            assert pc.pc_device_status(reset=True) == 4
        finally:
            pc.pc_debug_set_stall(0)
            pc.pc_set_wait_timeout_ns(2_000_000_000)
        again = gated_all(*ins, "silu")
        assert all(torch.equal(want[k], again[k]) for k in want)


def test_a_withheld_copy_of_group_norm_ends_with_the_status_word():
    g = gen(6)
    x, dy, w = randn(g, 3, 2000, 64), randn(g, 3, 2000, 64), randn(g, 64)
    want = gn_all(x, 4, w, w, "silu", None, dy)
    torch.cuda.synchronize()
    try:
        pc.pc_set_wait_timeout_ns(50_000_000)
        pc.pc_debug_set_stall(pc.PC_STALL_GROUP_NORM)
        pc.pc_group_norm(x, 4, w, w)
        assert pc.pc_device_status(reset=True) == 4
        pc.pc_group_norm_backward(dy, x, want["mean"], want["rstd"], 4, w, w)
        assert pc.pc_device_status(reset=True) == 4
    finally:
        pc.pc_debug_set_stall(0)
        pc.pc_set_wait_timeout_ns(2_000_000_000)
    again = gn_all(x, 4, w, w, "silu", None, dy)
    assert all(torch.equal(want[k], again[k]) for k in want)


def test_refusals():
    g = gen(0)
    x, w = randn(g, 4, 16), randn(g, 8, 16)
    for call, what in [
            (lambda: pc.pc_gated_linear(x.half(), w, w), "float32 or bfloat16"),
            (lambda: pc.pc_gated_linear(x.t(), w, w), "contiguous"),
            (lambda: pc.pc_gated_linear(x, w.t(), w), "w_gate"),
            (lambda: pc.pc_gated_linear(x, w, w[:4]), "w_up"),
            (lambda: pc.pc_gated_linear(x, w, w.bfloat16()), "w_up"),
            (lambda: pc.pc_gated_linear(x, w, w, w[:, 0].contiguous()), "go together"),
            (lambda: pc.pc_gated_linear(x, w, w, activation="swish"), "activation"),
            (lambda: pc.pc_gated_linear(x, w, w, out=x), "out"),
            (lambda: pc.pc_gated_linear_backward(x, x, w, w), "grad_out"),
            (lambda: pc.pc_group_norm(x, 2), r"\[B, L, C\]"),
            (lambda: pc.pc_group_norm(x[None], 3), "divide"),
            (lambda: pc.pc_group_norm(x[None], 0), "divide"),
            (lambda: pc.pc_group_norm(x[None], 2, w[0].bfloat16()), "weight"),
            (lambda: pc.pc_group_norm(x[None], 2, activation="tanh"), "activation"),
            (lambda: pc.pc_group_norm(x[None], 2, lengths=torch.ones(2, dtype=torch.int64,
                                                                     device=DEV)), "lengths"),
            (lambda: pc.pc_group_norm(x[None], 2, eps=-1.0), "eps"),
            (lambda: pc.pc_embedding(x, torch.zeros(3, dtype=torch.int32, device=DEV)), "int64"),
            (lambda: pc.pc_embedding(x[None], torch.zeros(3, dtype=torch.int64, device=DEV)),
             "idx"),
            (lambda: pc.pc_embedding(x.t(), torch.zeros(3, dtype=torch.int64, device=DEV)),
             "contiguous"),
            (lambda: pc.pc_embedding(x, torch.zeros(3, dtype=torch.int64, device=DEV),
                                     math.inf), "scale"),
            (lambda: pc.pc_embedding_backward(x, torch.zeros(3, dtype=torch.int64, device=DEV),
                                              (5, 16)), "grad_out"),
            (lambda: pc.pc_embedding_backward(x, torch.zeros(4, dtype=torch.int64, device=DEV),
                                              (16,)), "shape")]:
        with pytest.raises((ValueError, pc.PointCloudError), match=what):
            call()


@pytest.mark.parametrize("shape", [(300, 304, 65536), (4096, 304, 4096)])
def test_gated_linear_takes_each_value_of_grad_out_once(shape):
    """Many tiles a block, each with its own part of grad_out, which is copied a tile ahead:
    with rows of an identity the weights' gradients are da and du themselves."""
    rows, C, F = shape
    g = gen(31)
    _, wg, wu, _, _, dy = gated_inputs(g, rows, C, F, torch.bfloat16, bias=False)
    x = torch.eye(rows, C, device=DEV, dtype=torch.bfloat16)
    n = min(rows, C)
    want = gated_reference(x[:n], wg, wu, None, None, dy[:n], "silu")
    for _ in range(4):
        dx, dwg, dwu, _, _ = pc.pc_gated_linear_backward(dy, x, wg, wu)
        close(dwg, *want["dwg"], "dwg")
        close(dwu, *want["dwu"], "dwu")
        close(dx[:n], *want["dx"], "dx")


@pytest.mark.parametrize("shape", [(300, 384, 512), (4099, 64, 80), (40, 777, 1000), (6, 500, 900),
                                   (2100, 136, 3000), (20000, 520, 264), (129, 72, 17)])
def test_gated_linear_gradients_are_rounded_once(shape):
    """bfloat16: da and du enter the products of grad_x and the weights' gradients as two
    bfloat16 parts (off by 2^-18), so that the error in norm is that of rounding the float64
    gradients once, and 2% for what else there is: the approximate silu and its derivative
    (2^-21 (|a| + 8), here at most 2^-17), the parts, and sums that are cut off (below 2^-15 of
    the sum of magnitudes, which is at most 30 times a sum of as many terms of random sign)."""
    rows, C, F = shape
    ins = x, wg, wu, bg, bu, dy = gated_inputs(gen(21), rows, C, F, torch.bfloat16)
    got = gated_all(*ins, "silu")
    a, u = (x.double() @ w.double().T + b.double() for w, b in ((wg, bg), (wu, bu)))
    f, df = act64(a, "silu")
    da, du = dy.double() * u * df, dy.double() * f
    want = {"dx": da @ wg.double() + du @ wu.double(), "dwg": da.T @ x.double(),
            "dwu": du.T @ x.double(), "dbg": da.sum(0), "dbu": du.sum(0)}
    for name, w in want.items():
        e = float((got[name].double() - w).norm() / w.norm())
        r = float((w.bfloat16().double() - w).norm() / w.norm())
        assert e <= 1.02 * r, f"{name}: {e:.4g} against {r:.4g}"


def test_gated_linear_infinite_gradients_stay_infinite():
    """bfloat16: what rounding leaves of an infinity is no second part."""
    x, wg, wu, bg, bu, dy = gated_inputs(gen(22), 70, 64, 72, torch.bfloat16)
    dy[3, 5] = math.inf
    dx, dwg, dwu, _, _ = pc.pc_gated_linear_backward(dy, x, wg, wu, bg, bu)
    a, u = (x[3].double() @ w[5].double() + b[5].double() for w, b in ((wg, bg), (wu, bu)))
    f, df = act64(a, "silu")
    for got, ref in ((dwg[5], math.inf * u * df * x[3].double()),
                     (dwu[5], math.inf * f * x[3].double())):
        assert torch.equal(got.double(), ref)
    both = math.inf * u * df * wg[5].double() + math.inf * f * wu[5].double()  # inf, -inf or NaN
    assert torch.equal(dx[3].double().nan_to_num(7.0), both.nan_to_num(7.0))
    keep = torch.arange(70, device=DEV) != 3
    assert torch.isfinite(dx[keep]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 70, 300])
def test_gated_linear_bias_gradients_of_infinite_biases(rows, dtype):
    """The sums over the rows are those of the rows alone, whatever the biases are."""
    x, wg, wu, bg, bu, dy = gated_inputs(gen(23), rows, 64, 72, dtype)
    dy = dy.abs() + 0.5
    want = pc.pc_gated_linear_backward(dy, x, wg, wu, bg, bu, activation="sigmoid")
    bu = bu.clone()
    bu[5] = math.inf
    _, _, _, dbg, dbu = pc.pc_gated_linear_backward(dy, x, wg, wu, bg, bu, activation="sigmoid")
    assert dbg[5] == math.inf and torch.equal(dbu, want[4])
    keep = torch.arange(72, device=DEV) != 5
    assert torch.equal(dbg[keep], want[3][keep])


def test_gelu_s_far_side_in_bfloat16():
    """gelu(z) and its derivative where the normal distribution's function is small: half a
    unit of bfloat16 (its numbers from 1 to 2 are 2^-7 apart: at most 2^-8 of the value), and
    2^-16 for the approximation (9e-6 of the distribution's function, a few units of float32
    beside) of the terms that enter; below float32's normal numbers, 1e-37 |z|."""
    def gelu64(v):   # (by erfc: 1 + erf keeps no digits there)
        c = 0.5 * torch.erfc(-v * math.sqrt(0.5))
        return v * c, c, v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)

    z = torch.arange(-13.25, 4.0, 2.0 ** -6, device=DEV, dtype=torch.float64).bfloat16()
    z = z.unique()
    rows = z.numel()
    x = torch.zeros(rows, 8, device=DEV, dtype=torch.bfloat16)
    x[:, 0], x[:, 1] = z, 1.0
    wg, wu = (torch.zeros(8, 8, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    wg[:, 0], wu[:, 1] = 1.0, 1.0            # a = z, u = 1
    dy = torch.zeros(rows, 8, device=DEV, dtype=torch.bfloat16)
    dy[:, 3] = 1.0
    y = pc.pc_gated_linear(x, wg, wu, activation="gelu")
    dx, *_ = pc.pc_gated_linear_backward(dy, x, wg, wu, activation="gelu")
    z = z.double()
    f, c, g = gelu64(z)
    low = 1e-37 * (1 + z.abs())
    close(y, f[:, None].expand(rows, 8), (f.abs() * (HALF[torch.bfloat16] + 2.0 ** -16) + low)[:, None], "y")
    close(dx[:, 0], c + g, (c + g).abs() * HALF[torch.bfloat16] + (c + g.abs()) * 2.0 ** -16 + low,
          "dx")
    # group norm's results take the same function: one row of +-z is its own norm
    v = torch.cat([z, -z]).view(1, -1, 1)
    s = (v * v).mean().sqrt()
    h = pc.pc_group_norm((v / s).bfloat16(), 1, s.float().view(1), eps=0.0, activation="gelu")
    q = (v / s).bfloat16().double()
    w = float(s.float()) * (q - q.mean()) / ((q - q.mean()) ** 2).mean().sqrt()
    want, c, g = gelu64(w)
    # (w itself is off by a few units of float32 of the largest)
    close(h, want, want.abs() * (HALF[torch.bfloat16] + 2.0 ** -16)
          + (c + g).abs() * 64 * U * w.abs().max() + 1e-37 * (1 + w.abs()), "group norm")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(65, 40, 24, 3), (1025, 9, 40, 5), (8192, 32, 128, 32),
                                   (65536, 8, 16, 4)])
def test_group_norm_of_many_clouds(shape, dtype):
    """The parameters' gradients are sums over all clouds whose chains of additions do not grow
    with their number: a cloud's L points (and 8 joins), then 64 for every factor of 1024."""
    B, L, C, G = shape
    g = gen(B)
    x, dy = randn(g, B, L, C, dtype=dtype), randn(g, B, L, C, dtype=dtype)
    w, b = randn(g, C) + 1, randn(g, C)
    lengths = torch.randint(0, L + 1, (B,), generator=g, device=DEV)
    got = gn_all(x, G, w, b, "sigmoid", lengths, dy)
    for name, (want, tol) in gn_reference(x, G, w, b, 1e-5, "sigmoid", lengths, dy).items():
        close(got[name], want, tol, name)
    # a cloud's sum of 1 + 7 / 2^13: a chain over the clouds drops the fraction from 2^14 on
    if dtype is torch.float32 and L == 8:
        dy.fill_((1 + 7 * 2.0 ** -13) / 8)
        one = torch.ones(C, device=DEV)
        y, m, r = pc.pc_group_norm(x, G, one, one, return_stats=True)
        _, _, db = pc.pc_group_norm_backward(dy, x, m, r, G, one, one)
        want = torch.full((C,), B * (1 + 7 * 2.0 ** -13), device=DEV, dtype=torch.float64)
        close(db, want, (L + 8 + 2 * 64) * U * want, "db")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_group_norm_parameter_gradients_in_norm(act, dtype):
    """float32 sums of the derivative over 16,000 points, whose own errors have random signs:
    what the approximate functions of bfloat16 calls leave does not, so the error in norm is
    at most theirs (2^-21 of the terms, to be compared with the sums of as many terms of random
    sign: a factor of up to 2) beside twice that of the float32 form."""
    g = gen(41)
    B, L, C, G = 4, 4093, 195, 13
    x, dy = ((1.5 * randn(g, B, L, C)).to(dtype), randn(g, B, L, C, dtype=dtype))
    w, b = 1 + 0.1 * randn(g, C), 0.1 * randn(g, C)
    got = gn_all(x, G, w, b, act, None, dy)
    want = gn_reference(x, G, w, b, 1e-5, act, None, dy)
    v = x.float().view(B, L, G, -1)
    c = v - v.mean((1, 3), keepdim=True)
    xh = (c * torch.rsqrt((c * c).mean((1, 3), keepdim=True) + 1e-5)).view(B, L, C)
    z = xh * w + b
    if act == "gelu":
        slope = (0.5 * torch.erfc(-z * math.sqrt(0.5))
                 + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    else:
        s = torch.sigmoid(z)
        slope = s * (1 + z * (1 - s))
    d = dy.float() * slope
    for name, p in (("dw", (d * xh).sum((0, 1))), ("db", d.sum((0, 1)))):
        ref = want[name][0]
        e = float((got[name].double() - ref).norm() / ref.norm())
        r = float((p.double() - ref).norm() / ref.norm())
        assert e <= 2 * r + 2 * 2.0 ** -21, f"{name}: {e:.3g} against {r:.3g}"


@pytest.mark.parametrize("shape", [(2, 3000, 32, 4), (1, 14000, 8, 1), (1, 100000, 1, 1),
                                   (3, 1024, 384, 32), (1, 30000, 512, 32), (1, 5000, 515, 5)])
@pytest.mark.parametrize("mean", [1e2, 1e4])
def test_group_norm_of_large_means_in_norm(shape, mean):
    """Results around a large mean against the two-pass float32 form: the variance does not
    cancel, and the mean is off by a few units of float32 as any float32 mean is (its own
    rounding, at most 2^-24 of it, and sums of the same length)."""
    B, L, C, G = shape
    g = gen(L)
    x, dy = randn(g, B, L, C) + mean, randn(g, B, L, C)
    y, m, r = pc.pc_group_norm(x, G, return_stats=True)
    v = x.double().view(B, L, G, -1)
    m64 = v.mean((1, 3), keepdim=True)
    r64 = (v.var((1, 3), unbiased=False, keepdim=True) + 1e-5) ** -0.5
    want = (v - m64) * r64
    f = x.view(B, L, G, -1)
    c = f - f.mean((1, 3), keepdim=True)
    plain = c * torch.rsqrt((c * c).mean((1, 3), keepdim=True) + 1e-5)

    def off(a):
        return float((a.double() - want).norm() / want.norm())
    assert off(y.view_as(want)) <= 3 * off(plain) + U * mean
    # means that are off by at most e enter the joined squares as sums of n (d + e)^2 instead of
    # n d^2: a variance of 1 is off by at most 2 e + e^2, rstd by half of that; e is four of the
    # mean's half units.  Beside it 64 roundings of the sums.
    e = 4 * U * mean
    assert float((r.view_as(r64) / r64 - 1).abs().max()) <= 64 * U + e + e * e / 2


def longest_chain(T, run):
    """Additions of a row of T tokens: a run; the ends of each level of sums of 32 before the
    last, at most 31 on either side and a sum's own 32; what the last level has."""
    n, chain = -(-T // run), run + 32
    first = True
    while n > (32 if first else 256):
        n, chain, first = n // 32, chain + 31 + 31 + 32, False
    return chain + n


@pytest.mark.parametrize("T,C,run", [(600_000, 4, 16), (3_000_000, 4, 64), (20_000_000, 1, 64)])
def test_embedding_sum_of_a_row_with_most_of_the_tokens(T, C, run):
    """All of one sign and alike: a chain that is as long as the row has sums of 32 runs drops
    what is below a unit of what it has at each of them."""
    v = 1 + 15 * 2.0 ** -18
    dy = torch.full((T, C), v, device=DEV)
    idx = torch.full((T,), 3, device=DEV)
    idx[:5], idx[T // 2] = 1, 6                     # the row begins inside a run
    d = pc.pc_embedding_backward(dy, idx, (9, C))
    n = torch.zeros(9, 1, dtype=torch.float64, device=DEV)
    n[1], n[6], n[3] = 5, 1, T - 6
    want = (n * v).expand(9, C)
    close(d, want, longest_chain(T, run) * U * want + 1e-30, "grad_table")


@pytest.mark.parametrize("dtype", DTYPES)
def test_embedding_of_many_tokens_and_few_frequent_rows(dtype):
    g = gen(51)
    T, V, C = 2_500_000, 5000, 8
    u = torch.rand(T, generator=g, device=DEV)
    idx = (V * u ** 8).long().clamp_max(V - 1)
    idx[torch.rand(T, generator=g, device=DEV) < 0.3] = 777
    idx[torch.rand(T, generator=g, device=DEV) < 0.1] = -1
    dy = randn(g, T, C, dtype=dtype)
    d = pc.pc_embedding_backward(dy, idx, (V, C), 0.5)
    s, m = emb_reference(dy, idx, (V, C), 0.5)
    close(d, s, longest_chain(T, 64) * U * m + HALF[dtype] * s.abs() + 1e-30, "grad_table")
    assert torch.equal(d, pc.pc_embedding_backward(dy, idx, (V, C), 0.5))


@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_linear_workspace_of_unaligned_arrays(dtype):
    """What the C ABI asks for with PC_GATED_UNALIGNED is enough for arrays at any address: the
    call takes it (a call that it is too small for leaves it as it was)."""
    from point_cloud_neighbor_gb300.binding import lib
    L, code, shape = lib(), 0 if dtype is torch.float32 else 1, (300, 128, 200)

    def moved(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].copy_(
            t.reshape(-1)).view(t.shape)
    ins = gated_inputs(gen(8), *shape, dtype)
    want = gated_all(*ins, "silu")
    s = torch.cuda.current_stream().cuda_stream
    flag = pc.features.PC_GATED_UNALIGNED
    for which in ((0, 1, 2), (0,), (1,), (2,)):          # of x, w_gate and w_up
        x, wg, wu, bg, bu, dy = [moved(t) if i in which else t for i, t in enumerate(ins)]
        args = [x.data_ptr(), code, *shape, wg.data_ptr(), wu.data_ptr(), bg.data_ptr(),
                bu.data_ptr(), 1]
        outs = {k: torch.full_like(v, math.nan) for k, v in want.items()}
        for gradients in (0, 7):
            n = L.pc_gated_linear_workspace_bytes(code, *shape, gradients | flag)
            plain = L.pc_gated_linear_workspace_bytes(code, *shape, gradients)
            assert n > plain if dtype is torch.bfloat16 else n == plain
            for bytes_, used in ((n, True), (plain, dtype is torch.float32)):
                work = torch.full((n + 256,), 77, dtype=torch.uint8, device=DEV)
                if gradients:
                    assert L.pc_gated_linear_backward(
                        dy.data_ptr(), *args, *[outs[k].data_ptr() for k in
                                                ("dx", "dwg", "dwu", "dbg", "dbu")],
                        work.data_ptr(), bytes_, s) == 0
                else:
                    assert L.pc_gated_linear(*args, outs["y"].data_ptr(), work.data_ptr(), bytes_,
                                             s) == 0
                assert bool((work[:n] != 77).any()) == used
                assert (work[n:] == 77).all()
        for k in want:
            assert torch.equal(outs[k], want[k]), k


def test_large_calls_on_unaligned_views_take_one_workspace():
    """A call whose scratch comes from torch's allocator takes nothing from the library's pool:
    its size is that of the call's own arrays."""
    rows, C, F = 33000, 64, 512
    x, wg, wu, bg, bu, dy = gated_inputs(gen(9), rows, C, F, torch.bfloat16)
    want = gated_all(x, wg, wu, bg, bu, dy, "silu")
    flat = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].copy_(x.reshape(-1))
    xo = flat.view(x.shape)
    sizes, real = [], pc.features.torch.empty

    def empty(*a, **k):
        if k.get("dtype") is torch.uint8:
            sizes.append(a[0])
        return real(*a, **k)
    pc.features.torch.empty = empty
    try:
        got = gated_all(xo, wg, wu, bg, bu, dy, "silu")
    finally:
        pc.features.torch.empty = real
    for k in want:
        assert torch.equal(got[k], want[k]), k
    lib = pc.binding.lib()
    assert sizes == [lib.pc_gated_linear_workspace_bytes(1, rows, C, F, g) for g in (8, 15)]
    assert sizes[0] >= 2 * x.numel()


def test_gated_linear_of_infinities():
    """float32: NaN in what they enter, as documented, and nothing elsewhere; bfloat16: what the
    definition gives forward."""
    for dtype in DTYPES:
        x, wg, wu, bg, bu, dy = gated_inputs(gen(24), 40, 64, 72, dtype)
        want = pc.pc_gated_linear(x, wg, wu, bg, bu, activation="relu")
        for big in (math.inf, 3.4e38):
            w = wg.clone()
            w[7, 3] = big          # (3.4e38 is infinite in bfloat16)
            y = pc.pc_gated_linear(x, w, wu, bg, bu, activation="relu")
            keep = torch.arange(72, device=DEV) != 7
            assert torch.equal(y[:, keep], want[:, keep])
            if dtype is torch.float32:
                assert y[:, 7].isnan().all()
                continue
            u = x.double() @ wu[7].double() + bu[7].double()
            up = x[:, 3].double() > 0
            assert torch.equal(y[:, 7].double(), torch.where(up, math.inf * u, 0.0))


def test_group_norm_gradients_of_some_with_many_clouds():
    g = gen(61)
    x, dy = randn(g, 1100, 5, 24), randn(g, 1100, 5, 24)
    w, b = randn(g, 24), randn(g, 24)
    _, m, r = pc.pc_group_norm(x, 4, w, b, activation="silu", return_stats=True)
    full = pc.pc_group_norm_backward(dy, x, m, r, 4, w, b, activation="silu")
    for need in ({"need_x": False}, {"need_weight": False}, {"need_bias": False},
                 {"need_weight": False, "need_bias": False},
                 {"need_x": False, "need_weight": False}):
        some = pc.pc_group_norm_backward(dy, x, m, r, 4, w, b, activation="silu", **need)
        for f, s, k in zip(full, some, ("need_x", "need_weight", "need_bias")):
            assert (s is not None) == need.get(k, True)
            assert s is None or torch.equal(f, s)
