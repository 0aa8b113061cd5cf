"""GPU checks of the point-token operators (layer norm, rotary positions,
attention with a distance bias) against plain implementations in float64.

Tolerances are first-order error bounds of the float32 arithmetic, element by
element: u = 2^-24 a rounding, the number of roundings of the longest chain
times the sum of the magnitudes that enter it, plus half a unit of the result's
type.  In bfloat16 the attention kernels may round the weights P and dS to
bfloat16 before the second product: 2^-9 of each term.
"""
import math

import pytest
import torch

import point_cloud_neighbor_gb300 as pc

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a unit, at most
DTYPES = [torch.float32, torch.bfloat16]
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


# --- layer norm ----------------------------------------------------------------

def ln_reference(x, w, b, eps, dy):
    x, dy = x.double(), dy.double()
    C = x.shape[-1]
    w = torch.ones(C, device=DEV, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(C, device=DEV, dtype=torch.float64) if b is None else b.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / (((x - mean) ** 2).mean(-1, keepdim=True) + eps).sqrt()
    xh = (x - mean) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    flat = (-1, C)
    return dict(y=xh * w + b, mean=mean.squeeze(-1), rstd=rstd.squeeze(-1), dx=dx,
                dw=(dy * xh).reshape(flat).sum(0), db=dy.reshape(flat).sum(0), xh=xh, g=g, w=w, b=b)


@pytest.mark.parametrize("dtype,pdtype", [(torch.float32, torch.float32),
                                          (torch.bfloat16, torch.float32),
                                          (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("shape", [(1, 1), (3, 2), (1, 7), (5, 31), (2, 3, 64), (9, 257),
                                   (17, 384), (33, 515), (4, 1024), (3, 1025), (6, 2050),
                                   (2, 8192), (2, 8191), (1500, 48)])
def test_layer_norm(shape, dtype, pdtype):
    g = gen(sum(shape))
    C, rows = shape[-1], math.prod(shape[:-1])
    x = (randn(g, *shape) * 2 + randn(g, C)).to(dtype)
    w, b, dy = (randn(g, C) + 1).to(pdtype), randn(g, C).to(pdtype), randn(g, *shape, dtype=dtype)
    y, mean, rstd = pc.pc_layer_norm(x, w, b, 1e-5, return_stats=True)
    dx, dw, db = pc.pc_layer_norm_backward(dy, x, mean, rstd, w, b)
    assert torch.equal(y, pc.pc_layer_norm(x, w, b, 1e-5))
    r = ln_reference(x, w, b, 1e-5, dy)
    # the longest chain of a row's sum: 32 elements, 5 shuffles, 8 warps, a few more
    K = 64 * U
    a = x.double().abs().mean(-1, keepdim=True)
    close(mean, r["mean"], K * a.squeeze(-1) + 1e-30, "mean")
    # the variance's relative error: its own sum's, and the mean's error enters squared or against
    # a zero sum; centring costs u |x| an element
    rs = r["rstd"].unsqueeze(-1)
    rel = 2 * K + 8 * U * a * rs + (K * a * rs) ** 2
    close(rstd, r["rstd"], (rel * rs).squeeze(-1), "rstd")
    exh = rel * r["xh"].abs() + 2 * K * a * rs + U * x.double().abs() * rs
    close(y, r["y"], r["w"].abs() * exh + 2 * U * (r["w"] * r["xh"]).abs()
          + U * r["b"].abs() + HALF[dtype] * r["y"].abs() + 1e-30, "y")
    ga, xa = r["g"].abs(), r["xh"].abs()
    mg, mgx = ga.mean(-1, keepdim=True), (ga * xa).mean(-1, keepdim=True)
    edx = rs * (K * (ga + mg + xa * mgx) + exh * mgx + xa * (ga * exh).mean(-1, keepdim=True))
    close(dx, r["dx"], edx + rel * r["dx"].abs() + HALF[dtype] * r["dx"].abs() + 1e-30, "dx")
    n = (rows + 64) * U
    da = dy.double().abs().reshape(rows, C)
    close(dw, r["dw"], (da * (exh + n * xa).reshape(rows, C)).sum(0)
          + HALF[pdtype] * r["dw"].abs() + 1e-30, "dw")
    close(db, r["db"], n * da.sum(0) + HALF[pdtype] * r["db"].abs() + 1e-30, "db")


@pytest.mark.parametrize("dtype", DTYPES)
def test_layer_norm_without_parameters(dtype):
    g = gen(1)
    x, dy = randn(g, 11, 130, dtype=dtype), randn(g, 11, 130, dtype=dtype)
    y, mean, rstd = pc.pc_layer_norm(x, return_stats=True)
    one, zero = torch.ones(130, device=DEV), torch.zeros(130, device=DEV)
    assert torch.equal(y, pc.pc_layer_norm(x, one, zero))
    dx, dw, db = pc.pc_layer_norm_backward(dy, x, mean, rstd)
    assert dw is None and db is None
    assert torch.equal(dx, pc.pc_layer_norm_backward(dy, x, mean, rstd, one, zero)[0])
    _, dw, db = pc.pc_layer_norm_backward(dy, x, mean, rstd, one, None)
    assert dw is not None and db is None


def test_layer_norm_of_a_constant_row_and_a_large_mean():
    # a constant row: variance 0; y = bias exactly, gradients finite
    x = torch.full((2, 96), 3.25, device=DEV)
    b = torch.arange(96, device=DEV, dtype=torch.float32)
    y, mean, rstd = pc.pc_layer_norm(x, torch.ones(96, device=DEV), b, 1e-5, return_stats=True)
    assert torch.equal(y, b.expand(2, 96))
    # mean 4096 times the deviation: sums of squares would cancel in float32
    x = 4096 + randn(gen(2), 8, 640)
    want = ln_reference(x, None, None, 1e-5, x)["y"]
    got = pc.pc_layer_norm(x).double()
    # the mean is off by at most 64 u 4096, the centring by 1 u 4096
    assert (got - want).abs().max() <= 80 * U * 4096 * 1.2


def test_layer_norm_empty():
    for shape in ((0, 32), (4, 0), (2, 0, 8)):
        x = torch.empty(shape, device=DEV)
        w = torch.ones(shape[-1], device=DEV)
        y, mean, rstd = pc.pc_layer_norm(x, w, w, return_stats=True)
        dx, dw, db = pc.pc_layer_norm_backward(x, x, mean, rstd, w, w)
        assert y.shape == dx.shape == x.shape
        assert not dw.any() and not db.any()


# --- rotary ---------------------------------------------------------------------

def rotary_reference(x, pos, freqs, interleaved, inverse):
    x, y = x.double(), x.double().clone()
    A, F = freqs.shape
    e = torch.zeros_like(x)
    for a in range(A):
        for f in range(F):
            p = a * F + f
            i, j = (2 * p, 2 * p + 1) if interleaved else (p, A * F + p)
            t = (pos[..., a].double() * freqs[a, f].double()).unsqueeze(-1)
            s = -t.sin() if inverse else t.sin()
            y[..., i] = x[..., i] * t.cos() - x[..., j] * s
            y[..., j] = x[..., j] * t.cos() + x[..., i] * s
            e[..., i] = e[..., j] = x[..., i].abs() + x[..., j].abs()
    return y, e


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,L,H,Hkv,D,A,F", [
    (1, 1, 1, 1, 2, 1, 1), (2, 3, 4, 2, 64, 3, 10), (1, 77, 3, 1, 48, 3, 8), (2, 9, 5, 5, 7, 3, 1),
    (3, 130, 8, 2, 128, 3, 21), (1, 5, 2, 1, 32, 1, 16), (1, 300, 1, 1, 24, 4, 2),
    (4, 1, 8, 8, 64, 2, 16), (1, 3, 2, 2, 64, 3, 0)])
def test_rotary(B, L, H, Hkv, D, A, F, interleaved, dtype):
    g = gen(B + L + D)
    q, k = randn(g, B, L, H, D, dtype=dtype), randn(g, B, L, Hkv, D, dtype=dtype)
    pos, freqs = 3 * randn(g, B, L, A), 30 * torch.rand(A, F, generator=g, device=DEV)
    for inverse in (False, True):
        got = pc.pc_rotary(q, k, pos, freqs, interleaved=interleaved, inverse=inverse)
        for t, x in zip(got, (q, k)):
            want, e = rotary_reference(x, pos, freqs, interleaved, inverse)
            # sine and cosine 2 units, two products and a sum
            close(t, want, 6 * U * e + HALF[dtype] * want.abs() + 1e-30, "rotary")
    alone, none = pc.pc_rotary(q, None, pos, freqs, interleaved=interleaved, inverse=True)
    assert none is None and torch.equal(alone, got[0])


def test_rotary_angle_keeps_its_low_bits():
    # angles near 1e4: the float32 product alone is off by up to 5e-4
    g = gen(5)
    q = randn(g, 1, 64, 2, 32)
    pos, freqs = 1000 + randn(g, 1, 64, 2), 10 + torch.rand(2, 8, generator=g, device=DEV)
    got, _ = pc.pc_rotary(q, None, pos, freqs)
    want, e = rotary_reference(q, pos, freqs, True, False)
    close(got, want, 6 * U * e + 1e-30, "rotary")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("at", [0, 1])
def test_rotary_strided_views(dtype, at):
    # q and k as slices of one projection, and at an odd offset (no wide loads)
    g = gen(6)
    B, L, H, Hkv, D = 2, 19, 4, 2, 32
    base = randn(g, B, L, (H + 2 * Hkv) * D + 2, dtype=dtype)[..., at:]
    q = base[..., :H * D].unflatten(-1, (H, D))
    k = base[..., H * D:(H + Hkv) * D].unflatten(-1, (Hkv, D))
    pos, freqs = randn(g, B, L, 3), torch.rand(3, 5, generator=g, device=DEV)
    for il in (True, False):
        a = pc.pc_rotary(q, k, pos, freqs, interleaved=il)
        b = pc.pc_rotary(q.contiguous(), k.contiguous(), pos, freqs, interleaved=il)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    t = pc.pc_rotary(q.transpose(1, 2).contiguous().transpose(1, 2), k, pos, freqs)
    assert torch.equal(t[0], pc.pc_rotary(q.contiguous(), k, pos, freqs)[0])


# --- attention --------------------------------------------------------------------

class Ref:
    """Attention and its gradients in float64, with the error bounds."""

    def __init__(self, q, k, v, do, scale, kw, dtype):
        B, Lq, H, D = q.shape
        Lk, Hkv = k.shape[1], k.shape[2]
        G = H // Hkv
        nq = kw.get("query_lengths")
        nk = kw.get("ref_lengths")
        nq = [Lq] * B if nq is None else nq.clamp(0, Lq).tolist()
        nk = [Lk] * B if nk is None else nk.clamp(0, Lk).tolist()
        z64 = dict(dtype=torch.float64, device=DEV)
        self.out, self.dq = torch.zeros(B, Lq, H, D, **z64), torch.zeros(B, Lq, H, D, **z64)
        self.dk, self.dv = torch.zeros(B, Lk, Hkv, D, **z64), torch.zeros(B, Lk, Hkv, D, **z64)
        self.dslopes, self.eslopes = torch.zeros(H, **z64), torch.zeros(H, **z64)
        self.lse = torch.full((B, H, Lq), -math.inf, **z64)
        self.elses = torch.zeros(B, H, Lq, **z64)
        self.eout, self.edq = torch.zeros_like(self.out), torch.zeros_like(self.dq)
        self.edk, self.edv = torch.zeros_like(self.dk), torch.zeros_like(self.dv)
        narrow = dtype != torch.float32
        up = 2.0 ** -9 if narrow else 0.0        # P and dS as operands
        ua = 4 * U if narrow else U              # a sum's step on the tensor cores
        hf = HALF[dtype]
        for b in range(B):
            n, m = nk[b], nq[b]
            if n == 0 or m == 0:
                continue
            for h in range(H):
                kh = h // G
                Q, K, V = q[b, :m, h].double(), k[b, :n, kh].double(), v[b, :n, kh].double()
                g = do[b, :m, h].double()
                z = scale * Q @ K.T
                ez = ua * (D + 4) * scale * (Q.abs() @ K.abs().T)
                if "slopes" in kw:
                    w = kw["slopes"][h].double()
                    x, y = kw["query_xyz"][b, :m].double(), kw["ref_xyz"][b, :n].double()
                    d2 = ((x[:, None] - y[None]) ** 2).sum(-1)
                    z = z - w * d2
                    ez = ez + 10 * U * w.abs() * d2
                ez = ez + 4 * U * z.abs()
                lse = torch.logsumexp(z, 1, keepdim=True)
                P = torch.exp(z - lse)
                # relative error of a weight: its own exponent's, the row's, the sum's and exp's
                el = (P * ez).sum(1, keepdim=True) + U * (n + 8) + 4 * U * lse.abs()
                r = ez + el + 4 * U * (lse.abs() + 2)
                O = P @ V
                Va = V.abs()
                eO = (P * r) @ Va + (up + ua * (n + 4)) * (P @ Va)
                self.out[b, :m, h], self.lse[b, h, :m] = O, lse[:, 0]
                self.eout[b, :m, h] = eO + hf * O.abs()
                self.elses[b, h, :m] = el[:, 0]
                dP = g @ V.T
                edP = ua * (D + 2) * (g.abs() @ Va.T)
                dl = (P * dP).sum(1, keepdim=True)
                edl = ((eO + hf * O.abs()) * g.abs()).sum(1, keepdim=True) \
                    + U * (D + 2) * (O.abs() * g.abs()).sum(1, keepdim=True)
                dS = P * (dP - dl)
                edS = P * (edP + edl + 2 * U * (dP.abs() + dl.abs())) + dS.abs() * (r + up)
                Ka, Qa, ga = K.abs(), Q.abs(), g.abs()
                s = scale
                self.dq[b, :m, h] = s * dS @ K
                self.edq[b, :m, h] = s * (edS @ Ka + ua * (n + 4) * (dS.abs() @ Ka))
                self.dk[b, :n, kh] += s * dS.T @ Q
                self.edk[b, :n, kh] += s * (edS.T @ Qa + ua * (G * m + 4) * (dS.abs().T @ Qa))
                self.dv[b, :n, kh] += P.T @ g
                self.edv[b, :n, kh] += (P * (r + up + ua * (G * m + 4))).T @ ga
                if "slopes" in kw:
                    self.dslopes[h] -= (dS * d2).sum()
                    dPa = dP.abs()
                    row = (P * (dPa * (r + U * (n + 16)) + edP) * d2).sum(1) \
                        + (P * (dPa * (r + U * (n + 16)) + edP)).sum(1) * (P * d2).sum(1) \
                        + (P * dPa).sum(1) * (P * d2 * (r + U * (n + 16))).sum(1)
                    self.eslopes[h] += row.sum()
        self.edq += hf * self.dq.abs()
        self.edk += hf * self.dk.abs()
        self.edv += hf * self.dv.abs()


def lens(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


def attn_inputs(B, Lq, Lk, H, Hkv, D, dtype, bias, ql, rl, seed=0):
    g = gen(seed + B + 3 * Lq + 5 * Lk + 7 * D)
    q, k, v = (randn(g, B, L, h, D, dtype=dtype) for L, h in ((Lq, H), (Lk, Hkv), (Lk, Hkv)))
    do = randn(g, B, Lq, H, D, dtype=dtype)
    kw = {}
    if bias:
        kw["slopes"] = torch.rand(H, generator=g, device=DEV) * 3 - 0.5
        kw["query_xyz"], kw["ref_xyz"] = randn(g, B, Lq, 3), randn(g, B, Lk, 3)
    if ql is not None:
        kw["query_lengths"] = lens(ql)
    if rl is not None:
        kw["ref_lengths"] = lens(rl)
    return q, k, v, do, kw


def check_attention(q, k, v, do, kw, dtype, scale=None):
    sc = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    ref = Ref(q, k, v, do, sc, kw, dtype)
    out, lse = pc.pc_attention(q, k, v, scale=scale, return_lse=True, **kw)
    assert torch.equal(out, pc.pc_attention(q, k, v, scale=scale, **kw))
    tiny = 1e-30
    close(out, ref.out, ref.eout + tiny, "out")
    empty = ref.lse == -math.inf
    assert torch.equal(lse == -math.inf, empty), "rows without keys"
    close(torch.where(empty, 0.0, lse.double()), torch.where(empty, 0.0, ref.lse),
          ref.elses + tiny, "lse")
    dq, dk, dv, ds = pc.pc_attention_backward(do, q, k, v, out, lse, scale=scale, **kw)
    close(dq, ref.dq, ref.edq + tiny, "dq")
    close(dk, ref.dk, ref.edk + tiny, "dk")
    close(dv, ref.dv, ref.edv + tiny, "dv")
    if "slopes" in kw:
        close(ds, ref.dslopes, ref.eslopes + U * ref.dslopes.abs() + tiny, "dslopes")
    else:
        assert ds is None
    again = pc.pc_attention_backward(do, q, k, v, out, lse, scale=scale, **kw)
    assert all(a is None and b is None or torch.equal(a, b)
               for a, b in zip(again, (dq, dk, dv, ds))), "the same call twice"


SHAPES = [
    # B, Lq, Lk, H, Hkv, D, query lengths, ref lengths
    (1, 1, 1, 1, 1, 1, None, None),
    (1, 1, 1, 2, 1, 64, None, None),
    (2, 3, 5, 2, 2, 7, None, [5, 0]),
    (1, 64, 64, 1, 1, 64, None, None),
    (2, 65, 63, 3, 1, 64, [65, 1], [63, 62]),
    (1, 127, 129, 2, 2, 32, None, None),
    (1, 128, 128, 1, 1, 128, None, None),
    (3, 130, 257, 4, 2, 128, [130, 0, 77], [256, 257, 1]),
    (2, 200, 200, 6, 6, 48, [200, 64], [200, 64]),
    (1, 1, 5000, 4, 2, 64, None, None),
    (2, 2, 3001, 4, 1, 128, None, [3001, 17]),
    (1, 4, 700, 8, 8, 40, None, None),
    (1, 700, 3, 2, 2, 64, None, None),
    (1, 513, 1030, 2, 1, 96, [500], [1000]),
    (1, 300, 300, 1, 1, 100, None, None),
    (2, 90, 70, 2, 2, 33, None, None),
    (5, 40, 40, 2, 1, 24, [40, 0, 3, 40, 9], [0, 40, 40, 33, 1]),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D,ql,rl", SHAPES)
def test_attention(B, Lq, Lk, H, Hkv, D, ql, rl, bias, dtype):
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, dtype, bias, ql, rl)
    check_attention(q, k, v, do, kw, dtype)


# Many clouds and heads: blocks walk over several tiles and heads each, most of them
# with a ragged end (the keys' gradient over the query heads of a group too).
MANY = [
    (12, 333, 333, 16, 8, [333, 300, 257, 256, 255, 193, 129, 128, 65, 64, 1, 0],
     [333, 1, 64, 65, 128, 129, 193, 255, 256, 257, 300, 333]),
    (16, 90, 400, 12, 6, list(range(90, 10, -5)), list(range(400, 0, -25))),
    (40, 70, 70, 24, 4, [70 - i for i in range(40)], [31 + i for i in range(40)]),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,ql,rl", MANY)
def test_attention_many_ragged_clouds(B, Lq, Lk, H, Hkv, ql, rl, bias, D, dtype):
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, dtype, bias, ql, rl)
    for t in (q, do):
        for b in range(B):
            t[b, ql[b]:] = math.nan
    for t in (k, v):
        for b in range(B):
            t[b, rl[b]:] = math.nan
    check_attention(q, k, v, do, kw, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_scale_and_large_scores(dtype):
    # scores of several hundreds: the running maximum has to carry them
    q, k, v, do, kw = attn_inputs(1, 150, 400, 2, 1, 64, dtype, True, None, [390])
    check_attention(10 * q, k, v, do, kw, dtype, scale=0.5)
    # increasing scores along the keys: the maximum moves at every tile
    k = (k.float() * 0 + torch.linspace(0, 8, 400, device=DEV).view(1, -1, 1, 1)).to(dtype)
    check_attention(q.abs(), k, v, do, kw, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_far_from_the_origin(dtype):
    # the distance is formed from differences: an offset of the cloud changes nothing much
    q, k, v, do, kw = attn_inputs(1, 70, 90, 2, 2, 64, dtype, True, None, None)
    for n in ("query_xyz", "ref_xyz"):
        kw[n] = (kw[n] * 64).round() / 64 + 1024.0   # exact at this offset
    check_attention(q, k, v, do, kw, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128, 40])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, 3e38])
def test_attention_padding_is_not_read(dtype, D, junk):
    ql, rl = [100, 0, 33], [200, 77, 1]
    q, k, v, do, kw = attn_inputs(3, 130, 200, 2, 1, D, dtype, True, ql, rl)
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    want = (out, lse, *pc.pc_attention_backward(do, q, k, v, out, lse, **kw))
    for b in range(3):
        q[b, ql[b]:], do[b, ql[b]:], kw["query_xyz"][b, ql[b]:] = junk, junk, junk
        k[b, rl[b]:], v[b, rl[b]:], kw["ref_xyz"][b, rl[b]:] = junk, junk, junk
        assert not out[b, ql[b]:].any()
    out2, lse2 = pc.pc_attention(q, k, v, return_lse=True, **kw)
    for b in range(3):
        out2[b, ql[b]:] = 0
    got = (out2, lse2, *pc.pc_attention_backward(do, q, k, v, out2, lse2, **kw))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_lengths_are_clamped(dtype):
    q, k, v, do, kw = attn_inputs(2, 20, 30, 2, 1, 64, dtype, False, [-4, 1000], [77, -1])
    check_attention(q, k, v, do, kw, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Lq,Lk,B", [(0, 5, 2), (5, 0, 2), (0, 0, 1), (4, 4, 0)])
def test_attention_empty(Lq, Lk, B, dtype):
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, 2, 1, 64, dtype, True, None, None)
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    assert not out.any() and (lse == -math.inf).all()
    dq, dk, dv, ds = pc.pc_attention_backward(do, q, k, v, out, lse, **kw)
    assert not dq.any() and not dk.any() and not dv.any() and not ds.any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,at", [(64, 0), (64, 1), (40, 8), (128, 0)])
def test_attention_strided_views(dtype, D, at):
    # q, k, v as slices of one projection; an odd offset rules out wide loads
    g = gen(9)
    B, L, H, Hkv = 2, 150, 4, 2
    base = randn(g, B, L, (H + 2 * Hkv) * D + 8, dtype=dtype)[..., at:]
    q, k, v = (base[..., i * D:j * D].unflatten(-1, (j - i, D))
               for i, j in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv)))
    kw = dict(ref_lengths=lens([150, 91]))
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    do = randn(g, B, L, H, D, dtype=dtype)
    got = (out, lse, *pc.pc_attention_backward(do, q, k, v, out, lse, **kw))
    check_attention(q, k, v, do, kw, dtype)
    heads_first = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    out2, lse2 = pc.pc_attention(*heads_first, return_lse=True, **kw)
    want = (out2, lse2, *pc.pc_attention_backward(do, *heads_first, out2, lse2, **kw))
    if at % 8 == 0:  # the same kernel: the same bits
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, want))


def test_attention_on_a_side_stream():
    q, k, v, do, kw = attn_inputs(2, 200, 200, 4, 2, 64, torch.bfloat16, True, None, [200, 3])
    want = pc.pc_attention(q, k, v, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = pc.pc_attention(q, k, v, **kw)
    s.synchronize()
    assert torch.equal(got, want)


def test_attention_long_cache_offsets_beyond_32_bits():
    # 2^31 elements lie before the last cloud's keys
    B, Lk, H, D = 3, 8_400_000, 1, 128
    k = torch.zeros(B, Lk, H, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    g = gen(11)
    n = 70
    k[2, :n], v[2, :n] = randn(g, n, H, D, dtype=k.dtype), randn(g, n, H, D, dtype=k.dtype)
    q = randn(g, B, 1, 2, D, dtype=k.dtype)
    rl = lens([0, 5, n])
    out = pc.pc_attention(q, k, v, ref_lengths=rl)
    small = pc.pc_attention(q[2:], k[2:, :n].contiguous(), v[2:, :n].contiguous())
    ref = Ref(q[2:], k[2:, :n], v[2:, :n], q[2:], 1 / math.sqrt(D), {}, torch.bfloat16)
    close(out[2:], ref.out, ref.eout, "out")
    close(small, ref.out, ref.eout, "out, short")
    assert not out[:2].any()


# --- gradients against differences --------------------------------------------------

def directional(f, x, d, h):
    """(f(x + h d) - f(x - h d)) / 2h in float64."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_attention_gradient_against_differences():
    B, L, H, Hkv, D = 2, 37, 4, 2, 16
    q, k, v, do, kw = attn_inputs(B, L, L, H, Hkv, D, torch.float32, True, [37, 20], [30, 37])
    ts = [t.clone().requires_grad_() for t in (q, k, v, kw["slopes"])]
    pos = {n: t for n, t in kw.items() if n != "slopes"}
    pc.attention(*ts[:3], slopes=ts[3], **pos).backward(do)

    def loss(q, k, v, w):
        G = H // Hkv
        keys, vals = (t.repeat_interleave(G, 2) for t in (k, v))
        z = torch.einsum("bihd,bjhd->bhij", q, keys) / math.sqrt(D)
        d2 = ((pos["query_xyz"].double()[:, :, None] - pos["ref_xyz"].double()[:, None]) ** 2).sum(-1)
        z = z - w.view(1, H, 1, 1) * d2[:, None]
        at = torch.arange(L, device=DEV)
        z = z.masked_fill((at >= pos["ref_lengths"][:, None])[:, None, None], -math.inf)
        o = torch.einsum("bhij,bjhd->bihd", z.softmax(-1), vals)
        o = o * (at < pos["query_lengths"][:, None])[:, :, None, None]
        return float((o * do.double()).sum())

    args = [t.detach().double() for t in ts]
    for i in range(4):
        d = torch.randn(args[i].shape, generator=gen(20 + i), device=DEV, dtype=torch.float64)
        diff = directional(lambda t: loss(*args[:i], t, *args[i + 1:]), args[i], d, 1e-5)
        got = float((ts[i].grad.double() * d).sum())
        # differences: h^2 of the third derivative and 1e-16 |f| / h; the kernels' float32 sums
        size = float((ts[i].grad.double() * d).abs().sum())
        assert abs(got - diff) <= 512 * U * size + 1e-6, (i, got, diff)


def test_layer_norm_and_rotary_gradients_against_differences():
    g = gen(30)
    x, w, b, dy = randn(g, 13, 50), randn(g, 50), randn(g, 50), randn(g, 13, 50)
    ts = [t.clone().requires_grad_() for t in (x, w, b)]
    pc.layer_norm(*ts, 1e-3).backward(dy)

    def loss(x, w, b):
        return float((ln_reference(x, w, b, 1e-3, dy)["y"] * dy.double()).sum())

    args = [t.detach().double() for t in ts]
    for i in range(3):
        d = torch.randn(args[i].shape, generator=gen(40 + i), device=DEV, dtype=torch.float64)
        diff = directional(lambda t: loss(*args[:i], t, *args[i + 1:]), args[i], d, 1e-5)
        got = float((ts[i].grad.double() * d).sum())
        size = float((ts[i].grad.double() * d).abs().sum())
        assert abs(got - diff) <= 128 * U * size + 1e-6, (i, got, diff)

    q, k = randn(g, 2, 7, 3, 32), randn(g, 2, 7, 1, 32)
    pos, freqs = randn(g, 2, 7, 3), torch.rand(3, 5, generator=g, device=DEV)
    gq, gk = randn(g, 2, 7, 3, 32), randn(g, 2, 7, 1, 32)
    for il in (True, False):
        q_, k_ = q.clone().requires_grad_(), k.clone().requires_grad_()
        oq, ok = pc.rotary(q_, k_, pos, freqs, il)
        ((oq * gq).sum() + (ok * gk).sum()).backward()
        for t, gt in ((q_, gq), (k_, gk)):
            d = torch.randn(t.shape, generator=gen(50), device=DEV, dtype=torch.float64)
            f = lambda x: float((rotary_reference(x, pos, freqs, il, False)[0] * gt.double()).sum())  # noqa: E731
            diff = directional(f, t.detach().double(), d, 1e-3)  # linear: any step
            got = float((t.grad.double() * d).sum())
            size = float((t.grad.double() * d).abs().sum())
            assert abs(got - diff) <= 16 * U * size + 1e-9


def test_autograd_takes_strided_gradients_and_skips_what_is_not_asked():
    g = gen(60)
    q, k, v = (randn(g, 1, 33, 2, 64).requires_grad_() for _ in range(3))
    o = pc.attention(q, k, v)
    (o.transpose(1, 2).sum(-1) ** 2).sum().backward()      # an expanded, strided gradient
    assert all(torch.isfinite(t.grad).all() for t in (q, k, v))
    x = randn(g, 4, 16).requires_grad_()
    pc.layer_norm(x).sum().backward()
    assert torch.isfinite(x.grad).all()


# --- refusals ---------------------------------------------------------------------

def test_refusals():
    x = torch.zeros(4, 8, device=DEV)
    w = torch.zeros(8, device=DEV)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        pc.pc_layer_norm(x.half())
    with pytest.raises(ValueError, match="contiguous"):
        pc.pc_layer_norm(x.t())
    with pytest.raises(ValueError, match="weight"):
        pc.pc_layer_norm(x, w[:4])
    with pytest.raises(ValueError, match="same dtype"):
        pc.pc_layer_norm(x.bfloat16(), w, w.bfloat16())
    with pytest.raises(pc.PointCloudError, match="eps"):
        pc.pc_layer_norm(x, eps=-1.0)
    with pytest.raises(pc.PointCloudError, match="8192"):
        pc.pc_layer_norm(torch.zeros(1, 8193, device=DEV))
    q = torch.zeros(1, 4, 2, 64, device=DEV)
    k = torch.zeros(1, 6, 1, 64, device=DEV)
    pos, f = torch.zeros(1, 4, 3, device=DEV), torch.zeros(3, 10, device=DEV)
    with pytest.raises(ValueError, match="k must have shape"):
        pc.pc_rotary(q, k, pos, f)
    with pytest.raises(ValueError, match="positions"):
        pc.pc_rotary(q, None, pos[..., :2], f)
    with pytest.raises(pc.PointCloudError, match="turned channels"):
        pc.pc_rotary(q, None, pos, torch.zeros(3, 11, device=DEV))
    with pytest.raises(pc.PointCloudError, match="axes"):
        pc.pc_rotary(q, None, torch.zeros(1, 4, 5, device=DEV), torch.zeros(5, 1, device=DEV))
    with pytest.raises(ValueError, match="last axis"):
        pc.pc_rotary(torch.zeros(1, 4, 64, 2, device=DEV).transpose(2, 3), None, pos, f)
    with pytest.raises(ValueError, match="go together"):
        pc.pc_attention(q, k, k, slopes=torch.zeros(2, device=DEV))
    with pytest.raises(ValueError, match="divide"):
        pc.pc_attention(q, k.expand(1, 6, 3, 64), k.expand(1, 6, 3, 64))
    with pytest.raises(ValueError, match="float32 on"):
        pc.pc_attention(q, k.bfloat16(), k)
    with pytest.raises(ValueError, match="ref_lengths"):
        pc.pc_attention(q, k, k, ref_lengths=torch.zeros(2, dtype=torch.int64, device=DEV))
    with pytest.raises(pc.PointCloudError, match="scale"):
        pc.pc_attention(q, k, k, scale=0.0)
    with pytest.raises(pc.PointCloudError, match="128"):
        pc.pc_attention(torch.zeros(1, 4, 1, 129, device=DEV), *[torch.zeros(1, 4, 1, 129, device=DEV)] * 2)
    with pytest.raises(ValueError, match="lse"):
        pc.pc_attention_backward(q, q, k, k, q, torch.zeros(1, 2, 5, device=DEV))


def test_a_withheld_copy_ends_with_a_status():
    # the first block's copies never come: its waits run out, the context stays usable
    q, k, v, do, kw = attn_inputs(2, 200, 200, 2, 2, 64, torch.bfloat16, True, None, None)
    want = pc.pc_attention(q, k, v, return_lse=True, **kw)
    grads = pc.pc_attention_backward(do, q, k, v, *want, **kw)
    torch.cuda.synchronize()
    try:
        pc.pc_set_wait_timeout_ns(50_000_000)
        pc.pc_debug_set_stall(pc.PC_STALL_ATTENTION)
        pc.pc_attention(q, k, v, **kw)
        assert pc.pc_device_status(reset=True) == 4
        pc.pc_attention_backward(do, q, k, v, *want, **kw)
        assert pc.pc_device_status(reset=True) == 4
    finally:
        pc.pc_debug_set_stall(0)
        pc.pc_set_wait_timeout_ns(2_000_000_000)
    assert torch.equal(pc.pc_attention(q, k, v, **kw), want[0])
    assert all(torch.equal(a, b) for a, b in
               zip(pc.pc_attention_backward(do, q, k, v, *want, **kw), grads))
