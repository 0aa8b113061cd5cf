"""GPU checks of the point-token operators where they are easily wrong: values
that are not finite in valid places, weights and deltas that lose bits, long
sums, and the steady state of the kernels' loops.

Tolerances are derived from the arithmetic as in test_gpu_tokens.py.
"""
import ctypes
import math

import pytest
import torch

import point_cloud_neighbor_gb300 as pc
import test_gpu_tokens as base
from point_cloud_neighbor_gb300.binding import lib
from test_gpu_tokens import (DEV, DTYPES, HALF, U, Ref, attn_inputs,  # noqa: F401
                             clean_status, close, gen, lens, randn)

pytestmark = pytest.mark.gpu


# --- values that are not finite in valid places ------------------------------------

# One shape for each way a row's result is formed: few queries in one part and in many (a block
# per row joins them), tensor cores in one part and in a few (a thread per channels joins them),
# float32 instructions (channels not a multiple of 8), an only key.
ROWS = [(1, 1, 70, 2, 1, 64), (1, 2, 9000, 2, 2, 64), (2, 300, 130, 2, 1, 64),
        (1, 1200, 2000, 1, 1, 128), (1, 90, 70, 2, 1, 36), (1, 40, 2000, 1, 1, 36),
        (1, 20, 1, 2, 1, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", ROWS)
def test_attention_nan_in_a_query_reaches_its_row(B, Lq, Lk, H, Hkv, D, bias, dtype):
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, dtype, bias, None, None)
    at = (0, Lq // 2, H - 1)
    want, wlse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    wgrads = pc.pc_attention_backward(do, q, k, v, want, wlse, **kw)
    q[at][D // 3] = math.nan
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    dq, dk, dv, ds = pc.pc_attention_backward(do, q, k, v, out, lse, **kw)
    assert torch.isnan(out[at]).all() and torch.isnan(lse[0, H - 1, Lq // 2])
    # every key of the cloud and head meets that row
    hk = Hkv - 1
    assert torch.isnan(dq[at]).all()
    assert torch.isnan(dk[0, :, hk]).all() and torch.isnan(dv[0, :, hk]).all()
    assert ds is None or torch.isnan(ds[H - 1])
    # the other rows keep their values
    for t, w in ((out, want), (dq, wgrads[0])):
        t[at], w[at] = 0, 0
        assert torch.equal(t, w)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", ROWS)
def test_attention_nan_in_a_key_or_value_reaches_the_rows(B, Lq, Lk, H, Hkv, D, where, dtype):
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, dtype, False, None, None)
    (k if where == "k" else v)[0, Lk // 2, 0] = math.nan
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    G = H // Hkv
    assert torch.isnan(out[0, :, :G]).all()
    assert torch.isnan(lse[0, :G]).all() == (where == "k")
    assert torch.isfinite(out[1:]).all() and torch.isfinite(out[:, :, G:]).all()
    grads = pc.pc_attention_backward(do, q, k, v, out, lse, **kw)[:3]
    # dv is formed from the weights alone, which a value does not enter
    for t, n, bad in zip(grads, (G, 1, 1), (True, True, where == "k")):
        assert torch.isnan(t[0, :, :n]).all() == bad
        assert torch.isfinite(t[1:]).all() and torch.isfinite(t[:, :, n:]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", ROWS)
def test_attention_scores_that_overflow_are_not_zeros(B, Lq, Lk, H, Hkv, D, sign, dtype):
    # every score of a row is an infinity: no softmax, and not the zeros of a row without keys
    q, k, v, _, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, dtype, False, None, None)
    k = k.abs() + 1
    want, _ = pc.pc_attention(q, k, v, return_lse=True)
    big = 1e38
    q[0, Lq // 2, 0], k = sign * big, k * 1024
    q[0, :Lq // 2] /= 1024
    out, _ = pc.pc_attention(q, k, v, return_lse=True)
    assert torch.isnan(out[0, Lq // 2, 0]).all()
    assert torch.isfinite(out[0, :Lq // 2]).all() and torch.isfinite(want).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", ROWS)
def test_attention_rows_without_keys_are_zeros_among_rows_that_are_nan(B, Lq, Lk, H, Hkv, D,
                                                                        dtype):
    q, k, v, do, _ = attn_inputs(3, Lq, Lk, H, Hkv, D, dtype, False, None, None)
    q[:], k[:, :] = math.nan, math.nan
    ql, rl = lens([0, Lq, Lq - 1]), lens([Lk, 0, 1])
    out, lse = pc.pc_attention(q, k, v, return_lse=True, query_lengths=ql, ref_lengths=rl)
    assert not out[:2].any() and (lse[:2] == -math.inf).all()
    assert not out[2, Lq - 1:].any() and (lse[2, :, Lq - 1:] == -math.inf).all()
    assert torch.isnan(out[2, :Lq - 1]).all() and torch.isnan(lse[2, :, :Lq - 1]).all()
    grads = pc.pc_attention_backward(do, q, k, v, out, lse, query_lengths=ql, ref_lengths=rl)
    assert not any(t[:2].any() for t in grads[:3])
    assert not grads[0][2, Lq - 1:].any()
    assert not grads[1][2, 1:].any() and not grads[2][2, 1:].any()


# --- one key ---------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D,rl", [
    (3, 1, 1, 4, 4, 64, None), (2, 1, 300, 2, 2, 64, [1, 0]), (2, 2, 9000, 2, 2, 128, [1, 1]),
    (4, 30, 1, 4, 2, 64, None), (1, 3000, 1, 8, 1, 128, None), (2, 100, 200, 2, 2, 40, [1, 1]),
    (3, 20, 1, 2, 1, 36, None), (1, 3000, 70, 2, 1, 36, [1]), (1, 40, 2000, 1, 1, 128, [1])])
def test_attention_of_one_key_has_no_gradient_through_its_scores(B, Lq, Lk, H, Hkv, D, rl, dtype):
    # the weight is 1 whatever the score
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, dtype, True, None, rl)
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    dq, dk, dv, ds = pc.pc_attention_backward(do, q, k, v, out, lse, **kw)
    assert not dq.any() and not dk.any() and not ds.any()
    n = torch.tensor([1] * B if rl is None else rl, device=DEV).view(B, 1, 1, 1)
    G = H // Hkv
    # a bfloat16 value as it is; of a float32's three parts up to 4 units a sum are cut off
    one = (n * v[:, :1].repeat_interleave(G, 2)).expand(B, Lq, H, D).double()
    close(out, one, (0.0 if dtype is torch.bfloat16 else 8 * U) * one.abs() + 1e-30, "out")
    g = do.double().view(B, Lq, Hkv, G, D)
    # (G Lq terms, up to 4 units a step on the tensor cores, and weights within 2^-16 of 1)
    size = g.abs().sum((1, 3)).unsqueeze(1) * n
    want = g.sum((1, 3)).unsqueeze(1) * n
    tol = (4 * U * (G * Lq + 4) + 2.0 ** -16) * size + HALF[dtype] * want.abs() + 1e-30
    close(dv[:, :1], want, tol, "dv")
    assert not dv[:, 1:].any()


# --- more clouds than an index of three parts holds -----------------------------------

def test_attention_more_clouds_than_a_third_of_2_31():
    # float32 on the tensor cores numbers 3 B planes in 32 bits; past that the other kernels run
    B = 2 ** 31 // 3 + 2
    q = torch.zeros(B, 1, 1, 1, device=DEV)
    v = torch.zeros(B, 1, 1, 1, device=DEV)
    v[-3:, 0, 0, 0] = torch.tensor([1.5, -2.0, 7.0], device=DEV)
    v[:3, 0, 0, 0] = torch.tensor([3.0, 0.25, -1.0], device=DEV)
    out = pc.pc_attention(q, q, v)   # one key: its value
    assert torch.equal(out, v)


# --- bits of the weights' gradients ---------------------------------------------------

def gradients64(q, k, v, do, kw):
    """dq, dk, dv, dslopes in float64, no lengths."""
    B, Lq, H, D = q.shape
    Hkv = k.shape[2]
    G = H // Hkv
    s = 1 / math.sqrt(D)
    dq, dk, dv = (torch.zeros(t.shape, dtype=torch.float64, device=DEV) for t in (q, k, v))
    ds = torch.zeros(H, dtype=torch.float64, device=DEV)
    for b in range(B):
        d2 = 0.0
        if "slopes" in kw:
            x, y = kw["query_xyz"][b].double(), kw["ref_xyz"][b].double()
            d2 = ((x[:, None] - y[None]) ** 2).sum(-1)
        for h in range(H):
            Q, K, V, g = q[b, :, h].double(), k[b, :, h // G].double(), v[b, :, h // G].double(), \
                do[b, :, h].double()
            z = s * Q @ K.T
            if "slopes" in kw:
                z = z - kw["slopes"][h].double() * d2
            P = torch.softmax(z, 1)
            dP = g @ V.T
            dS = P * (dP - (P * dP).sum(1, keepdim=True))
            dq[b, :, h] = s * dS @ K
            dk[b, :, h // G] += s * dS.T @ Q
            dv[b, :, h // G] += P.T @ g
            ds[h] = ds[h] - (dS * d2).sum()
    return dq, dk, dv, ds


def norm_error(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("Lq,Lk,H,Hkv,D", [(1024, 1024, 4, 2, 64), (600, 700, 2, 1, 40),
                                           (520, 2000, 2, 2, 128), (1500, 513, 2, 1, 96),
                                           (2048, 2048, 2, 2, 64)])
def test_attention_gradients_are_as_exact_as_their_type(Lq, Lk, H, Hkv, D, bias):
    # A result rounded once to bfloat16 is off by 2^-8 / sqrt(3) of its binade, which for
    # normally distributed values is 0.0017 of the norm.  Weights of 8 bits in the sums would add
    # 0.0017 again (0.0024 together); with 16 bits and a flat softmax (delta's error averages
    # out, as the outputs are small) at most a tenth is added.
    q, k, v, do, kw = attn_inputs(1, Lq, Lk, H, Hkv, D, torch.bfloat16, bias, None, None)
    if bias:
        kw["slopes"] = 0.05 * kw["slopes"]
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    got = pc.pc_attention_backward(do, q, k, v, out, lse, **kw)
    for t, w in zip(got[:3], gradients64(q, k, v, do, kw)):
        assert norm_error(t, w) <= 0.0019


# Few keys, or a steep bias: a row's delta is near its largest dP, and what the rounding of the
# output does to it stays in dS whole.
PEAKED = [(8, 2, 2, 4, 2, 64), (4, 16, 16, 4, 4, 64), (2, 64, 64, 4, 2, 64), (2, 65, 33, 2, 1, 36),
          (1, 300, 300, 2, 2, 128), (2, 1, 40, 4, 2, 64), (1, 3, 5000, 2, 2, 128),
          (1, 600, 2000, 1, 1, 64), (1, 40, 2000, 1, 1, 36)]


@pytest.mark.parametrize("steep", [0.0, 4.0, 60.0])
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", PEAKED)
def test_attention_delta_keeps_the_output_s_low_part(B, Lq, Lk, H, Hkv, D, steep):
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, torch.bfloat16, True, None, None)
    kw["slopes"] = torch.full((H,), steep, device=DEV)
    out, lse, low = pc.pc_attention(q, k, v, return_lse=True, return_low=True, **kw)
    got = pc.pc_attention_backward(do, q, k, v, out, lse, out_low=low, **kw)
    ts = [t.clone().requires_grad_() for t in (q, k, v, kw["slopes"])]
    pos = {n: t for n, t in kw.items() if n != "slopes"}
    pc.attention(*ts[:3], slopes=ts[3], **pos).backward(do)
    assert all(torch.equal(t.grad, g) for t, g in zip(ts, got))
    # float32's bounds, and: the weights' two parts (2^-16 twice), the bias through the products
    # (2^-20 slope R^2 of a score, at most 2^-20 * 256), what out + low leaves of the output
    ref = Ref(q, k, v, do, 1 / math.sqrt(D), kw, torch.float32)
    s, P = 1 / math.sqrt(D), 2.0 ** -16
    for b in range(B):
        R2 = float(torch.cat([kw["query_xyz"][b], kw["ref_xyz"][b]]).double().norm(dim=1).max()) ** 2 * 4
        ez = 2 * min(steep * R2, 256.0) * 2.0 ** -20
        for h in range(H):
            kh = h // (H // Hkv)
            Q, K, V, g = (t.double() for t in (q[b, :, h], k[b, :, kh], v[b, :, kh], do[b, :, h]))
            d2 = ((kw["query_xyz"][b].double()[:, None] - kw["ref_xyz"][b].double()[None]) ** 2).sum(-1)
            W = torch.softmax(s * Q @ K.T - steep * d2, 1)
            eO = (ez + 2 * P) * (W @ V.abs())
            dS = W * (g @ V.T - (W * (g @ V.T)).sum(1, keepdim=True))
            edl = ((eO + 2 * P * ref.out[b, :, h].abs()) * g.abs()).sum(1, keepdim=True)
            eS = W * edl + (ez + P) * dS.abs()
            ref.eout[b, :, h] += eO
            ref.edq[b, :, h] += s * eS @ K.abs()
            ref.edk[b, :, kh] += s * eS.T @ Q.abs()
            ref.edv[b, :, kh] += (ez + P) * W.T @ g.abs()
    close(out.double() + low.double(), ref.out, 4 * ref.eout + P * ref.out.abs() + 1e-30, "out + low")
    assert (low.abs().double() <= HALF[torch.bfloat16] * out.abs().double() + 1e-30).all()
    half = HALF[torch.bfloat16]
    # (the tensor cores' sums round with up to 4 units a step where float32's bounds have 1)
    for t, w, err, name in ((got[0], ref.dq, ref.edq, "dq"), (got[1], ref.dk, ref.edk, "dk"),
                            (got[2], ref.dv, ref.edv, "dv")):
        close(t, w, 4 * err + half * w.abs() + 1e-30, name)


def test_attention_low_part_refusals():
    q = torch.zeros(1, 4, 2, 64, device=DEV)
    with pytest.raises(ValueError, match="return_lse"):
        pc.pc_attention(q, q, q, return_low=True)
    out, lse, low = pc.pc_attention(q, q, q, return_lse=True, return_low=True)
    assert low is None      # a float32 output has none
    with pytest.raises(ValueError, match="out_low"):
        pc.pc_attention_backward(q, q, q, q, out, lse, out_low=q)
    b = q.bfloat16()
    out, lse, low = pc.pc_attention(b, b, b, return_lse=True, return_low=True)
    with pytest.raises(ValueError, match="out_low"):
        pc.pc_attention_backward(b, b, b, b, out, lse, out_low=low[:, :2])


@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", PEAKED[1:])
def test_attention_delta_in_norm(B, Lq, Lk, H, Hkv, D):
    # A result rounded once is off by at most 2^-8 / sqrt(3) of its binade in the mean square (and
    # that at its binade's lower end).  What 16 bits of the weights and of the output leave in dS is
    # 2^-16 of P (|out| |dout| + |dP|), at most; the rounded output would leave 2^-9 of it.
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, torch.bfloat16, True, None, None)
    kw["slopes"] = torch.full((H,), 3.0, device=DEV)
    out, lse, low = pc.pc_attention(q, k, v, return_lse=True, return_low=True, **kw)
    got = pc.pc_attention_backward(do, q, k, v, out, lse, out_low=low, **kw)
    want = gradients64(q, k, v, do, kw)
    s, P = 1 / math.sqrt(D), 2.0 ** -16
    edq, edk = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    for b in range(B):
        d2 = torch.cdist(kw["query_xyz"][b].double(), kw["ref_xyz"][b].double()) ** 2
        for h in range(H):
            kh = h // (H // Hkv)
            Q, K, V, g = (t.double() for t in (q[b, :, h], k[b, :, kh], v[b, :, kh], do[b, :, h]))
            W = torch.softmax(s * Q @ K.T - 3.0 * d2, 1)
            eS = P * W * ((W @ V * g).abs().sum(1, keepdim=True) + (g @ V.T).abs())
            edq[b, :, h] = s * eS @ K.abs()
            edk[b, :, kh] += s * eS.T @ Q.abs()
    for t, w, e in zip(got, want, (edq, edk)):
        assert float((t.double() - w).norm()) <= 2.0 ** -8 / math.sqrt(3) * float(w.norm()) + float(e.norm())


@pytest.mark.parametrize("ragged", [True, False])
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", PEAKED)
def test_attention_backward_without_the_low_part_forms_it(B, Lq, Lk, H, Hkv, D, ragged):
    # the plain calls are as exact as those that keep the low part: the same bits
    ql, rl = ([max(Lq - b, 0) for b in range(B)], [max(Lk - 2 * b, 0) for b in range(B)]) \
        if ragged else (None, None)
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, torch.bfloat16, True, ql, rl)
    out, lse, low = pc.pc_attention(q, k, v, return_lse=True, return_low=True, **kw)
    want = pc.pc_attention_backward(do, q, k, v, out, lse, out_low=low, **kw)
    got = pc.pc_attention_backward(do, q, k, v, out, lse, **kw)
    assert all(torch.equal(t, w) for t, w in zip(got, want))
    # and through strided views
    base = torch.cat([t.flatten(2) for t in (k, v)], -1)
    k2, v2 = (t.unflatten(-1, (Hkv, D)) for t in base.split(Hkv * D, -1))
    got = pc.pc_attention_backward(do, q, k2, v2, out, lse, **kw)
    assert all(torch.equal(t, w) for t, w in zip(got, want))


# --- long sums -------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,B,Lq,n,H,Hkv,D", [
    (torch.float32, 1, 2432, 2 ** 17, 8, 8, 64),     # tensor cores, one part a row
    (torch.float32, 1, 1216, 2 ** 16, 8, 8, 128),    # 64 rows a block
    (torch.bfloat16, 1, 2432, 2 ** 17, 8, 8, 64),
    (torch.bfloat16, 40, 20, 2 ** 15, 8, 1, 36),     # float32 instructions
    (torch.float32, 152, 1, 2 ** 15, 8, 8, 4),       # few queries
    (torch.bfloat16, 152, 1, 2 ** 15, 8, 8, 8),
    (torch.float32, 1, 1, 2 ** 17, 1, 1, 64)])       # many parts
def test_attention_slopes_gradient_does_not_lose_with_length(dtype, B, Lq, n, H, Hkv, D):
    # Equal weights 1 / n, one half of the keys at distance^2 c1 with dP = 1, the other at c2 with
    # dP = -1: a row's sum is (c1 - c2) / 2, of n terms of equal size.  One float32 chain of n / 4 of
    # them is off by n / 16 units or so, always to the same side.
    q = torch.zeros(B, Lq, H, D, dtype=dtype, device=DEV)
    k = torch.zeros(B, n, Hkv, D, dtype=dtype, device=DEV)
    v, do = torch.zeros_like(k), torch.zeros_like(q)
    v[:, :n // 2, :, 0], v[:, n // 2:, :, 0], do[..., 0] = 1, -1, 1
    x, y = torch.zeros(B, Lq, 3, device=DEV), torch.zeros(B, n, 3, device=DEV)
    y[:, :n // 2, 0], y[:, n // 2:, 1] = 1.1, 0.7
    kw = dict(slopes=torch.zeros(H, device=DEV), query_xyz=x, ref_xyz=y)
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    assert not out.any()
    ds = pc.pc_attention_backward(do, q, k, v, out, lse, **kw)[3]
    c1, c2 = float(y[0, 0, 0].double() ** 2), float(y[0, -1, 1].double() ** 2)
    # the weight's exponent log2 n through log, times ln 2 and back, and exp2: the same for all;
    # a distance 2 roundings, a product 1; chains of 16 or of a tile's 4, joins of 2^8
    lg = math.log2(n)
    rel = 4 * U * lg * math.log(2) + 2.0 ** -22 + (2 + 1 + 16 + 8) * U
    close(ds, torch.full((H,), -B * Lq * (c1 - c2) / 2, dtype=torch.float64, device=DEV),
          rel * B * Lq * (c1 + c2) / 2, "dslopes")


@pytest.mark.parametrize("steepest", [8.0, 60.0])
@pytest.mark.parametrize("Lq,Lk,H,Hkv,D", [(286, 286, 1, 1, 80), (300, 500, 8, 4, 64),
                                           (1500, 1500, 4, 4, 64), (128, 4000, 4, 2, 128),
                                           (1, 3000, 8, 8, 64), (50, 70, 4, 2, 36)])
def test_attention_slopes_gradient_of_bfloat16_inputs_is_float32(Lq, Lk, H, Hkv, D,
                                                                     steepest):
    # It is float32 though the inputs are not: no further from the definition than one and a half
    # times the elementary form in float32 is, or 1e-6 of it.  (The forward pass forms the bias
    # through the products here, slope R^2 < 256, and its lse is off by 2^-20 slope R^2.)
    q, k, v, do, kw = attn_inputs(1, Lq, Lk, H, Hkv, D, torch.bfloat16, True, None, None)
    for n in ("query_xyz", "ref_xyz"):
        kw[n] = kw[n] / kw[n].norm(dim=-1, keepdim=True)
    if Lq == Lk:
        kw["query_xyz"] = kw["ref_xyz"]
    kw["slopes"] = steepest * 2.0 ** (-8.0 * torch.arange(H, device=DEV) / H)
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    got = pc.pc_attention_backward(do, q, k, v, out, lse, **kw)[3]
    want = gradients64(q, k, v, do, kw)[3]
    d2 = ((kw["query_xyz"][0][:, None] - kw["ref_xyz"][0][None]) ** 2).sum(-1)
    plain = []
    for h in range(H):
        Q, K, V, g = (t.float() for t in (q[0, :, h], k[0, :, h * Hkv // H], v[0, :, h * Hkv // H],
                                          do[0, :, h]))
        P = torch.softmax((Q @ K.T) / math.sqrt(D) - kw["slopes"][h] * d2, 1)
        dP = g @ V.T
        plain.append(-(P * (dP - (P * dP).sum(1, keepdim=True)) * d2).sum())
    error = norm_error(torch.stack(plain), want)
    assert norm_error(got, want) <= max(1.5 * error, 1e-6)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,Lq,Lk,H,D,Hkv", [(8, 900, 900, 1, 100, 1), (6, 1100, 1100, 1, 64, 1),
                                             (24, 1, 900, 2, 64, 2), (8, 40, 600, 1, 128, 1),
                                             (1, 128, 4000, 4, 128, 2)])
def test_attention_slopes_gradient_over_clouds_that_cancel(B, Lq, Lk, H, D, Hkv, dtype):
    # The rows' parts have either sign, so what an lse rounded to float32 does to a row's weights (3e-7
    # of them at lse = 8) is not small against their sum.  As above: one and a half times the
    # elementary form's error, or 1e-6.
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, dtype, True, None, None)
    for n in ("query_xyz", "ref_xyz"):
        kw[n] = kw[n] / kw[n].norm(dim=-1, keepdim=True)
    kw["slopes"] = 8.0 * 2.0 ** (-8.0 * torch.arange(H, device=DEV) / H)
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    got = pc.pc_attention_backward(do, q, k, v, out, lse, **kw)[3]
    want = gradients64(q, k, v, do, kw)[3]
    d2 = ((kw["query_xyz"][:, :, None] - kw["ref_xyz"][:, None]) ** 2).sum(-1)
    plain = []
    for h in range(H):
        Q, K, V, g = (t.float() for t in (q[:, :, h], k[:, :, h * Hkv // H], v[:, :, h * Hkv // H],
                                          do[:, :, h]))
        P = torch.softmax((Q @ K.transpose(1, 2)) / math.sqrt(D) - kw["slopes"][h] * d2, 2)
        dP = g @ V.transpose(1, 2)
        plain.append(-(P * (dP - (P * dP).sum(2, keepdim=True)) * d2).sum())
    error = norm_error(torch.stack(plain), want)
    assert norm_error(got, want) <= max(1.5 * error, 1e-6)


@pytest.mark.parametrize("side", ["out", "dv"])
def test_attention_long_sums_on_the_tensor_cores_have_no_bias(side):
    # The tensor cores cut off what an addition leaves below their accumulator's last place: about
    # 4.4e-7 of a sum of numbers of one sign a tile of 64 rows.  Parts of at most 16,384 streamed
    # rows bound that by 1.2e-4; one chain over 2^18 rows would be off by 1.8e-3.  The mean of the
    # relative errors of many outputs, each rounded to bfloat16 (0.0017 at most, either way), is
    # within 1e-4 of the bias.
    n, rows, H, D = 2 ** 18, 4864 if side == "out" else 2432, 8, 64   # (a block a SM, one part)
    g = gen(70)
    bf = torch.bfloat16
    near_one = lambda *s: (1 + 0.25 * torch.randn(*s, generator=g, device=DEV)).to(bf)  # noqa: E731
    few, many = randn(g, 1, rows, H, D, dtype=bf), randn(g, 1, n, H, D, dtype=bf)
    if side == "out":
        v = near_one(1, n, H, D) * (0.75 + 0.5 * torch.rand(H, D, generator=g, device=DEV)).to(bf)
        got = pc.pc_attention(few, many, v)[0]
        want = torch.stack([torch.softmax(few[0, :, h].double() @ many[0, :, h].double().T / 8, 1)
                            @ v[0, :, h].double() for h in range(2)], 1)
    else:
        do, v = near_one(1, n, H, D), randn(g, 1, rows, H, D, dtype=bf)
        out, lse = pc.pc_attention(many, few, v, return_lse=True)
        got = pc.pc_attention_backward(do, many, few, v, out, lse)[2][0]
        want = torch.zeros(rows, 2, D, dtype=torch.float64, device=DEV)
        for h in range(2):
            K = few[0, :, h].double()
            for i in range(0, n, 32768):
                P = torch.softmax(many[0, i:i + 32768, h].double() @ K.T / 8, 1)
                want[:, h] += P.T @ do[0, i:i + 32768, h].double()
    err = (got[:, :2].double() - want) / want
    assert abs(float(err.mean())) <= 1.2e-4 + 1e-4


# --- second derivatives -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
def test_second_derivatives_raise_or_are_right(dtype):
    g = gen(110)
    x, q = randn(g, 4, 16, dtype=dtype).requires_grad_(), randn(g, 1, 9, 2, 16, dtype=dtype).requires_grad_()
    for y, at in ((pc.layer_norm(x), x), (pc.attention(q, q, q), q)):
        d, = torch.autograd.grad(y.square().sum(), at, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (d.float().square().sum() + at.float().square().sum()).backward()
    pos, f = randn(g, 1, 9, 3), torch.rand(3, 2, generator=g, device=DEV)
    d, = torch.autograd.grad(pc.rotary(q, None, pos, f)[0].square().sum(), q, create_graph=True)
    # |R q|^2 = |q|^2: the gradient is 2 q, its square's 8 q
    dd, = torch.autograd.grad(d.square().sum(), q)
    want = 8 * q.detach().double()
    # four turns, each rounded to the type and 6 units of both channels of a pair
    size = want.abs() + want.unflatten(-1, (-1, 2)).flip(-1).flatten(-2).abs()
    close(dd, want, 5 * (HALF[dtype] + 6 * U) * size, "second derivative")


# --- gradients that are not asked for -----------------------------------------------------

GRAD_SHAPES = [(2, 70, 90, 4, 2, 64), (1, 1, 300, 2, 2, 64), (1, 30, 40, 2, 1, 36),
               (1, 1, 9000, 2, 2, 64), (1, 40, 3000, 1, 1, 128), (2, 0, 5, 2, 1, 64),
               (2, 5, 0, 2, 1, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", GRAD_SHAPES)
def test_attention_backward_of_some_inputs(B, Lq, Lk, H, Hkv, D, dtype):
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, dtype, True, None, None)
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    # (whether the slopes' gradient is asked for chooses how dq's pass forms the bias)
    for slopes in (True, False):
        full = pc.pc_attention_backward(do, q, k, v, out, lse, need_slopes=slopes, **kw)
        for nq in (True, False):
            for nkv in (True, False):
                got = pc.pc_attention_backward(do, q, k, v, out, lse, need_q=nq, need_kv=nkv,
                                               need_slopes=slopes, **kw)
                for t, w, need in zip(got, full, (nq, nkv, nkv, slopes)):
                    assert t is None if not need else torch.equal(t, w)


def test_layer_norm_backward_of_some_parameters():
    g = gen(80)
    x, dy, w, b = randn(g, 300, 96), randn(g, 300, 96), randn(g, 96), randn(g, 96)
    y, mean, rstd = pc.pc_layer_norm(x, w, b, return_stats=True)
    full = pc.pc_layer_norm_backward(dy, x, mean, rstd, w, b)
    for nw in (True, False):
        for nb in (True, False):
            got = pc.pc_layer_norm_backward(dy, x, mean, rstd, w, b, need_weight=nw, need_bias=nb)
            for t, f, need in zip(got, full, (True, nw, nb)):
                assert t is None if not need else torch.equal(t, f)


def test_autograd_of_frozen_inputs():
    g = gen(81)
    q, k, v = (randn(g, 1, 40, 2, 64) for _ in range(3))
    full = [t.clone().requires_grad_() for t in (q, k, v)]
    pc.attention(*full).square().sum().backward()
    for only in range(3):
        ts = [t.clone().requires_grad_(i == only) for i, t in enumerate((q, k, v))]
        pc.attention(*ts).square().sum().backward()
        for i in range(3):
            assert ts[i].grad is None if i != only else torch.equal(ts[i].grad, full[i].grad)
    pos, f = randn(g, 1, 40, 3), torch.rand(3, 10, generator=g, device=DEV)
    a, b = q.clone().requires_grad_(), k.clone().requires_grad_()
    (sum(t.square().sum() for t in pc.rotary(a, b, pos, f))).backward()
    for only in range(2):
        ts = [t.clone().requires_grad_(i == only) for i, t in enumerate((q, k))]
        (sum(t.square().sum() for t in pc.rotary(*ts, pos, f))).backward()
        assert ts[1 - only].grad is None and torch.equal(ts[only].grad, (a, b)[only].grad)


# --- scratch --------------------------------------------------------------------------------

class _Props(ctypes.Structure):          # CUDA_MEM_ALLOC_NODE_PARAMS of the driver
    _fields_ = [("pool", ctypes.c_byte * 88), ("access", ctypes.c_void_p),
                ("accesses", ctypes.c_size_t), ("bytes", ctypes.c_size_t), ("ptr", ctypes.c_uint64)]


def allocations(call, stream):
    """The sizes of the stream-ordered allocations a call makes, from a capture of it."""
    cu = ctypes.CDLL("libcuda.so.1")

    def ok(status):
        assert status == 0, f"driver status {status}"

    s, graph, count, kind = ctypes.c_void_p(stream), ctypes.c_void_p(), ctypes.c_size_t(), ctypes.c_int()
    ok(cu.cuStreamBeginCapture_v2(s, ctypes.c_int(2)))
    try:
        call()
    finally:
        ok(cu.cuStreamEndCapture(s, ctypes.byref(graph)))
    sizes = []
    ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(count)))
    nodes = (ctypes.c_void_p * count.value)()
    ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(count)))
    for n in nodes:
        ok(cu.cuGraphNodeGetType(ctypes.c_void_p(n), ctypes.byref(kind)))
        if kind.value == 10:             # CU_GRAPH_NODE_TYPE_MEM_ALLOC
            p = _Props()
            ok(cu.cuGraphMemAllocNodeGetParams(ctypes.c_void_p(n), ctypes.byref(p)))
            sizes.append(p.bytes)
    ok(cu.cuGraphDestroy(graph))
    return sizes


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [7, 32, 96, 515, 2050, 8192])
def test_layer_norm_backward_scratch_is_bounded(C, dtype):
    # 8 blocks a SM with a row of 2 C float32 each, as the header says
    rows = max(4, 40_000_000 // C // 16)
    x, dy = torch.zeros(rows, C, dtype=dtype, device=DEV), torch.zeros(rows, C, dtype=dtype, device=DEV)
    w, b = torch.ones(C, device=DEV), torch.zeros(C, device=DEV)
    y, mean, rstd = pc.pc_layer_norm(x, w, b, return_stats=True)
    dx, dw, db = pc.pc_layer_norm_backward(dy, x, mean, rstd, w, b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    sizes = allocations(lambda: lib().pc_layer_norm_backward(
        dy.data_ptr(), x.data_ptr(), 0 if dtype is torch.float32 else 1, rows, C, mean.data_ptr(),
        rstd.data_ptr(), w.data_ptr(), 0, dx.data_ptr(), dw.data_ptr(), db.data_ptr(),
        s.cuda_stream), s.cuda_stream)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert len(sizes) == 1 and 0 < sizes[0] <= 8 * sms * 2 * C * 4


# --- the loops' steady state -----------------------------------------------------------

# More rows than the blocks that are resident together take in a round (at most 8 blocks of 4 to 16
# rows a SM, one of 8 for rows of a block), several rounds and a part of one.
@pytest.mark.parametrize("dtype,pdtype", [(torch.float32, torch.float32),
                                          (torch.bfloat16, torch.float32),
                                          (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("shape", [(100_003, 33), (60_001, 96), (20_003, 515), (9_001, 1025),
                                   (9_001, 1024), (5_003, 2051), (4_001, 8192)])
def test_layer_norm_of_many_rounds(shape, dtype, pdtype):
    base.test_layer_norm(shape, dtype, pdtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(7, 33), (20_003, 515), (5_003, 2051)])
def test_layer_norm_of_unaligned_rows(shape, dtype):
    # one element off a vector: an element a load; the same values within the bounds of both
    g = gen(90)
    rows, C = shape
    x, dy = (randn(g, rows * C + 1, dtype=dtype)[1:].view(rows, C) for _ in range(2))
    w, b = randn(g, C) + 1, randn(g, C)
    y, mean, rstd = pc.pc_layer_norm(x, w, b, return_stats=True)
    dx, dw, db = pc.pc_layer_norm_backward(dy, x, mean, rstd, w, b)
    r = base.ln_reference(x, w, b, 1e-5, dy)
    # (rows of mean about 0 and deviation 1: the bounds of the aligned test with |x| rstd <= 8)
    K, half = 64 * U, HALF[dtype]
    exh = (2 * K + 8 * U * 8) * (r["xh"].abs() + 1)
    close(y, r["y"], r["w"].abs() * exh + 4 * U * (r["y"].abs() + r["b"].abs()) + half * r["y"].abs(), "y")
    ga, xa, rs = r["g"].abs(), r["xh"].abs(), r["rstd"].unsqueeze(-1)
    mg, mgx = ga.mean(-1, keepdim=True), (ga * xa).mean(-1, keepdim=True)
    edx = rs * (K * (ga + mg + xa * mgx) + exh * mgx + xa * (ga * exh).mean(-1, keepdim=True))
    close(dx, r["dx"], 2 * edx + half * r["dx"].abs() + 1e-30, "dx")
    da, n = dy.double().abs(), (rows + 64) * U
    close(dw, r["dw"], (da * (exh + n * xa)).sum(0) + U * r["dw"].abs(), "dw")
    close(db, r["db"], n * da.sum(0) + U * r["db"].abs(), "db")


# Enough tokens that a thread goes over five heads and more, several of them in flight; every
# remainder of the pairs by the elements of a vector.
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,L,H,Hkv,D,A,F", [
    (2, 4099, 9, 4, 64, 1, 8), (1, 8201, 9, 4, 64, 1, 9), (3, 6007, 11, 2, 64, 2, 5),
    (1, 20011, 7, 2, 64, 1, 11), (2, 4099, 9, 4, 128, 3, 20), (1, 20011, 5, 0, 64, 1, 13),
    (2, 9001, 13, 0, 64, 2, 15), (1, 20011, 3, 4, 64, 3, 5), (2, 8191, 9, 4, 64, 3, 10)])
def test_rotary_of_many_heads_a_thread(B, L, H, Hkv, D, A, F, interleaved, dtype):
    if Hkv:
        base.test_rotary(B, L, H, Hkv, D, A, F, interleaved, dtype)
        return
    g = gen(B + L)
    q, pos = randn(g, B, L, H, D, dtype=dtype), randn(g, B, L, A)
    freqs = 30 * torch.rand(A, F, generator=g, device=DEV)
    got, none = pc.pc_rotary(q, None, pos, freqs, interleaved=interleaved)
    want, e = base.rotary_reference(q, pos, freqs, interleaved, False)
    assert none is None
    close(got, want, 6 * U * e + HALF[dtype] * want.abs() + 1e-30, "rotary")


# --- attention: both ways to form the bias, both sides long ------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D,ql,rl", [
    (1, 600, 700, 2, 1, 64, None, None), (1, 600, 700, 2, 1, 40, [600], [650]),
    (3, 1024, 1024, 8, 2, 64, [1024, 700, 31], [1024, 700, 31]),
    (2, 1024, 1024, 4, 1, 40, [1024, 513], [1024, 513])])
@pytest.mark.parametrize("bias", [True, False])
def test_attention_both_sides_long(B, Lq, Lk, H, Hkv, D, ql, rl, bias, dtype):
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, dtype, bias, ql, rl)
    base.check_attention(q, k, v, do, kw, dtype)


def spread(B, L, g, most):
    """Points whose distance from the origin grows from 0 to `most` along the cloud."""
    p = randn(g, B, L, 3)
    r = torch.linspace(0, most, L, device=DEV).view(1, L, 1)
    return p / p.norm(dim=-1, keepdim=True) * r


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128, 40])
@pytest.mark.parametrize("most,slope", [(8.0, 10.0), (60.0, 0.3), (3.0, 100.0), (3.0, -5.0)])
@pytest.mark.parametrize("B,Lq,Lk,H,Hkv", [(1, 500, 700, 2, 1), (2, 130, 330, 4, 4)])
def test_attention_tiles_near_and_far(B, Lq, Lk, H, Hkv, D, most, slope, dtype):
    # slope R^2 passes 256 within the cloud: some tiles of a block take the bias through the
    # products, the others from the coordinates' differences (a scene in metres, a steep bias)
    g = gen(100)
    q, k, v, do, kw = attn_inputs(B, Lq, Lk, H, Hkv, D, dtype, True, None, None)
    kw["query_xyz"], kw["ref_xyz"] = spread(B, Lq, g, most), spread(B, Lk, g, most)
    kw["slopes"] = slope * (0.5 + torch.rand(H, generator=g, device=DEV))
    base.check_attention(q, k, v, do, kw, dtype)
    # without the slopes' gradient the pass of dq takes the bias as the others do
    ref = Ref(q, k, v, do, 1 / math.sqrt(D), kw, dtype)
    out, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    dq, dk, dv, ds = pc.pc_attention_backward(do, q, k, v, out, lse, need_slopes=False, **kw)
    assert ds is None
    for t, w, e, name in ((dq, ref.dq, ref.edq, "dq"), (dk, ref.dk, ref.edk, "dk"),
                          (dv, ref.dv, ref.edv, "dv")):
        close(t, w, e + 1e-30, name)


@pytest.mark.parametrize("dtype,D", [(torch.float32, 64), (torch.float32, 128), (torch.bfloat16, 128)])
def test_a_withheld_copy_ends_with_a_status_in_every_kernel(dtype, D):
    # the first block's copies never come: its waits run out, the context stays usable
    q, k, v, do, kw = attn_inputs(2, 200, 200, 2, 2, D, dtype, True, None, None)
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
