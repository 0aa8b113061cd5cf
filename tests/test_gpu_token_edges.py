"""GPU checks of the point-token operators where they are easily wrong: values
that are not finite in valid places, weights and deltas that lose bits, long
sums, and the steady state of the kernels' loops.

Tolerances are derived from the arithmetic as in test_gpu_tokens.py.
"""
import math

import pytest
import torch

import point_cloud_neighbor_gb300 as pc
import test_gpu_tokens as base
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
