"""Host-side checks of the point-token operators that need no GPU: argument
validation of the C ABI, and the autograd rules over stand-ins of the calls."""
import ctypes

import pytest
import torch

from point_cloud_neighbor_gb300 import build, tokens
from point_cloud_neighbor_gb300.binding import lib

FAKE = ctypes.c_void_p(0x1000)   # never read: the checks come first


@pytest.fixture(scope="module")
def L():
    build.build()
    return lib()


def test_the_output_s_low_part_is_bfloat16_s(L):
    def forward(dtype, low, B=0):
        return L.pc_attention_ex(FAKE, FAKE, FAKE, dtype, B, 4, 4, 2, 1, 64, None, None, None,
                                 0.125, None, None, None, None, None, FAKE, low, None, None)

    def backward(dtype, low):
        return L.pc_attention_backward_ex(FAKE, FAKE, FAKE, FAKE, FAKE, low, FAKE, dtype, 0, 4, 4,
                                          2, 1, 64, None, None, None, 0.125, None, None, None,
                                          None, None, FAKE, FAKE, FAKE, None, None)
    for call in (forward, backward):
        assert call(1, FAKE) == 0 and call(0, None) == 0
        assert call(0, FAKE) == 1
        assert "out_low" in L.pc_last_error_message().decode()


# --- autograd over stand-ins: as the library's calls, they are hidden from autograd -------

def _turned(x, pos, freqs, inverse):
    a = (pos[..., None] * freqs).flatten(-2)[:, :, None]
    R = a.shape[-1]
    c, s = a.cos(), -a.sin() if inverse else a.sin()
    u, v = x[..., 0:2 * R:2], x[..., 1:2 * R:2]
    return torch.cat([torch.stack([u * c - v * s, v * c + u * s], -1).flatten(-2), x[..., 2 * R:]], -1)


@pytest.fixture
def stand_ins(monkeypatch):
    """float64 restatements of the plain calls on CPU tensors; what was asked of each."""
    asked = []

    @torch.no_grad()
    def layer_norm(x, w=None, b=None, eps=1e-5, *, return_stats=False):
        mean, var = x.mean(-1), x.var(-1, unbiased=False)
        rstd = (var + eps).rsqrt()
        y = (x - mean[..., None]) * rstd[..., None]
        y = y * (1 if w is None else w) + (0 if b is None else b)
        return (y, mean, rstd) if return_stats else y

    def layer_norm_backward(g, x, mean, rstd, w=None, b=None, **need):
        asked.append(need)
        with torch.enable_grad():
            ts = [t.detach().requires_grad_() for t in (x, w, b) if t is not None]
            y = torch.nn.functional.layer_norm(ts[0], ts[0].shape[-1:], *ts[1:])
            grads = list(torch.autograd.grad(y, ts, g.detach()))
        return tuple(grads + [None] * (3 - len(grads)))

    @torch.no_grad()
    def rotary(q, k, pos, freqs, *, interleaved=True, inverse=False):
        asked.append((q is not None, k is not None))
        return tuple(None if t is None else _turned(t, pos, freqs, inverse) for t in (q, k))

    def scores(q, k, v):
        p = torch.softmax(torch.einsum("bihd,bjhd->bhij", q, k) / q.shape[-1] ** 0.5, -1)
        return torch.einsum("bhij,bjhd->bihd", p, v)

    @torch.no_grad()
    def attention(q, k, v, **kw):
        return scores(q, k, v), None, None

    def attention_backward(g, q, k, v, out, lse, **kw):
        asked.append({n: x for n, x in kw.items() if n.startswith("need")})
        with torch.enable_grad():
            ts = [t.detach().requires_grad_() for t in (q, k, v)]
            return (*torch.autograd.grad(scores(*ts), ts, g.detach()), None)

    for name, f in (("pc_layer_norm", layer_norm), ("pc_layer_norm_backward", layer_norm_backward),
                    ("pc_rotary", rotary), ("pc_attention", attention),
                    ("pc_attention_backward", attention_backward)):
        monkeypatch.setattr(tokens, name, f)
    return asked


def _leaf(*shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=torch.float64).requires_grad_()


def test_second_derivatives_raise(stand_ins):
    x, w, b = _leaf(3, 8, seed=1), _leaf(8, seed=2), _leaf(8, seed=3)
    q, k, v = (_leaf(1, 4, 2, 8, seed=i) for i in (4, 5, 6))
    for y, at in ((tokens.layer_norm(x, w, b), x), (tokens.attention(q, k, v), q)):
        g, = torch.autograd.grad(y.square().sum(), at, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (g.square().sum() + at.square().sum()).backward()


def test_second_derivatives_of_rotary(stand_ins):
    q, k = _leaf(1, 5, 2, 8, seed=7), _leaf(1, 5, 1, 8, seed=8)
    pos, freqs = _leaf(1, 5, 3, seed=9).detach(), _leaf(3, 1, seed=10).detach()
    results = []
    for turn in (tokens.rotary, lambda q, k, p, f: (_turned(q, p, f, False), _turned(k, p, f, False))):
        a, b = turn(q, k, pos, freqs)
        loss = (a ** 3).sum() + (b ** 2).sum()
        gq, gk = torch.autograd.grad(loss, (q, k), create_graph=True)
        results.append(torch.autograd.grad(gq.pow(2).sum() + gk.pow(3).sum(), (q, k)))
    for got, want in zip(*results):
        assert torch.allclose(got, want, rtol=1e-12, atol=1e-12)
    alone, none = tokens.rotary(q, None, pos, freqs)
    g, = torch.autograd.grad((alone ** 3).sum(), q, create_graph=True)
    assert none is None and g.requires_grad


def test_positions_that_ask_for_a_gradient_are_refused(stand_ins):
    q, pos, freqs = _leaf(1, 5, 2, 8, seed=7), _leaf(1, 5, 3, seed=9), _leaf(3, 1, seed=10)
    for args, name in (((pos, freqs.detach()), "positions"), ((pos.detach(), freqs), "freqs")):
        with pytest.raises(ValueError, match=name):
            tokens.rotary(q, None, *args)
    for name in ("query_xyz", "ref_xyz"):
        kw = dict(query_xyz=pos.detach(), ref_xyz=pos.detach(), slopes=torch.ones(2))
        with pytest.raises(ValueError, match=name):
            tokens.attention(q, q, q, **{**kw, name: pos})
    with torch.no_grad():
        tokens.rotary(q, None, pos, freqs)


def test_only_what_is_asked_for_is_formed(stand_ins):
    x, w, b = _leaf(3, 8, seed=1), _leaf(8, seed=2), _leaf(8, seed=3)
    tokens.layer_norm(x, w.detach(), b).sum().backward()
    assert stand_ins.pop() == {"need_weight": False, "need_bias": True}
    tokens.layer_norm(x, w, b.detach()).sum().backward()
    assert stand_ins.pop() == {"need_weight": True, "need_bias": False}
    q, k, v = (_leaf(1, 4, 2, 8, seed=i) for i in (4, 5, 6))
    tokens.attention(q, k.detach(), v.detach()).sum().backward()
    assert stand_ins.pop() == {"need_slopes": False, "need_q": True, "need_kv": False}
    tokens.attention(q.detach(), k.detach(), v).sum().backward()
    assert stand_ins.pop() == {"need_slopes": False, "need_q": False, "need_kv": True}
    pos, freqs = _leaf(1, 4, 3, seed=9).detach(), _leaf(3, 1, seed=10).detach()
    for i, ts in enumerate(((q.detach(), k), (q, k.detach()))):
        stand_ins.clear()
        ts[1 - i].grad = None
        a, b = tokens.rotary(*ts, pos, freqs)
        ((a ** 2).sum() + (b ** 2).sum()).backward()
        assert stand_ins == [(True, True), (True, False)]   # one turn back, of one tensor
        assert torch.allclose(ts[1 - i].grad, 2 * ts[1 - i].detach())


def test_the_pass_of_a_null_gradient(L):
    def backward(dq, dk, dv, slopes=None, ds=None, Lq=4, Lk=4):
        return L.pc_attention_backward(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 1, Lq, Lk, 2, 1, 64,
                                       None, None, None, 0.125, slopes, slopes, slopes, None, None,
                                       dq, dk, dv, ds, None)
    assert backward(FAKE, FAKE, None) == 1 and backward(FAKE, None, FAKE) == 1
    assert "go together" in L.pc_last_error_message().decode()
    assert backward(None, FAKE, FAKE, FAKE, FAKE) == 1


def test_a_scale_that_float32_does_not_hold_is_refused(L):
    def forward(scale):
        return L.pc_attention(FAKE, FAKE, FAKE, 0, 0, 4, 4, 2, 1, 64, None, None, None, scale, FAKE,
                              FAKE, FAKE, None, None, FAKE, None, None)
    assert forward(1e-30) == 0 and forward(1.0) == 0 and forward(1e30) == 0
    for scale in (1e-50, 1e-39, 2e30, 0.0, float("nan")):
        assert forward(scale) == 1
        assert "scale" in L.pc_last_error_message().decode()


def test_attention_keeps_nothing_where_no_gradient_is_asked(stand_ins, monkeypatch):
    asked, plain = [], tokens.pc_attention

    def attention(q, k, v, **kw):
        asked.append((kw.pop("return_lse", False), kw.pop("return_low", False)))
        out = plain(q, k, v, **kw)
        return out if asked[-1][0] else out[0]

    monkeypatch.setattr(tokens, "pc_attention", attention)
    q, k, v = (_leaf(1, 4, 2, 8, seed=i) for i in (4, 5, 6))
    want = tokens.attention(q, k, v)
    with torch.no_grad():
        a = tokens.attention(q, k, v)
    b = tokens.attention(*(t.detach() for t in (q, k, v)))
    assert asked == [(True, True), (False, False), (False, False)]
    assert want.requires_grad and torch.equal(a, want) and torch.equal(b, want)
