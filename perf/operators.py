"""Cases and plain forms of the point-token operators: layer norm, rotary
positions over several axes, and attention with a bias by squared distance.

A case is a dict of plain values.  ``run`` computes it with elementary torch
operations in float32 (``own = False``) or through the package's entry points
(``own = True``); ``exact`` is the definition in float64.
"""
import math

import torch

own = False

DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


# --- cases --------------------------------------------------------------------

def _ln(name, rows, C, dtype, train):
    c = {"op": "layer_norm", "rows": rows, "C": C, "dtype": dtype, "train": train}
    return c if name is None else {"name": name, **c}


def _rope(name, B, L, H, Hkv, D, A, F, dtype, train, interleaved=True):
    c = {"op": "rotary", "B": B, "L": L, "H": H, "Hkv": Hkv, "D": D, "A": A, "F": F,
         "dtype": dtype, "train": train, "interleaved": interleaved}
    return c if name is None else {"name": name, **c}


def _attn(name, B, Lq, Lk, H, Hkv, D, dtype, train, bias=True, ragged=False):
    c = {"op": "attention", "B": B, "Lq": Lq, "Lk": Lk, "H": H, "Hkv": Hkv, "D": D,
         "dtype": dtype, "train": train, "bias": bias, "ragged": ragged}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # 64 sampled centers of a 1024-point cloud, one block's norm while serving: latency
        _ln("ln_fwd_64x384_bf16", 64, 384, "bf16", False),
        # 16 clouds of 1024 tokens, a training step of one norm
        _ln("ln_train_16384x384_bf16", 16384, 384, "bf16", True),
        # a 100,000-point cloud, 512 features with the 3 coordinates appended
        _ln("ln_train_100000x515_f32", 100_000, 515, "f32", True),
        # one new token in each of 32 clouds (a class token, a decoded patch)
        _rope("rope_fwd_32x1_bf16", 32, 1, 8, 8, 64, 3, 10, "bf16", False),
        # 32 clouds grouped into 512 tokens each, 6 heads of 64
        _rope("rope_train_32x512_f32", 32, 512, 6, 6, 64, 3, 10, "f32", True),
        # 16,384 samples of a 1M-point cloud, shared key heads, the half-split pairing
        _rope("rope_train_1x16384_bf16", 1, 16384, 16, 4, 128, 3, 21, "bf16", True, False),
        # one query reads every point of a 100,000-point cloud
        _attn("attn_read_1x100000_bf16", 1, 1, 100_000, 8, 8, 64, "bf16", False),
        # 32 ragged clouds of up to 512 tokens, an encoder's forward pass
        _attn("attn_fwd_32x512_bf16", 32, 512, 512, 6, 6, 64, "bf16", False, ragged=True),
        # 16 ragged clouds of up to 1024 tokens, shared key heads, a training step
        _attn("attn_train_16x1024_bf16", 16, 1024, 1024, 8, 2, 64, "bf16", True, ragged=True),
        # odd lengths and head size in float32, a training step
        _attn("attn_train_4x1021_f32", 4, 1021, 1021, 6, 6, 48, "f32", True),
        # 4096 centers of a 100,000-point cloud, a training step
        _attn("attn_train_1x4096_bf16", 1, 4096, 4096, 16, 4, 128, "bf16", True),
        # 16,384 samples of a 1M-point cloud, forward
        _attn("attn_fwd_1x16384_bf16", 1, 16384, 16384, 8, 8, 128, "bf16", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "rotary", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    train = rng.random() < 0.5
    if op == "layer_norm":
        C = _log(rng, 16, 2048)
        rows = _log(rng, 1, min(131072, 51_000_000 // C))
        return _ln(None, rows, C, dtype, train)
    Hkv = rng.choice([1, 2, 3, 4, 6, 8])
    H = Hkv * rng.choice([1, 1, 2, 4])
    if op == "rotary":
        D = 2 * rng.randint(8, 64)
        A = rng.choice([1, 2, 3, 3])
        F = rng.randint(1, D // 2 // A)
        B = _log(rng, 1, 32)
        most = max(1, min(16384, 16384 * 20 * 128 // (B * (H + Hkv) * D)))
        L = _log(rng, 1, most)
        return _rope(None, B, L, H, Hkv, D, A, F, dtype, train, rng.random() < 0.5)
    D = rng.choice([16, 24, 32, 40, 48, 64, 64, 64, 80, 96, 100, 128, 128])
    B = _log(rng, 1, 32)
    # scores x channels of a pass: at most a fraction of the largest listed case
    most = 2.7e11 / (16 if dtype == "f32" else 2) / (4 if train else 1)
    Lk = _log(rng, 1, min(16384.0, math.sqrt(most / (B * H * D))))
    if rng.random() < 0.25:
        Lq = rng.choice([1, 1, 2, 4])
    elif rng.random() < 0.6:
        Lq = Lk
    else:
        Lq = _log(rng, 1, Lk)
    return _attn(None, B, Lq, Lk, H, Hkv, D, dtype, train, rng.random() < 0.75,
                 rng.random() < 0.5)


# --- inputs -------------------------------------------------------------------

def _points(B, L, g, jitter=0.01):
    """Points near the unit sphere, [B, L, 3] float32."""
    v = torch.randn(B, L, 3, generator=g, device=DEV)
    v = v / v.norm(dim=-1, keepdim=True).clamp_min(1e-6)
    return v + jitter * torch.randn(B, L, 3, generator=g, device=DEV)


def _lengths(B, L, g):
    """Valid points of each cloud, [B] int64: the first is full, the others
    between 1 and L, the last of five or more empty."""
    n = 1 + (torch.rand(B, generator=g, device=DEV) * L).long().clamp_max(L - 1)
    n[0] = L
    if B >= 5:
        n[B - 1] = 0
    return n


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def randn(*shape, s=1.0):
        return (s * torch.randn(*shape, generator=g, device=DEV)).to(t)

    st = {"case": case}
    if case["op"] == "layer_norm":
        rows, C = case["rows"], case["C"]
        shift = torch.randn(C, generator=g, device=DEV)
        st["x"] = (1.5 * torch.randn(rows, C, generator=g, device=DEV) + 0.5 * shift).to(t)
        st["w"] = 1.0 + 0.1 * torch.randn(C, generator=g, device=DEV)
        st["b"] = 0.1 * torch.randn(C, generator=g, device=DEV)
        if case["train"]:
            st["dy"] = randn(rows, C)
        return st
    B, H, Hkv, D = case["B"], case["H"], case["Hkv"], case["D"]
    if case["op"] == "rotary":
        L, A, F = case["L"], case["A"], case["F"]
        st["q"], st["k"] = randn(B, L, H, D), randn(B, L, Hkv, D)
        p = _points(B, L, g)
        st["pos"] = p[..., :A].contiguous()
        # wave lengths from the cloud's diameter down to a 32nd of it
        st["freqs"] = (math.pi * 2.0 ** torch.linspace(0, 5, F, device=DEV)).expand(A, F).contiguous()
        if case["train"]:
            st["dq"], st["dk"] = randn(B, L, H, D), randn(B, L, Hkv, D)
        return st
    Lq, Lk = case["Lq"], case["Lk"]
    st["q"], st["k"], st["v"] = randn(B, Lq, H, D), randn(B, Lk, Hkv, D), randn(B, Lk, Hkv, D)
    if case["train"]:
        st["do"] = randn(B, Lq, H, D)
    kw = {}
    if case["bias"]:
        y = _points(B, Lk, g)
        # the queries are the points themselves or, where there are fewer, centers among them
        kw["query_xyz"] = y if Lq == Lk else y[:, :Lq].contiguous()
        kw["ref_xyz"] = y
        kw["slopes"] = 8.0 * 2.0 ** (-8.0 * torch.arange(H, device=DEV) / H)
    if case["ragged"]:
        n = _lengths(B, Lk, g)
        kw["ref_lengths"] = n
        kw["query_lengths"] = n if Lq == Lk else _lengths(B, Lq, g)
    st["kw"] = kw
    return st


# --- plain forms ----------------------------------------------------------------

def _plain_layer_norm(st):
    t = st["x"].dtype
    x, w, b = st["x"].float(), st["w"], st["b"]
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + 1e-5)
    xhat = xc * rstd
    y = xhat * w + b
    if not st["case"]["train"]:
        return {"y": y.to(t)}
    dy = st["dy"].float()
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    return {"y": y.to(t), "dx": dx.to(t), "dw": (dy * xhat).sum(0), "db": dy.sum(0)}


def _turn(x, c, s, interleaved):
    """x [B, L, h, D] float32 with its pairs turned by (c, s) [B, L, 1, R]; the
    channels beyond the R pairs of an interleaved row, or beyond 2 R of a
    half-split one, stay."""
    R = c.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * R:2], x[..., 1:2 * R:2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :R], x[..., R:2 * R]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, x[..., 2 * R:]], -1)


def _plain_rotary(st):
    t, il = st["q"].dtype, st["case"]["interleaved"]
    angle = (st["pos"].unsqueeze(-1) * st["freqs"]).flatten(-2).unsqueeze(2)
    c, s = angle.cos(), angle.sin()
    out = {"q": _turn(st["q"].float(), c, s, il).to(t), "k": _turn(st["k"].float(), c, s, il).to(t)}
    if st["case"]["train"]:
        out["dq"] = _turn(st["dq"].float(), c, -s, il).to(t)
        out["dk"] = _turn(st["dk"].float(), c, -s, il).to(t)
    return out


def _plain_attention(st):
    t, kw = st["q"].dtype, st["kw"]
    q, k, v = (st[n].float().transpose(1, 2) for n in ("q", "k", "v"))
    B, H, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    G = H // Hkv
    scale = 1.0 / math.sqrt(D)
    k, v = (x.unsqueeze(2).expand(B, Hkv, G, Lk, D).reshape(B, H, Lk, D) for x in (k, v))
    z = (q @ k.transpose(-1, -2)) * scale
    if "slopes" in kw:
        diff = kw["query_xyz"].unsqueeze(2) - kw["ref_xyz"].unsqueeze(1)
        d2 = (diff * diff).sum(-1).unsqueeze(1)
        z = z - kw["slopes"].view(1, H, 1, 1) * d2
    keep = None
    if "ref_lengths" in kw:
        at = torch.arange(Lk, device=q.device)
        keep = (at < kw["ref_lengths"].view(B, 1))[:, None, None, :]
        rows = (torch.arange(Lq, device=q.device) < kw["query_lengths"].view(B, 1))[:, None, :, None]
        keep = keep & rows
        z = z.masked_fill(~keep, -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l == 0, torch.ones_like(l), l)
    o = p @ v
    out = {"o": o.transpose(1, 2).to(t)}
    if not st["case"]["train"]:
        return out
    do = st["do"].float().transpose(1, 2)
    dp = do @ v.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    dv = p.transpose(-1, -2) @ do
    dq = scale * (ds @ k)
    dk = scale * (ds.transpose(-1, -2) @ q)
    out["dq"] = dq.transpose(1, 2).to(t)
    out["dk"] = dk.view(B, Hkv, G, Lk, D).sum(2).transpose(1, 2).to(t)
    out["dv"] = dv.view(B, Hkv, G, Lk, D).sum(2).transpose(1, 2).to(t)
    if "slopes" in kw:
        out["dslopes"] = -(ds * d2).sum((0, 2, 3))
    return out


# --- the package's entry points ---------------------------------------------------

def _own_layer_norm(st):
    import point_cloud_neighbor_gb300 as pc
    if not st["case"]["train"]:
        return {"y": pc.pc_layer_norm(st["x"], st["w"], st["b"], 1e-5)}
    y, mean, rstd = pc.pc_layer_norm(st["x"], st["w"], st["b"], 1e-5, return_stats=True)
    dx, dw, db = pc.pc_layer_norm_backward(st["dy"], st["x"], mean, rstd, st["w"], st["b"])
    return {"y": y, "dx": dx, "dw": dw, "db": db}


def _own_rotary(st):
    import point_cloud_neighbor_gb300 as pc
    il = st["case"]["interleaved"]
    q, k = pc.pc_rotary(st["q"], st["k"], st["pos"], st["freqs"], interleaved=il)
    out = {"q": q, "k": k}
    if st["case"]["train"]:
        out["dq"], out["dk"] = pc.pc_rotary(st["dq"], st["dk"], st["pos"], st["freqs"],
                                            interleaved=il, inverse=True)
    return out


def _own_attention(st):
    import point_cloud_neighbor_gb300 as pc
    q, k, v, kw = st["q"], st["k"], st["v"], st["kw"]
    if not st["case"]["train"]:
        return {"o": pc.pc_attention(q, k, v, **kw)}
    o, lse = pc.pc_attention(q, k, v, return_lse=True, **kw)
    dq, dk, dv, dslopes = pc.pc_attention_backward(st["do"], q, k, v, o, lse, **kw)
    out = {"o": o, "dq": dq, "dk": dk, "dv": dv}
    if "slopes" in kw:
        out["dslopes"] = dslopes
    return out


_PLAIN = {"layer_norm": _plain_layer_norm, "rotary": _plain_rotary, "attention": _plain_attention}
_OWN = {"layer_norm": _own_layer_norm, "rotary": _own_rotary, "attention": _own_attention}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# --- work ---------------------------------------------------------------------------

def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] == "layer_norm":
        n, C = case["rows"] * case["C"], case["C"]
        if not case["train"]:
            return {"bytes": 2 * n * e + 8 * C, "flops": 8 * n}
        return {"bytes": 4 * n * e + 16 * C, "flops": 22 * n}
    B, H, Hkv, D = case["B"], case["H"], case["Hkv"], case["D"]
    if case["op"] == "rotary":
        tok = B * case["L"]
        n, pairs = tok * (H + Hkv) * D, case["A"] * case["F"]
        passes = 2 if case["train"] else 1
        return {"bytes": passes * 2 * n * e + 4 * tok * case["A"] + 4 * pairs,
                "flops": passes * 6 * tok * (H + Hkv) * pairs}
    Lq, Lk = case["Lq"], case["Lk"]
    nq, nk = B * Lq * H * D, B * Lk * Hkv * D
    scores = B * H * Lq * Lk
    if case["ragged"]:
        # lengths are drawn evenly: half of each side on average where there are many clouds
        full = (1 + (B - 1) * 0.25) / B
        half = (1 + (B - 1) * 0.5) / B
        scores, nq, nk = scores * full, nq * half, nk * half
    pos = 12 * B * (Lq + Lk) if case["bias"] else 0
    if not case["train"]:
        return {"bytes": e * (2 * nq + 2 * nk) + pos, "flops": 4 * scores * D}
    return {"bytes": e * (4 * nq + 4 * nk) + pos, "flops": 14 * scores * D}


# --- the definition in 64 bits ----------------------------------------------------------

def exact(case, seed):
    """What run() returns for these inputs, from the definitions in float64."""

    def layer_norm(st):
        x = st["x"].double()
        w, b = st["w"].double(), st["b"].double()
        C = x.shape[1]
        mean = x.sum(1) / C
        var = ((x - mean[:, None]) ** 2).sum(1) / C
        xhat = (x - mean[:, None]) / (var + 1e-5).sqrt()[:, None]
        if not st["case"]["train"]:
            return {"y": w * xhat + b}
        dy = st["dy"].double()
        dxhat = dy * w
        s0, s1 = dxhat.sum(1) / C, (dxhat * xhat).sum(1) / C
        dx = (dxhat - s0[:, None] - xhat * s1[:, None]) / (var + 1e-5).sqrt()[:, None]
        return {"y": w * xhat + b, "dx": dx, "dw": torch.einsum("rc,rc->c", dy, xhat), "db": dy.sum(0)}

    def rotary(st):
        case = st["case"]
        A, F = case["A"], case["F"]
        out = {}
        for name in ("q", "k", "dq", "dk"):
            if name not in st:
                continue
            x, y = st[name].double(), st[name].double().clone()
            sign = -1.0 if name.startswith("d") else 1.0
            for a in range(A):
                for f in range(F):
                    p = a * F + f
                    i, j = (2 * p, 2 * p + 1) if case["interleaved"] else (p, A * F + p)
                    t = (st["pos"][:, :, a].double() * st["freqs"][a, f].double())[:, :, None]
                    y[..., i] = x[..., i] * t.cos() - sign * x[..., j] * t.sin()
                    y[..., j] = x[..., j] * t.cos() + sign * x[..., i] * t.sin()
            out[name] = y
        return out

    def attention(st):
        case, kw = st["case"], st["kw"]
        B, H, Hkv, Lq, Lk, D = (case[n] for n in ("B", "H", "Hkv", "Lq", "Lk", "D"))
        G = H // Hkv
        q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
        out = {"o": torch.zeros_like(q)}
        train = case["train"]
        if train:
            do = st["do"].double()
            out.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
            if "slopes" in kw:
                out["dslopes"] = torch.zeros(H, dtype=torch.float64, device=q.device)
        nq = kw["query_lengths"].tolist() if "query_lengths" in kw else [Lq] * B
        nk = kw["ref_lengths"].tolist() if "ref_lengths" in kw else [Lk] * B
        for b in range(B):
            n = nk[b]
            if n == 0:
                continue
            for i0 in range(0, nq[b], 4096):
                i1 = min(i0 + 4096, nq[b])
                if "slopes" in kw:
                    d2 = torch.zeros(i1 - i0, n, dtype=torch.float64, device=q.device)
                    for a in range(3):
                        x, y = kw["query_xyz"][b, i0:i1, a].double(), kw["ref_xyz"][b, :n, a].double()
                        d2 += (x[:, None] - y[None, :]) ** 2
                for h in range(H):
                    kh, vh = k[b, :n, h // G], v[b, :n, h // G]
                    z = torch.einsum("id,jd->ij", q[b, i0:i1, h], kh) / D ** 0.5
                    if "slopes" in kw:
                        z -= kw["slopes"][h].double() * d2
                    p = torch.softmax(z, 1)
                    del z
                    out["o"][b, i0:i1, h] = p @ vh
                    if not train:
                        continue
                    g = do[b, i0:i1, h]
                    dp = g @ vh.T
                    ds = p * (dp - torch.einsum("ij,ij->i", p, dp)[:, None])
                    out["dv"][b, :n, h // G] += p.T @ g
                    out["dq"][b, i0:i1, h] = ds @ kh / D ** 0.5
                    out["dk"][b, :n, h // G] += ds.T @ q[b, i0:i1, h] / D ** 0.5
                    if "slopes" in kw:
                        out["dslopes"][h] -= torch.einsum("ij,ij->", ds, d2)
        return out

    st = prepare(case, seed)
    return {"layer_norm": layer_norm, "rotary": rotary, "attention": attention}[case["op"]](st)
