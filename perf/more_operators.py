"""Cases and plain forms of the operators around attention in a network over
point tokens: the gated feed-forward projection, group norm with an activation
over a cloud's valid points, and the lookup of feature rows with its gradient.

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
_EPS = 1e-5


# --- cases --------------------------------------------------------------------

def _glu(name, rows, C, F, act, dtype, train, bias=False):
    c = {"op": "gated_linear", "rows": rows, "C": C, "F": F, "act": act, "dtype": dtype,
         "train": train, "bias": bias}
    return c if name is None else {"name": name, **c}


def _gn(name, B, L, C, G, act, dtype, train, ragged=False):
    c = {"op": "group_norm", "B": B, "L": L, "C": C, "G": G, "act": act, "dtype": dtype,
         "train": train, "ragged": ragged}
    return c if name is None else {"name": name, **c}


def _emb(name, B, T, V, C, dtype, train, ids="even"):
    """B = 0: one table [V, C] and T indices; else a table for each of B clouds and
    T indices into each."""
    c = {"op": "embedding", "B": B, "T": T, "V": V, "C": C, "dtype": dtype, "train": train,
         "ids": ids}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # one new token in each of 32 clouds: latency, bound by the weights
        _glu("glu_fwd_32x384_bf16", 32, 384, 1024, "silu", "bf16", False),
        # 16 clouds of 1024 tokens, a training step of one block's projection
        _glu("glu_train_16384x384_bf16", 16384, 384, 1024, "silu", "bf16", True),
        # every point of a 100,000-point cloud through a wider block, with biases
        _glu("glu_fwd_100000x512_bf16", 100_000, 512, 2048, "gelu", "bf16", False, True),
        # odd numbers of tokens, channels and hidden units in float32, with biases
        _glu("glu_train_4084x387_f32", 4084, 387, 1021, "gelu", "f32", True, True),
        # 32 clouds of 1024 tokens, a large model's block
        _glu("glu_train_32768x1024_bf16", 32768, 1024, 4096, "silu", "bf16", True),
        # 64 sampled centers of one cloud while serving: latency
        _gn("gn_fwd_1x64x384_bf16", 1, 64, 384, 32, "silu", "bf16", False),
        # 16 ragged clouds of up to 1024 points, a training step
        _gn("gn_train_16x1024x384_bf16", 16, 1024, 384, 32, "silu", "bf16", True, True),
        # odd lengths and channels, groups of 15
        _gn("gn_train_4x4093x195_bf16", 4, 4093, 195, 13, "gelu", "bf16", True),
        # one 100,000-point cloud, whose groups reach over all of it
        _gn("gn_train_1x100000x512_f32", 1, 100_000, 512, 32, "silu", "f32", True),
        # category tokens of 512 centers from a small table: latency
        _emb("emb_fwd_512x384_bf16", 0, 512, 40, 384, "bf16", False),
        # 16 clouds: features of 1024 points at 512 centers' 32 neighbours each, some absent
        _emb("emb_train_16x16384x128_bf16", 16, 16384, 1024, 128, "bf16", True, "near"),
        # 500,000 voxel tokens, a few of them very frequent, in a table of 100,000 rows
        _emb("emb_train_500000x256_f32", 0, 500_000, 100_000, 256, "f32", True, "skewed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated_linear", "gated_linear", "group_norm", "embedding"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    train = rng.random() < 0.6
    if op == "gated_linear":
        C = _log(rng, 16, 2048)
        F = int(C * rng.uniform(1.0, 4.0))
        if rng.random() < 0.6:
            C, F = (C + 7) // 8 * 8, (F + 7) // 8 * 8
        # products of a pass: at most a part of the largest listed case
        most = 1.2e11 / (6 if dtype == "f32" else 1)
        rows = _log(rng, 1, max(1.0, min(131072.0, most / (C * F))))
        acts = ["silu", "silu", "gelu", "sigmoid"]
        if not (train and dtype == "f32"):  # (the step of relu's derivative has no error bound)
            acts.append("relu")
        return _glu(None, rows, C, F, rng.choice(acts), dtype, train, rng.random() < 0.4)
    if op == "group_norm":
        G = rng.choice([1, 2, 4, 5, 8, 13, 16, 32, 32])
        C = G * _log(rng, 2, min(64, 2048 // G))
        B = _log(rng, 1, 32)
        # (a group of a few values has hardly a gradient: what is left of it is rounding)
        L = _log(rng, max(1, 32 * G // C), min(131072, 51_000_000 // (B * C)))
        acts = ["none", "silu", "silu", "gelu", "sigmoid"] + ([] if train else ["relu"])
        return _gn(None, B, L, C, G, rng.choice(acts), dtype, train, rng.random() < 0.5)
    C = _log(rng, 8, 1024)
    B = rng.choice([0, 0, _log(rng, 1, 32)])
    n = max(B, 1)
    T = _log(rng, 1, min(524288, 128_000_000 // C) // n)
    V = _log(rng, 1, min(131072, 51_000_000 // C) // n)
    return _emb(None, B, T, V, C, dtype, train, rng.choice(["even", "near", "skewed"]))


# --- inputs -------------------------------------------------------------------

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
    if case["op"] == "gated_linear":
        rows, C, F = case["rows"], case["C"], case["F"]
        st["x"] = randn(rows, C)
        # (a trained layer's sizes: projections of a normalised row have variance about 1.5)
        st["wg"], st["wu"] = randn(F, C, s=1.2 / math.sqrt(C)), randn(F, C, s=1.2 / math.sqrt(C))
        st["bg"] = randn(F, s=0.2) if case["bias"] else None
        st["bu"] = randn(F, s=0.2) if case["bias"] else None
        if case["train"]:
            st["dy"] = randn(rows, F)
        return st
    if case["op"] == "group_norm":
        B, L, C = case["B"], case["L"], case["C"]
        shift = torch.randn(C, generator=g, device=DEV)
        st["x"] = (1.5 * torch.randn(B, L, C, generator=g, device=DEV) + 0.5 * shift).to(t)
        st["w"] = 1.0 + 0.1 * torch.randn(C, generator=g, device=DEV)
        st["b"] = 0.1 * torch.randn(C, generator=g, device=DEV)
        st["lengths"] = _lengths(B, L, g) if case["ragged"] else None
        if case["train"]:
            st["dy"] = randn(B, L, C)
        return st
    B, T, V, C = case["B"], case["T"], case["V"], case["C"]
    shape = (B, T) if B else (T,)
    u = torch.rand(shape, generator=g, device=DEV, dtype=torch.float64)
    if case["ids"] == "skewed":  # density falling as one over the index
        ids = (torch.exp(u * math.log(V + 1.0)) - 1.0).long()
    else:
        ids = (u * V).long()
    ids = ids.clamp_(0, V - 1)
    if case["ids"] == "near":  # neighbours that were not found
        ids[torch.rand(shape, generator=g, device=DEV) < 0.1] = -1
    st["ids"] = ids
    st["table"] = randn(B, V, C) if B else randn(V, C)
    st["scale"] = math.sqrt(C) if case["ids"] == "skewed" else 1.0
    if case["train"]:
        st["dy"] = randn(*shape, C)
    return st


# --- plain forms ----------------------------------------------------------------

def _act(z, act):
    """act(z) and act'(z)."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        p = (z > 0).to(z.dtype)
        return z * p, p
    if act == "gelu":
        c = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * c, c + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    s = 1.0 / (1.0 + torch.exp(-z))
    if act == "sigmoid":
        return s, s * (1.0 - s)
    return z * s, s * (1.0 + z * (1.0 - s))


def _plain_gated_linear(st):
    case, t = st["case"], st["x"].dtype
    x, wg, wu = st["x"].float(), st["wg"].float(), st["wu"].float()
    a, u = x @ wg.T, x @ wu.T
    if case["bias"]:
        a, u = a + st["bg"].float(), u + st["bu"].float()
    f, df = _act(a, case["act"])
    out = {"y": (f * u).to(t)}
    if not case["train"]:
        return out
    dy = st["dy"].float()
    da, du = dy * u * df, dy * f
    out["dx"] = (da @ wg + du @ wu).to(t)
    out["dwg"], out["dwu"] = (da.T @ x).to(t), (du.T @ x).to(t)
    if case["bias"]:
        out["dbg"], out["dbu"] = da.sum(0).to(t), du.sum(0).to(t)
    return out


def _plain_group_norm(st):
    case, t = st["case"], st["x"].dtype
    B, L, C, G = case["B"], case["L"], case["C"], case["G"]
    x = st["x"].float().view(B, L, G, C // G)
    w, b = st["w"].view(G, C // G), st["b"].view(G, C // G)
    keep = None
    n = L * (C // G)
    if st["lengths"] is not None:
        keep = (torch.arange(L, device=x.device) < st["lengths"].view(B, 1)).view(B, L, 1, 1)
        x = torch.where(keep, x, 0.0)
        n = (st["lengths"] * (C // G)).clamp_min(1).view(B, 1, 1, 1).float()
    xc = x - x.sum((1, 3), keepdim=True) / n
    if keep is not None:
        xc = torch.where(keep, xc, 0.0)
    rstd = torch.rsqrt((xc * xc).sum((1, 3), keepdim=True) / n + _EPS)
    xhat = xc * rstd
    f, df = _act(xhat * w + b, case["act"])
    if keep is not None:
        f = torch.where(keep, f, 0.0)
    out = {"y": f.reshape(B, L, C).to(t)}
    if not case["train"]:
        return out
    d = st["dy"].float().view(B, L, G, C // G) * df
    if keep is not None:
        d = torch.where(keep, d, 0.0)
    g = d * w
    dx = rstd * (g - g.sum((1, 3), keepdim=True) / n
                 - xhat * ((g * xhat).sum((1, 3), keepdim=True) / n))
    if keep is not None:
        dx = torch.where(keep, dx, 0.0)
    out["dx"] = dx.reshape(B, L, C).to(t)
    out["dw"], out["db"] = (d * xhat).sum((0, 1)).view(C), d.sum((0, 1)).view(C)
    return out


def _plain_embedding(st):
    case, t = st["case"], st["table"].dtype
    B, V, C = case["B"], case["V"], case["C"]
    ids, n = st["ids"], max(B, 1) * V
    found = (ids >= 0).unsqueeze(-1)
    at = ids.clamp_min(0)
    if B:
        at = at + V * torch.arange(B, device=ids.device).view(B, 1)
    y = torch.where(found, st["table"].view(n, C)[at].float() * st["scale"], 0.0)
    out = {"y": y.to(t)}
    if not case["train"]:
        return out
    dy = torch.where(found, st["dy"].float() * st["scale"], 0.0)
    d = torch.zeros(n, C, device=ids.device).index_add_(0, at.view(-1), dy.view(-1, C))
    out["dtable"] = d.view_as(st["table"]).to(t)
    return out


# --- the package's entry points ---------------------------------------------------

def _own_gated_linear(st):
    import point_cloud_neighbor_gb300 as pc
    case = st["case"]
    args = (st["x"], st["wg"], st["wu"], st["bg"], st["bu"])
    out = {"y": pc.pc_gated_linear(*args, activation=case["act"])}
    if case["train"]:
        out["dx"], out["dwg"], out["dwu"], dbg, dbu = pc.pc_gated_linear_backward(
            st["dy"], *args, activation=case["act"])
        if case["bias"]:
            out["dbg"], out["dbu"] = dbg, dbu
    return out


def _own_group_norm(st):
    import point_cloud_neighbor_gb300 as pc
    case = st["case"]
    kw = {"eps": _EPS, "activation": case["act"], "lengths": st["lengths"]}
    if not case["train"]:
        return {"y": pc.pc_group_norm(st["x"], case["G"], st["w"], st["b"], **kw)}
    y, mean, rstd = pc.pc_group_norm(st["x"], case["G"], st["w"], st["b"], return_stats=True, **kw)
    dx, dw, db = pc.pc_group_norm_backward(st["dy"], st["x"], mean, rstd, case["G"], st["w"],
                                           st["b"], activation=case["act"],
                                           lengths=st["lengths"])
    return {"y": y, "dx": dx, "dw": dw, "db": db}


def _own_embedding(st):
    import point_cloud_neighbor_gb300 as pc
    out = {"y": pc.pc_embedding(st["table"], st["ids"], st["scale"])}
    if st["case"]["train"]:
        out["dtable"] = pc.pc_embedding_backward(st["dy"], st["ids"], st["table"].shape,
                                                 st["scale"])
    return out


_PLAIN = {"gated_linear": _plain_gated_linear, "group_norm": _plain_group_norm,
          "embedding": _plain_embedding}
_OWN = {"gated_linear": _own_gated_linear, "group_norm": _own_group_norm,
        "embedding": _own_embedding}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# --- work ---------------------------------------------------------------------------

def work(case):
    e = _BYTES[case["dtype"]]
    C, train = case["C"], case["train"]
    if case["op"] == "gated_linear":
        M, F = case["rows"], case["F"]
        nw = 2 * F * C + (2 * F if case["bias"] else 0)
        if not train:
            return {"bytes": e * (M * C + nw + M * F), "flops": 4 * M * C * F}
        # x, dy and the weights read; y, dx and the weights' gradients written
        return {"bytes": e * (2 * M * C + 2 * nw + 2 * M * F), "flops": 12 * M * C * F}
    if case["op"] == "group_norm":
        n = case["B"] * case["L"] * C
        if case["ragged"]:  # lengths are drawn evenly; all of the outputs is written
            valid = n * (1 + (case["B"] - 1) * 0.5) / case["B"]
        else:
            valid = n
        if not train:
            return {"bytes": e * (n + valid) + 8 * C, "flops": 12 * valid}
        return {"bytes": e * (2 * n + 2 * valid) + 16 * C, "flops": 36 * valid}
    n = max(case["B"], 1)
    tokens, rows = n * case["T"], n * case["V"]
    nbytes = e * C * (tokens + min(tokens, rows)) + 8 * tokens
    if not train:
        return {"bytes": nbytes, "flops": tokens * C}
    return {"bytes": nbytes + e * C * (tokens + rows), "flops": 3 * tokens * C}


# --- the definition in 64 bits ----------------------------------------------------------

def exact(case, seed):
    """What run() returns for these inputs, from the definitions in float64."""

    def act(z, name):
        # act and its derivative, from the functions' definitions
        if name == "none":
            return z.clone(), torch.full_like(z, 1.0)
        if name == "relu":
            return z.clamp_min(0.0), torch.where(z > 0, 1.0, 0.0).double()
        if name == "gelu":
            cdf = torch.special.ndtr(z)
            return z * cdf, cdf + z * torch.exp(-z ** 2 / 2) / math.sqrt(2 * math.pi)
        s = torch.special.expit(z)
        if name == "sigmoid":
            return s, s - s ** 2
        return z * s, s + z * (s - s ** 2)

    def gated_linear(st):
        x, wg, wu = st["x"].double(), st["wg"].double(), st["wu"].double()
        rows, C = x.shape
        F = wg.shape[0]
        out = {"y": torch.empty(rows, F, dtype=torch.float64, device=x.device)}
        if case["train"]:
            out.update(dx=torch.empty_like(x), dwg=torch.zeros_like(wg), dwu=torch.zeros_like(wu))
            sums = torch.zeros(2, F, dtype=torch.float64, device=x.device)
        for r in range(0, rows, 8192):
            xs = x[r:r + 8192]
            a, u = torch.einsum("rc,fc->rf", xs, wg), torch.einsum("rc,fc->rf", xs, wu)
            if case["bias"]:
                a += st["bg"].double()
                u += st["bu"].double()
            f, df = act(a, case["act"])
            out["y"][r:r + 8192] = f * u
            if case["train"]:
                dy = st["dy"][r:r + 8192].double()
                da, du = dy * u * df, dy * f
                out["dx"][r:r + 8192] = torch.einsum("rf,fc->rc", da, wg)
                out["dx"][r:r + 8192] += torch.einsum("rf,fc->rc", du, wu)
                out["dwg"] += torch.einsum("rf,rc->fc", da, xs)
                out["dwu"] += torch.einsum("rf,rc->fc", du, xs)
                sums += torch.stack([da.sum(0), du.sum(0)])
        if case["train"] and case["bias"]:
            out["dbg"], out["dbu"] = sums[0], sums[1]
        return out

    def group_norm(st):
        B, L, C, G = (case[n] for n in ("B", "L", "C", "G"))
        w, b = st["w"].double(), st["b"].double()
        n = [L] * B if st["lengths"] is None else st["lengths"].tolist()
        names = ("y", "dx") if case["train"] else ("y",)
        out = {k: torch.zeros(B, L, C, dtype=torch.float64, device=w.device) for k in names}
        dw, db = torch.zeros_like(w), torch.zeros_like(w)
        for i in range(B):
            if n[i] == 0:
                continue
            for g in range(G):
                s = slice(g * (C // G), (g + 1) * (C // G))
                x = st["x"][i, :n[i], s].double()
                std = (x.var(unbiased=False) + _EPS).sqrt()
                xhat = (x - x.mean()) / std
                f, df = act(xhat * w[s] + b[s], case["act"])
                out["y"][i, :n[i], s] = f
                if case["train"]:
                    d = st["dy"][i, :n[i], s].double() * df
                    dw[s] += (d * xhat).sum(0)
                    db[s] += d.sum(0)
                    h = d * w[s]
                    out["dx"][i, :n[i], s] = (h - h.mean() - xhat * (h * xhat).mean()) / std
        if case["train"]:
            out["dw"], out["db"] = dw, db
        return out

    def embedding(st):
        B, V, C = case["B"], case["V"], case["C"]
        ids = st["ids"].view(max(B, 1), -1)
        table = st["table"].view(max(B, 1), V, C)
        y = torch.zeros(*ids.shape, C, dtype=torch.float64, device=ids.device)
        d = torch.zeros(max(B, 1), V, C, dtype=torch.float64, device=ids.device)
        for i in range(max(B, 1)):
            there = (ids[i] >= 0).nonzero().squeeze(1)
            y[i, there] = table[i].double().index_select(0, ids[i, there]) * st["scale"]
            if case["train"]:
                dy = st["dy"].view(max(B, 1), -1, C)[i, there].double()
                d[i].index_put_((ids[i, there],), dy * st["scale"], accumulate=True)
        out = {"y": y.view(*st["ids"].shape, C)}
        if case["train"]:
            out["dtable"] = d.view_as(st["table"])
        return out

    st = prepare(case, seed)
    return {"gated_linear": gated_linear, "group_norm": group_norm,
            "embedding": embedding}[case["op"]](st)
