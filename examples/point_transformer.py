"""A small transformer over point tokens, from the cloud to a training step and
a single query: farthest point sampling and kNN make the tokens; layer norm,
rotary positions over x, y, z and attention with a distance bias make the
blocks; afterwards one class query reads a whole cloud's tokens.

    python examples/point_transformer.py [--steps 100] [--dtype bf16]

The clouds are ellipsoids of random axes; the model learns the axes' lengths.
Needs a CUDA device; build the library first (python -m
point_cloud_neighbor_gb300.build).
"""
import argparse
import math
import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import point_cloud_neighbor_gb300 as pc  # noqa: E402


def clouds(B, N, generator, device):
    """Points [B, N, 3] on ellipsoids, their half axes [B, 3], and how many of
    the points of each cloud are valid [B] (the others are padding)."""
    axes = 0.25 + torch.rand(B, 3, generator=generator, device=device)
    v = torch.randn(B, N, 3, generator=generator, device=device)
    x = v / v.norm(dim=-1, keepdim=True) * axes[:, None]
    lengths = N - (torch.rand(B, generator=generator, device=device) * N / 4).long()
    return x.contiguous(), axes, lengths


class Norm(nn.Module):
    def __init__(self, C):
        super().__init__()
        self.weight, self.bias = nn.Parameter(torch.ones(C)), nn.Parameter(torch.zeros(C))

    def forward(self, x):
        return pc.layer_norm(x, self.weight, self.bias)


class Block(nn.Module):
    """Pre-norm attention and MLP; H query heads share H // 2 key heads."""

    def __init__(self, C, H):
        super().__init__()
        self.H, self.Hkv, self.D = H, H // 2, C // H
        self.norm1, self.norm2 = Norm(C), Norm(C)
        self.qkv = nn.Linear(C, (H + 2 * self.Hkv) * self.D)
        self.out = nn.Linear(C, C)
        self.mlp = nn.Sequential(nn.Linear(C, 2 * C), nn.GELU(), nn.Linear(2 * C, C))
        self.slopes = nn.Parameter(2.0 ** (1.0 - torch.arange(H)))
        F = self.D // 6  # pairs an axis
        self.register_buffer("freqs", (math.pi * 2.0 ** torch.linspace(0, 4, F)).expand(3, F)
                             .contiguous())

    def project(self, x, centers):
        q, k, v = self.qkv(x).split([n * self.D for n in (self.H, self.Hkv, self.Hkv)], -1)
        q, k, v = (t.unflatten(-1, (-1, self.D)) for t in (q, k, v))  # strided views
        q, k = pc.rotary(q, k, centers, self.freqs)
        return q, k, v

    def forward(self, x, centers, lengths):
        q, k, v = self.project(self.norm1(x), centers)
        o = pc.attention(q, k, v, query_xyz=centers, ref_xyz=centers, slopes=self.slopes,
                         query_lengths=lengths, ref_lengths=lengths)
        x = x + self.out(o.flatten(2))
        return x + self.mlp(self.norm2(x))

    def read(self, query, at, k, v, centers, lengths):
        """One query a cloud against the keys and values kept from ``project``."""
        q = self.qkv(self.norm1(query))[..., :self.H * self.D].unflatten(-1, (-1, self.D))
        q, _ = pc.pc_rotary(q, None, at, self.freqs)
        o = pc.pc_attention(q, k, v, query_xyz=at, ref_xyz=centers, slopes=self.slopes,
                            ref_lengths=lengths)
        return self.out(o.flatten(2))


class PointTransformer(nn.Module):
    def __init__(self, C=96, H=4, depth=2, tokens=64, k=16):
        super().__init__()
        self.tokens, self.k = tokens, k
        self.embed = nn.Sequential(nn.Linear(9, C), nn.GELU(), nn.Linear(C, C))
        self.blocks = nn.ModuleList(Block(C, H) for _ in range(depth))
        self.norm, self.head = Norm(C), nn.Linear(C, 3)

    def group(self, x, lengths):
        """Centers [B, tokens, 3] and the tokens of their neighbourhoods."""
        idx = pc.pc_fps(x, self.tokens)
        centers = x.gather(1, idx[..., None].expand(-1, -1, 3))
        _, near = pc.pc_knn(centers, x, self.k, ref_lengths=lengths)
        points = pc.pc_gather_points(x, near)
        local = torch.cat([points - centers[:, :, None], points, points.abs()], -1)
        return centers, self.embed(local.to(self.head.weight.dtype)).amax(2)

    def forward(self, x, lengths, tokens_valid):
        centers, t = self.group(x, lengths)
        for block in self.blocks:
            t = block(t, centers, tokens_valid)
        keep = (torch.arange(self.tokens, device=x.device) < tokens_valid[:, None])[..., None]
        pooled = self.norm(t).masked_fill(~keep, -math.inf).amax(1)
        return self.head(pooled), centers, t


def train(steps=100, B=32, N=1024, dtype=torch.bfloat16, device="cuda", seed=0):
    """Losses of `steps` steps, and the model with its last batch's tokens."""
    g = torch.Generator(device=device).manual_seed(seed)
    torch.manual_seed(seed)
    model = PointTransformer().to(device)
    master = {n: p.detach().clone() for n, p in model.named_parameters()}
    model.to(dtype)
    for block in model.blocks:  # positions and slopes stay float32
        block.slopes.data = block.slopes.data.float()
        block.freqs = block.freqs.float()
    opt = torch.optim.Adam(list(master.values()), lr=2e-3)
    losses = []
    for _ in range(steps):
        x, axes, lengths = clouds(B, N, g, device)
        valid = torch.full((B,), model.tokens, dtype=torch.int64, device=device)
        valid[::4] = model.tokens * 3 // 4  # some clouds with fewer tokens
        out, centers, t = model(x, lengths, valid)
        loss = (out.float() - axes).square().mean()
        loss.backward()
        for n, p in model.named_parameters():
            master[n].grad = p.grad.float()
            p.grad = None
        opt.step()
        with torch.no_grad():
            for n, p in model.named_parameters():
                p.copy_(master[n])
        losses.append(float(loss.detach()))
    return losses, model, (centers, t.detach(), valid)


@torch.no_grad()
def serve(model, centers, t, valid):
    """A class query at the origin reads the tokens: [B, 1, C]."""
    block = model.blocks[-1]
    _, k, v = block.project(block.norm1(t), centers)
    query = t.mean(1, keepdim=True)
    at = torch.zeros(t.shape[0], 1, 3, device=t.device)
    return block.read(query, at, k, v, centers, valid)


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args()
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    losses, model, last = train(a.steps, dtype=dtype)
    for i, v in enumerate(losses):
        print(f"step {i:3d}  loss {v:.5f}")
    print("class query:", tuple(serve(model, *last).shape))


if __name__ == "__main__":
    main()
