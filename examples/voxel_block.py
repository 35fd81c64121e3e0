"""A voxel-transformer block and its training step, on the library's operators.

    x -> norm -> attention within windows of voxels -> + x -> norm -> submanifold convolution -> + -> out

The voxels of a scene are sorted by window (cubes of --window voxels a side),
so a window is a run of rows and the windows are the packed sets of the
attention; its scores are lowered by slope * distance.  The second norm adds
the residual, writes the convolution's input and, in the same pass, its 8-bit
form: the backward pass keeps only that for the convolution's weight
gradient, and only the 8-bit form of x for the first norm's.  Dense
projections are torch matrix products.

Usage: python examples/voxel_block.py [--steps K] [--channels C] [--heads H]
                                      [--kv-heads G] [--window W] [--scale S]
Trains one block towards a fixed random map of its input (synthetic ring-scan
scene, random features) and prints the loss and the time per step.
"""
import argparse
import os
import sys
import time
from typing import NamedTuple

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from convolution_voxelised_point_amd import synth, ts  # noqa: E402


class Scene(NamedTuple):
    """Voxels sorted by window, the windows' first rows, and the 3x3x3 kernel map."""
    coords: torch.Tensor
    starts: torch.Tensor
    kmap: ts.Kmap

    @classmethod
    def of(cls, coords: np.ndarray, window: int) -> "Scene":
        cell = np.concatenate([coords[:, :1], coords[:, 1:] // window], axis=1)
        order = np.lexsort(cell.T[::-1])
        cell = cell[order]
        first = np.flatnonzero(np.any(cell[1:] != cell[:-1], axis=1)) + 1
        starts = np.concatenate([[0], first, [len(cell)]]).astype(np.int64)
        c = torch.from_numpy(np.ascontiguousarray(coords[order], dtype=np.int32)).cuda()
        return cls(c, torch.from_numpy(starts).cuda(), ts.build_kmap(c, ts.HashTable(c, 2.0), 3, 1, ts.TS_KMAP_PAIRS))


class Params(NamedTuple):
    """Also the gradients, in the same order, in float32."""
    norm1: torch.Tensor  # float32 [c]
    qkv: torch.Tensor    # [c][(hq + 2 hk) d]
    out: torch.Tensor    # [hq d][c]
    norm2: torch.Tensor  # float32 [c]
    conv: torch.Tensor   # [27][c][c]


class Saved(NamedTuple):
    """What the backward pass reads, besides the parameters."""
    x8: ts.Act8
    rstd1: torch.Tensor
    n1: torch.Tensor
    qkv: torch.Tensor
    att: torch.Tensor
    lse: torch.Tensor
    h: torch.Tensor
    rstd2: torch.Tensor
    n2: ts.Act8


class Block:
    def __init__(self, channels: int, heads: int, kv_heads: int):
        self.c, self.hq, self.hk, self.d = channels, heads, kv_heads, channels // heads
        # head h's scores fall by 2^(-8 (h + 1) / heads) per voxel of distance
        self.slopes = torch.exp2(-8.0 * torch.arange(1, heads + 1, device="cuda") / heads)

    def init(self, seed: int) -> Params:
        g = torch.Generator("cuda").manual_seed(seed)

        def normal(*shape, fan):
            return torch.randn(*shape, generator=g, device="cuda") * fan ** -0.5
        c, wide = self.c, (self.hq + 2 * self.hk) * self.d
        return Params(torch.ones(c, device="cuda"), normal(c, wide, fan=c), normal(self.hq * self.d, c, fan=c),
                      torch.ones(c, device="cuda"), normal(27, c, c, fan=9 * c))

    def _heads(self, m: torch.Tensor):
        """q, k, v as columns of one projected matrix: no copies."""
        rows = m.view(m.shape[0], self.hq + 2 * self.hk, self.d)
        return rows.split((self.hq, self.hk, self.hk), dim=1)

    def forward(self, s: Scene, p: Params, x: torch.Tensor):
        """p's matrices in x's type (see typed)."""
        a = ts.norm_fwd(x, p.norm1, h8=True)
        qkv = a.y @ p.qkv
        att, lse = ts.attn_fwd(*self._heads(qkv), s.starts, slopes=self.slopes, q_coords=s.coords)
        b = ts.norm_fwd(att.flatten(1) @ p.out, p.norm2, residual=x, y8=True)
        y = b.h + ts.conv_fwd(s.kmap, b.y, p.conv)
        return y, Saved(a.h8, a.rstd, a.y, qkv, att, lse, b.h, b.rstd, b.y8)

    def backward(self, s: Scene, p: Params, k: Saved, dy: torch.Tensor):
        """(gradient of x, gradients of the parameters)."""
        d_conv = ts.conv_wgrad_act8(s.kmap, k.n2, dy)
        dh, d_norm2 = ts.norm_bwd(ts.conv_dgrad(s.kmap, dy, p.conv), k.h, p.norm2, k.rstd2, dh=dy)
        d_out = torch.mm(k.att.flatten(1).t(), dh)
        d_att = (dh @ p.out.t()).view_as(k.att)
        d_qkv = torch.empty_like(k.qkv)
        ts.attn_bwd(d_att, *self._heads(k.qkv), k.att, k.lse, s.starts, slopes=self.slopes, q_coords=s.coords,
                    into=self._heads(d_qkv))
        d_w = torch.mm(k.n1.t(), d_qkv)
        dx, d_norm1 = ts.norm_bwd(d_qkv @ p.qkv.t(), k.x8, p.norm1, k.rstd1, dh=dh)
        return dx, Params(d_norm1, d_w.float(), d_out.float(), d_norm2, d_conv)


def typed(p: Params, dtype: torch.dtype) -> Params:
    return Params(p.norm1, p.qkv.to(dtype), p.out.to(dtype), p.norm2, p.conv.to(dtype))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--channels", type=int, default=64)
    ap.add_argument("--heads", type=int, default=4)
    ap.add_argument("--kv-heads", type=int, default=2)
    ap.add_argument("--window", type=int, default=16)
    ap.add_argument("--scale", type=float, default=0.2, help="part of the 103k-voxel scene")
    ap.add_argument("--lr", type=float, default=0.05)
    args = ap.parse_args()
    scene = Scene.of(synth.make("lidar", args.scale).coords, args.window)
    n = scene.coords.shape[0]
    block = Block(args.channels, args.heads, args.kv_heads)
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(n, args.channels, generator=g, device="cuda", dtype=torch.bfloat16)
    target, _ = block.forward(scene, typed(block.init(2), x.dtype), x)
    p = block.init(3)
    for step in range(args.steps):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        low = typed(p, x.dtype)
        y, saved = block.forward(scene, low, x)
        diff = y.float() - target.float()
        _, grads = block.backward(scene, low, saved, (diff * (2.0 / args.channels)).to(x.dtype))
        for w, dw in zip(p, grads):
            # the gradients are sums over the voxels
            w.sub_(dw, alpha=args.lr * args.channels / n)
        loss = diff.square().mean().item()
        print(f"step {step:3d}  loss {loss:.4f}  {1e3 * (time.perf_counter() - t0):.2f} ms  ({n} voxels, "
              f"{scene.starts.numel() - 1} windows)", flush=True)


if __name__ == "__main__":
    main()
