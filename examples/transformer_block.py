"""Trains one equivariant transformer block on a synthetic periodic cell.

    h        = layer norm by degree of x
    a        = convolution of h over the edges (harmonics, coupling, sum)
    t        = attention over the same edges, q = h, k = v = a, with a learned
               bias from the edge length (beyond the cut-off of a head: masked)
    x', h'   = x + dropout(t), layer norm of it
    energy   = readout: one learned query for each cell attends to its atoms'
               scalars

Every step runs forward and backward through the HIP library.  The targets are
the energies of a second block with other weights; the loss is their mean
square error.

Usage: python examples/transformer_block.py [--steps 30] [--atoms 400] [--channels 32] [--lmax 2]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import spherical_harmonic_cg_amd as eq  # noqa: E402
from spherical_harmonic_cg_amd import autograd as ag  # noqa: E402
from spherical_harmonic_cg_amd import synth  # noqa: E402

CELLS = 4  # graphs in the batch


def batch(atoms, lmax, channels, seed, dev):
    """CELLS periodic cells of `atoms` atoms as one graph: vec, src, row_ptr, x, cell_ptr."""
    rng = np.random.default_rng(seed)
    box = (atoms / synth.DENSITY) ** (1.0 / 3.0)
    r_cut = min(4.0, 0.49 * box)
    vecs, srcs, counts = [], [], []
    for c in range(CELLS):
        pos = rng.uniform(0.0, box, (atoms, 3))
        src, dst = synth.radius_edges(pos, r_cut, box)
        order = np.lexsort((src, dst))
        src, dst = src[order], dst[order]
        d = pos[src] - pos[dst]
        vecs.append(d - box * np.round(d / box))
        srcs.append(src + c * atoms)
        counts.append(np.bincount(dst, minlength=atoms))
    T = lambda a, t: torch.from_numpy(np.ascontiguousarray(a, dtype=t)).to(dev)  # noqa: E731
    ptr = lambda n: np.concatenate([[0], np.cumsum(n)])  # noqa: E731
    x = rng.standard_normal((CELLS * atoms, channels, (lmax + 1) ** 2))
    return dict(vec=T(np.concatenate(vecs), np.float32), src=T(np.concatenate(srcs), np.int32),
                row_ptr=T(ptr(np.concatenate(counts)), np.int32), x=T(x, np.float32),
                cell_ptr=T(ptr([atoms] * CELLS), np.int32), r_cut=r_cut)


class Block(torch.nn.Module):
    def __init__(self, channels, lmax, heads, dev, seed):
        super().__init__()
        g = torch.Generator().manual_seed(seed)
        P = eq.eqtp_num_paths(lmax)
        par = lambda t: torch.nn.Parameter(t.to(dev))  # noqa: E731
        self.lmax, self.heads = lmax, heads
        self.norm_w = torch.nn.ParameterList([par(torch.ones(lmax + 1, channels)) for _ in range(2)])
        self.norm_b = torch.nn.ParameterList([par(torch.zeros(channels)) for _ in range(2)])
        self.conv = par(torch.randn(P, channels, generator=g) / math.sqrt(P))
        self.slope = par(0.3 * torch.randn(heads, generator=g))          # bias = -slope r
        self.query = par(torch.randn(1, channels, generator=g))
        self.value = par(torch.randn(channels, generator=g) / math.sqrt(channels))

    def forward(self, b, plans, rng, p):
        L, H = self.lmax, self.heads
        h = ag.equivariant_layer_norm(b["x"], L, self.norm_w[0], self.norm_b[0])
        a = ag.equivariant_conv(b["vec"], h, self.conv, b["src"], L, row_ptr=b["row_ptr"]) / 8.0
        r = b["vec"].norm(dim=1, keepdim=True)
        reach = b["r_cut"] * (1.0 - 0.1 * torch.arange(H, device=r.device))  # heads see less and less far
        bias = (-self.slope * r).masked_fill(r > reach, -math.inf)
        t = ag.graph_attention(h, a, a, b["src"], b["row_ptr"], L, H, bias=bias, plan=plans[0])
        h, x = ag.dropout_add_norm(t, b["x"], rng, p, L, self.norm_w[1], self.norm_b[1])
        s = h[:, :, 0].contiguous()
        items = torch.arange(s.shape[0], dtype=torch.int32, device=s.device)
        q = self.query.expand(b["cell_ptr"].shape[0] - 1, -1).contiguous()
        pooled = ag.graph_attention(q, s, s, items, b["cell_ptr"], 0, H, plan=plans[1])
        return pooled @ self.value + x[:, :, 0].mean()


def train(steps=30, atoms=400, channels=32, lmax=2, heads=4, p=0.1, seed=0, log=print):
    """Returns the loss of each step."""
    dev = torch.device("cuda")
    b = batch(atoms, lmax, channels, seed, dev)
    items = torch.arange(CELLS * atoms, dtype=torch.int32, device=dev)
    plans = (ag.attention_plan(b["src"], b["row_ptr"], CELLS * atoms), ag.attention_plan(items, b["cell_ptr"], CELLS * atoms))
    teacher, model = (Block(channels, lmax, heads, dev, s) for s in (seed + 1, seed + 2))
    rng = torch.tensor([seed, 0], device=dev)
    with torch.no_grad():
        target = teacher(b, plans, rng, 0.0)
    opt = torch.optim.Adam(model.parameters(), lr=2e-2)
    losses = []
    for step in range(steps):
        opt.zero_grad(set_to_none=True)
        loss = (model(b, plans, rng, p) - target).square().mean()
        loss.backward()
        opt.step()
        rng[1] += 1  # another mask for the next step
        losses.append(float(loss.detach()))
        if log and (step % 10 == 0 or step == steps - 1):
            log("step %3d  loss %.5f" % (step, losses[-1]))
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--atoms", type=int, default=400)
    ap.add_argument("--channels", type=int, default=32)
    ap.add_argument("--lmax", type=int, default=2)
    a = ap.parse_args()
    train(a.steps, a.atoms, a.channels, a.lmax)
