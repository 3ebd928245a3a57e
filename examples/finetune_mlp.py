#!/usr/bin/env python3
"""Fine-tunes low-rank adapters beside a frozen W4A4 gated MLP, and serves several of them at once.

One block: norm -> gate and up projection (one W4A4 matmul, adapters beside it) -> gated activation -> down projection
(W4A4, adapters beside it) -> norm, gate and residual -> norm.  The projections' weights stay quantized and fixed; what
the backward pass needs of the activations is kept in 8 bits (act8).  The gradient through a frozen projection is a
plain product with its weights (straight through the quantizers).

    python examples/finetune_mlp.py [--steps 30] [--tokens 512] [--d 512] [--hidden 1024]
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import aware_block_transforms_amd as W                                               # noqa: E402
from aware_block_transforms_amd.layer import (AdapterSet, W4A4Layer, act8_store, request_table)   # noqa: E402

BF = torch.bfloat16


class MlpBlock:
    """The block above for token rows of width d; weights are drawn from the seed."""

    def __init__(self, d, hidden, nad=2, rmax=16, seed=0, device="cuda"):
        r = np.random.default_rng([seed, d, hidden])
        self.d, self.h, self.dev = d, hidden, device
        Wgu = (r.standard_normal((2 * hidden, d)) / np.sqrt(d)).astype(np.float32)
        Wdn = (r.standard_normal((d, hidden)) / np.sqrt(hidden)).astype(np.float32)
        self.gate_up = W4A4Layer("mxfp4", "hadamard", Wgu)
        self.down = W4A4Layer("mxfp4", "hadamard", Wdn)
        self.Wgu, self.Wdn = (torch.from_numpy(w).to(device).to(BF) for w in (Wgu, Wdn))
        self.ad_gu = AdapterSet(nad, rmax, d, 2 * hidden, seed=seed + 1)
        self.ad_dn = AdapterSet(nad, rmax, hidden, d, seed=seed + 2)
        ones = lambda k: torch.ones(k, device=device)  # noqa: E731
        self.w_in, self.w_post, self.w_out, self.scale = ones(d), ones(d), ones(d), ones(d)

    def forward(self, R, requests, train=False):
        """R: bfloat16 [n][d] residual rows.  Returns the next block's input, and what the backward pass reads."""
        n, d, h = R.shape[0], self.d, self.h
        new = lambda *s, dt=BF: torch.empty(s, dtype=dt, device=self.dev)  # noqa: E731
        U = new(n, d)
        W.wush_block_norm(None, None, None, R, self.w_in, None, U)
        GU = self.gate_up.forward(U)
        GU, V1 = self.ad_gu.forward(U, requests, GU, out=GU, keep=True)
        H = new(n, h)
        gc, uc = (new(n, h, dt=torch.int8), new(n, h, dt=torch.int8)) if train else (None, None)
        gs, us = (new(n, h // 32, dt=torch.uint8), new(n, h // 32, dt=torch.uint8)) if train else (None, None)
        W.wush_act8_swiglu(GU[:, :h], GU[:, h:], H, gc, gs, uc, us)
        Y = self.down.forward(H)
        Y, V2 = self.ad_dn.forward(H, requests, Y, out=Y, keep=True)
        Rout, out = new(n, d), new(n, d)
        k1, k2 = new(n, dt=torch.float32), new(n, dt=torch.float32)
        W.wush_block_norm(Y, self.w_post, self.scale, R, self.w_out, Rout, out, k1, k2)
        kept = (act8_store(U), V1, (gc, gs, uc, us), act8_store(H), V2, Y, Rout, k1, k2) if train else None
        return out, kept

    def backward(self, dOut, requests, kept):
        """Gradients of both adapter sets: ((dA, dBt) of gate and up, (dA, dBt) of down)."""
        (u8, us8), V1, (gc, gs, uc, us), (h8, hs8), V2, Y, Rout, k1, k2 = kept
        n, d, h = dOut.shape[0], self.d, self.h
        dY, dscale = torch.empty_like(Y), torch.empty_like(self.scale)
        dwp, dwo = torch.empty_like(self.w_post), torch.empty_like(self.w_out)
        W.wush_block_norm_bwd(dOut, None, Y, self.w_post, self.scale, Rout, self.w_out, k1, k2, dY, None, dscale, dwp,
                              dwo)
        dY = dY.to(BF)
        dH, dA2, dB2 = self.ad_dn.backward(dY, h8, requests, V2, dX0=dY @ self.Wdn, x_scales=hs8)
        dGU = torch.empty((n, 2 * h), dtype=BF, device=self.dev)
        W.wush_act8_swiglu_bwd(dH, gc, gs, uc, us, dGU[:, :h], dGU[:, h:])
        _, dA1, dB1 = self.ad_gu.backward(dGU, u8, requests, V1, x_scales=us8)
        return (dA1, dB1), (dA2, dB2)


def finetune(block, R, target, requests, steps, lr=2e-3, tell=None):
    """Adam on the adapters' factors (fp32 masters); returns the losses."""
    sets = (block.ad_gu, block.ad_dn)
    params = [p.float().requires_grad_() for s in sets for p in (s.A, s.Bt)]
    adam = torch.optim.Adam(params, lr=lr)
    losses = []
    for step in range(steps):
        out, kept = block.forward(R, requests, train=True)
        diff = out.float() - target
        losses.append(float((diff * diff).mean()))
        dOut = (diff * (2.0 / diff.numel())).to(BF)
        grads = [g for pair in block.backward(dOut, requests, kept) for g in pair]
        for p, g in zip(params, grads):
            p.grad = g
        adam.step()
        with torch.no_grad():
            for p, q in zip(params, (t for s in sets for t in (s.A, s.Bt))):
                q.copy_(p)
        if tell:
            tell("step %d loss %.5f" % (step, losses[-1]))
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--d", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1024)
    a = ap.parse_args()
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    block = MlpBlock(a.d, a.hidden)
    R = torch.randn((a.tokens, a.d), generator=g, device="cuda").to(BF)
    target = torch.randn((a.tokens, a.d), generator=g, device="cuda")
    # three sequences: two train an adapter each, the third has none
    third = a.tokens // 3
    requests = request_table([third, third, a.tokens - 2 * third], [0, 1, -1])
    losses = finetune(block, R, target, requests, a.steps, tell=print)
    print("loss %.5f -> %.5f" % (losses[0], losses[-1]))
    # serving: one token of each of eight requests, with either adapter or none, in one pass
    one = request_table([1] * 8, [0, 1, -1, 0, 1, -1, 0, 1])
    out, _ = block.forward(R[:8].contiguous(), one)
    torch.cuda.synchronize()
    print("served 8 requests of one token each:", tuple(out.shape))


if __name__ == "__main__":
    main()
