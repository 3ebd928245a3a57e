"""Adapters, act8 and block norm in the layers that use them: the layer helpers and the fine-tuning example."""

import os
import sys

import numpy as np
import pytest
import torch

from aware_block_transforms_amd.layer import AdapterSet, W4A4Layer, request_table
from oracle import block_ops as bo
from gpu_util import DEV

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_layer_with_adapters():
    # the layer's own output is unchanged, and the adapters add what the 64-bit form adds to it
    r = np.random.default_rng(3)
    Wt = (r.standard_normal((264, 256)) * 0.06).astype(np.float32)
    layer = W4A4Layer("mxfp4", "hadamard", Wt)
    X = torch.from_numpy(r.standard_normal((40, 256)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    ad = AdapterSet(3, 16, 256, 264, rank=[16, 5, 16], alpha=[1.0, 0.5, 2.0])
    ad.Bt.normal_(0, 0.1)
    lengths, ids = [7, 0, 13, 20], [1, 0, -1, 2]
    base = layer.forward(X)
    Y = layer.forward(X, adapters=ad, requests=request_table(lengths, ids))
    torch.cuda.synchronize()
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    off = np.concatenate(([0], np.cumsum(lengths)))
    ref, mag = bo.adapter_forward(f(X), off, ids, f(ad.A), f(ad.Bt), [16, 5, 16], [1.0, 0.5, 2.0], f(base), 264)
    assert (np.abs(f(Y) - ref[0]) <= (256 + 16 + 32) * 2.0 ** -24 * mag[0]).all()
    assert torch.equal(Y[7:20], base[7:20])


def test_finetuning_lowers_the_loss_of_its_own_requests():
    from finetune_mlp import MlpBlock, finetune
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    block = MlpBlock(256, 512, nad=2)
    R = torch.randn((300, 256), generator=g, device=DEV).to(torch.bfloat16)
    target = torch.randn((300, 256), generator=g, device=DEV)
    req = request_table([100, 100, 100], [0, 1, -1])
    before, _ = block.forward(R, req)
    losses = finetune(block, R, target, req, 25)
    after, _ = block.forward(R, req)
    assert losses[-1] < 0.9 * losses[0], losses
    # the request without an adapter sees the frozen model
    assert torch.equal(before[200:], after[200:])
    assert not torch.equal(before[:100], after[:100])
    # a token served alone gets what it got among the others, up to the order of fp32 sums and one bf16 rounding each
    # of the matmuls' outputs (2^-7 of the row's size at most)
    one, _ = block.forward(R[:3].contiguous(), request_table([1, 1, 1], [0, 0, 0]))
    assert ((one.float() - after[:3].float()).abs() <= 0.05 * after[:3].float().abs().amax(1, keepdim=True)).all()


def test_example_gradients_against_differences():
    # the loss along a direction of the down adapters' factors: its slope, by a centred difference through the whole
    # forward pass, against the backward pass's gradient.  bf16 factors and outputs, 4-bit re-quantized activations and
    # 8-bit checkpoints leave the two within a tenth of the slope.
    from finetune_mlp import MlpBlock
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    block = MlpBlock(256, 512, nad=1)
    R = torch.randn((256, 256), generator=g, device=DEV).to(torch.bfloat16)
    c = torch.randn((256, 256), generator=g, device=DEV)
    req = request_table([256], [0])
    block.ad_dn.Bt.copy_(torch.randn(block.ad_dn.Bt.shape, generator=g, device=DEV) * 0.1)
    out, kept = block.forward(R, req, train=True)
    (_, _), (dA, dB) = block.backward(c.to(torch.bfloat16), req, kept)
    for name, grad in (("A", dA), ("Bt", dB)):
        p = getattr(block.ad_dn, name)
        keep = p.clone()
        v = grad / grad.abs().max() * p.float().abs().mean() * 0.5
        hi = (keep.float() + v).to(torch.bfloat16)
        lo = (keep.float() - v).to(torch.bfloat16)
        loss = []
        for q in (hi, lo):
            p.copy_(q)
            o, _ = block.forward(R, req)
            loss.append(float((o.double() * c.double()).sum()))
        p.copy_(keep)
        want = float((grad.double() * (hi.double() - lo.double())).sum())
        assert abs(loss[0] - loss[1] - want) <= 0.1 * abs(want), (name, loss, want)
