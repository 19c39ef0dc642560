"""A classifier's head trained on the features of the 8-bit patch network, on
one GPU.

  fused_normalize          images -> normalised, augmented fp16
  patch_layers.Network     patches -> features (8-bit, frozen)
  dropout, layer_norm      of the features: dropout, addition to a learned
                           position, norm in one pass
  linear_cross_entropy     the mean feature of an image against the classes, with
                           label smoothing; no logits are kept
  ..._backward             back through the head, the norm and the dropout

    python examples/train_head.py [--images 64] [--classes 1000] [--steps 20]

Images and labels are random: the run shows the calls and that the loss of the
batch falls.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from augmentation_amd import binding as fn  # noqa: E402
from augmentation_amd import synth  # noqa: E402
from examples import patch_layers  # noqa: E402

EPS, SMOOTHING, DROPOUT, LOSS_SCALE = 1e-5, 0.1, 0.1, 1024.0


class Block(torch.autograd.Function):
    """layer_norm(position + dropout(x))."""

    @staticmethod
    def forward(ctx, x, position, weight, bias, seed):
        out, mean, rstd, h = fn.layer_norm(x, weight, bias, EPS, residual=position, p=DROPOUT, seed=seed)
        ctx.save_for_backward(h, weight, mean, rstd)
        ctx.seed = seed
        return out

    @staticmethod
    def backward(ctx, dout):
        h, weight, mean, rstd = ctx.saved_tensors
        dh, dx, dweight, dbias = fn.layer_norm_backward(dout.contiguous(), h, weight, mean, rstd, p=DROPOUT,
                                                        seed=ctx.seed)
        return dx, dh, dweight.to(weight.dtype), dbias.to(weight.dtype), None


class HeadLoss(torch.autograd.Function):
    """The mean cross entropy of a linear head."""

    @staticmethod
    def forward(ctx, x, weight, bias, targets):
        losses, lse = fn.linear_cross_entropy(x, weight, targets, bias=bias, smoothing=SMOOTHING)
        ctx.save_for_backward(x, weight, bias, targets, lse)
        return losses.mean()

    @staticmethod
    def backward(ctx, dloss):
        x, weight, bias, targets, lse = ctx.saved_tensors
        dlosses = (dloss / len(lse)).expand(len(lse))
        dx, dweight, dbias = fn.linear_cross_entropy_backward(dlosses, x, weight, targets, lse, bias=bias,
                                                              smoothing=SMOOTHING)
        return dx, dweight, dbias, None


class Head:
    def __init__(self, tokens: int, width: int, classes: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.position = (0.02 * torch.randn(tokens, width, generator=g)).half().cuda().requires_grad_()
        self.norm_weight = torch.ones(width, dtype=torch.half, device="cuda", requires_grad=True)
        self.norm_bias = torch.zeros(width, dtype=torch.half, device="cuda", requires_grad=True)
        self.weight = (torch.randn(classes, width, generator=g) / width ** 0.5).half().cuda().requires_grad_()
        self.bias = torch.zeros(classes, device="cuda", requires_grad=True)

    def parameters(self):
        return [self.position, self.norm_weight, self.norm_bias, self.weight, self.bias]

    def loss(self, features: torch.Tensor, labels: torch.Tensor, seed: int) -> torch.Tensor:
        """features: (images, tokens, width)."""
        position = self.position.expand_as(features).contiguous()
        pooled = Block.apply(features, position, self.norm_weight, self.norm_bias, seed).mean(1)
        return HeadLoss.apply(pooled, self.weight, self.bias, labels)


def features_of(images: int, width: int, layers: int, seed: int = 0) -> torch.Tensor:
    w = synth.WORKLOADS["imagenet_train"]
    x = torch.from_numpy(w.make_input()[:images]).cuda()
    pixels = fn.fused_normalize(x, w.mean, w.std, w.flip_p, w.erase_p, w.scale, w.ratio, seed, fn.FN_OUT_FP16)
    patches = patch_layers.patches_of(pixels)
    return patch_layers.Network(width, layers, seed=seed).features(patches)[0].view(images, -1, width)


def run(images: int, width: int, layers: int, classes: int, steps: int, seed: int = 0):
    """(losses of the steps, head, features, labels)."""
    features = features_of(images, width, layers, seed)
    labels = torch.randint(0, classes, (images,), generator=torch.Generator().manual_seed(seed)).cuda()
    head = Head(features.size(1), width, classes, seed)
    losses = []
    for step in range(steps):
        loss = head.loss(features, labels, seed=1000 * seed + step)
        (loss * LOSS_SCALE).backward()
        with torch.no_grad():
            for p in head.parameters():
                p -= (0.5 / LOSS_SCALE) * p.grad
                p.grad = None
        losses.append(loss.detach())
    return losses, head, features, labels


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--images", type=int, default=64)
    ap.add_argument("--width", type=int, default=384)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--classes", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    losses, _, features, _ = run(a.images, a.width, a.layers, a.classes, a.steps)
    print(f"{a.images} images, {features.size(1)} patches each, {a.classes} classes: loss "
          + " ".join(f"{x.item():.3f}" for x in losses))


if __name__ == "__main__":
    main()
