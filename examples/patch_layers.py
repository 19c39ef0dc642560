"""From uint8 images to the features of an 8-bit patch network, on one GPU.

One batch goes through everything that this package does for it:

  fused_normalize   images -> normalised, augmented fp16 (NHWC)
  rms_norm_q8       patches -> 8-bit codes and a scale per patch
  matmul_q8         codes x 8-bit weights -> the patch embedding
  per layer:        rms_norm_q8 of (branch + residual), matmul_q8 up, GELU,
                    quantize_rows, matmul_q8 down
  rms_norm          the last norm, in fp16, with its backward pass

    python examples/patch_layers.py [--images 64] [--width 384] [--layers 4]

Weights are random: the run shows the calls and compares the features with the
same network in fp32, unquantised.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from augmentation_amd import binding as fn  # noqa: E402
from augmentation_amd import synth  # noqa: E402

PATCH = 16


def patches_of(images: torch.Tensor) -> torch.Tensor:
    """(N, H, W, C) -> (N * H/16 * W/16, 16 * 16 * C), a row per patch."""
    n, h, w, c = images.shape
    x = images.view(n, h // PATCH, PATCH, w // PATCH, PATCH, c)
    return x.permute(0, 1, 3, 2, 4, 5).reshape(-1, PATCH * PATCH * c)


class Network:
    """Random fp16 weights, their 8-bit codes (a scale per output channel) and
    the norms' weights."""

    def __init__(self, width: int, layers: int, channels: int = 3, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        inputs = PATCH * PATCH * channels

        def weight(n, k):
            return (torch.randn(n, k, generator=g) / k ** 0.5).half().cuda()

        self.weights = [weight(width, inputs)]
        for _ in range(layers):
            self.weights += [weight(2 * width, width), weight(width, 2 * width)]
        self.bias = (0.1 * torch.randn(width, generator=g)).cuda()
        self.codes = [fn.quantize_rows(w) for w in self.weights]
        self.norm_in = torch.ones(inputs, dtype=torch.half, device="cuda")
        self.norms = [(1 + 0.1 * torch.randn(width, generator=g)).half().cuda()
                      for _ in range(layers + 1)]

    def product(self, codes, scales, k, bias=None):
        return fn.matmul_q8(codes, scales, *self.codes[k], bias=bias, out_dtype=fn.FN_OUT_FP16)

    def features(self, patches: torch.Tensor):
        """(features, 1/rms, h) of the last norm; h is the stream that the
        layers add to, which every norm updates in place."""
        codes, scales, _ = fn.rms_norm_q8(patches, self.norm_in)
        h = self.product(codes, scales, 0, self.bias)
        branch = torch.zeros_like(h)
        for k in range(len(self.norms) - 1):
            codes, scales, h = fn.rms_norm_q8(branch, self.norms[k], residual=h, sum_out=h)
            up = torch.nn.functional.gelu(self.product(codes, scales, 2 * k + 1))
            branch = self.product(*fn.quantize_rows(up), 2 * k + 2)
        return fn.rms_norm(branch, self.norms[-1], residual=h, sum_out=h)

    def reference(self, patches: torch.Tensor) -> torch.Tensor:
        """The features in fp32, nothing quantised."""
        def norm(x, w):
            return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * w.float()

        w = [v.float() for v in self.weights]
        h = norm(patches.float(), self.norm_in) @ w[0].t() + self.bias
        for k in range(len(self.norms) - 1):
            up = torch.nn.functional.gelu(norm(h, self.norms[k]) @ w[2 * k + 1].t())
            h = h + up @ w[2 * k + 2].t()
        return norm(h, self.norms[-1])


def run(images: int, width: int, layers: int, seed: int = 0):
    """(features, fp32 features, gradients (dh, dweight) of a loss at the
    last norm) of one synthetic batch."""
    w = synth.WORKLOADS["imagenet_train"]
    x = torch.from_numpy(w.make_input()[:images]).cuda()
    pixels = fn.fused_normalize(x, w.mean, w.std, w.flip_p, w.erase_p, w.scale, w.ratio, seed,
                                fn.FN_OUT_FP16)
    patches = patches_of(pixels)
    net = Network(width, layers, seed=seed)
    out, rstd, h = net.features(patches)
    # a loss of the features' squares: its gradient is the features themselves
    dh, dweight = fn.rms_norm_backward(out, h, net.norms[-1], rstd)
    return out, net.reference(patches), (dh, dweight), (net, patches, h, rstd)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--images", type=int, default=64)
    ap.add_argument("--width", type=int, default=384)
    ap.add_argument("--layers", type=int, default=4)
    a = ap.parse_args()
    out, ref, (dh, dweight), (net, patches, _, _) = run(a.images, a.width, a.layers)
    off = ((out.float() - ref).norm() / ref.norm()).item()
    print(f"{a.images} images, {patches.size(0)} patches, width {a.width}, {a.layers} layers: "
          f"8-bit features are {100 * off:.2f}% from fp32; gradient norms {dh.float().norm():.3g}, "
          f"{dweight.norm():.3g}")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        net.features(patches)
    start.record()
    for _ in range(20):
        net.features(patches)
    end.record()
    torch.cuda.synchronize()
    ms = start.elapsed_time(end) / 20
    print(f"{ms:.3f} ms a batch, {a.images / ms * 1000:.0f} images/s through the layers")


if __name__ == "__main__":
    main()
