"""The example that runs the pixel operation and the 8-bit layers together.

A row's quantisation step is its largest value / 127; values spread normally
have a largest value of about four times their rms, so an operand is off by
4 / 127 / sqrt(12) = 0.9% of its norm, a product of two by 1.3%.  Features sum
the embedding and two products per layer in a stream that all add to: with L
layers at most 1.3% sqrt(1 + 2 L), and twice that is allowed for rows whose
largest value is further out."""
from __future__ import annotations

import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import patch_layers
    return patch_layers


@pytest.mark.parametrize("images,width,layers", [(1, 128, 1), (8, 384, 2), (3, 200, 3)])
def test_features_are_near_fp32(example, images, width, layers):
    out, ref, (dh, dweight), (net, patches, h, rstd) = example.run(images, width, layers)
    assert patches.shape == (images * 196, 768)
    assert torch.isfinite(out).all()
    off = ((out.float() - ref).norm() / ref.norm()).item()
    assert off <= 2 * 0.013 * (1 + 2 * layers) ** 0.5, off
    # the gradients of the last norm, by autograd in 64 bits
    x = h.double().requires_grad_()
    w = net.norms[-1].double().requires_grad_()
    y = x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-6) * w
    gx, gw = torch.autograd.grad((y * out.double()).sum(), (x, w))
    assert (dh.double() - gx).norm() <= 2 ** -10 * gx.norm()
    assert (dweight.double() - gw).norm() <= 1e-5 * gw.norm()


def test_layers_in_a_graph(example):
    """The whole network captured once and replayed on new patches."""
    _, _, _, (net, patches, _, _) = example.run(2, 128, 2)
    want = net.features(patches)[0].clone()
    other = patches.flip(0).contiguous()
    want_other = net.features(other)[0].clone()
    fixed = patches.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        net.features(fixed)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = net.features(fixed)[0]
    for k in range(4):
        fixed.copy_(other if k % 2 else patches)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_other if k % 2 else want), k
        net.features(patches)
