"""Whatever a workspace held, whatever stands round an operand's rows: the
results are the same bits.  (A number that only meets a zero would still show, if
it is a NaN.)"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


def dirty(n):
    """n bytes of NaN in every type."""
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def inside(m, left, right, below):
    """m as a range of columns and rows of a buffer full of NaN."""
    rows, width = m.shape
    big = torch.full((rows + below, left + width + right), float("nan"), dtype=m.dtype, device="cuda")
    big[:rows, left:left + width] = m
    return big[:rows, left:left + width]


def same(a, b):
    for p, q in zip(a, b):
        assert torch.equal(p, q) and torch.isfinite(p.float()).all()


# few rows, few and many tiles, odd sizes (copies), pieces of the classes, products
# whose contraction is split, fp32 in parts
SIZES = [(1, 10, 8), (3, 1000, 24), (16, 70000, 64), (17, 65, 72), (64, 1000, 768), (200, 1003, 130),
         (1030, 1025, 264), (2048, 2048, 1025), (700, 130000, 40), (5000, 60, 64), (40, 4000, 4096)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,classes,width", SIZES)
def test_linear_cross_entropy(fn, rows, classes, width, t):
    g = torch.Generator(device="cuda").manual_seed(rows + classes)
    x = torch.randn(rows, width, generator=g, device="cuda").to(t)
    w = (torch.randn(classes, width, generator=g, device="cuda") / width ** 0.5).to(t)
    b = torch.randn(classes, generator=g, device="cuda")
    y = torch.randint(-1, classes, (rows,), generator=g, device="cuda")
    d = torch.rand(rows, generator=g, device="cuda") + 0.5
    want = fn.linear_cross_entropy(x, w, y, bias=b, smoothing=0.1)
    grads = fn.linear_cross_entropy_backward(d, x, w, y, want[1], bias=b, smoothing=0.1)
    assert all(torch.isfinite(v.float()).all() for v in (*want, *grads))
    e = 16 // x.element_size()
    # as they are; in buffers of NaN, read in place if the width allows; off 16 bytes
    for x_, w_ in ((x, w), (inside(x, e, e, 3), inside(w, 2 * e, e, 3)), (inside(x, 1, 2, 1), inside(w, 3, 0, 1))):
        ws = dirty(fn.linear_cross_entropy_workspace(x_, w_).numel())
        got = fn.linear_cross_entropy(x_, w_, y, bias=b, smoothing=0.1, workspace=ws)
        same(got, want)
        ws = dirty(fn.linear_cross_entropy_workspace(x_, w_, True).numel())
        got = fn.linear_cross_entropy_backward(d, x_, w_, y, want[1], bias=b, smoothing=0.1, workspace=ws)
        same(got, grads)


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,width", [(1, 1), (2, 5), (9, 8), (70, 67), (24, 2048), (25, 2560), (6, 4096), (7, 4096),
                                        (5, 8192), (2, 16384), (3, 16384), (300, 770), (3, 16400), (70, 33000)])
def test_layer_norm(fn, rows, width, t):
    g = torch.Generator(device="cuda").manual_seed(rows + width)
    x, r, dout, dsum = (torch.randn(rows, width, generator=g, device="cuda").to(t) for _ in range(4))
    w, b = (torch.randn(width, generator=g, device="cuda").to(t) for _ in range(2))
    forward = dict(residual=r, p=0.2, seed=3)
    want = fn.layer_norm(x, w, b, **forward)
    _, mean, rstd, h = want
    grads = fn.layer_norm_backward(dout, h, w, mean, rstd, dsum=dsum, p=0.2, seed=3)
    assert all(torch.isfinite(v.float()).all() for v in (*want, *grads))
    got = fn.layer_norm(inside(x, 1, 2, 1), w, b, **dict(forward, residual=inside(r, 3, 1, 1)))
    same(got, want)
    ws = dirty(fn.layer_norm_backward_workspace(rows, width).numel())
    got = fn.layer_norm_backward(inside(dout, 1, 1, 1), inside(h, 2, 1, 1), w, mean, rstd, dsum=inside(dsum, 3, 1, 1),
                                 p=0.2, seed=3, workspace=ws)
    same(got, grads)
