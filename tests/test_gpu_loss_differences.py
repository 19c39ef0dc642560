"""The linear cross entropy's gradients against differences of its losses, where
every term of the gradient (probability, target, smoothing) is far larger than
what the differences are off by.

Central differences with a step h are off by h^2 / 6 of the third derivative: that
is the third central moment, under p, of what the step does to the logits, and a
variable of range R has one of sqrt(3) / 18 R^3 at most.  A step in a class's bias
moves that logit by 1, one in w[v, k] by x[t, k], one in x[t, k] all by w[:, k].
And each loss is off by its roundings, E in the weighted sum, which makes E / h."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STEP = 2.0 ** -5


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


@pytest.mark.parametrize("smoothing", [0.0, 0.5, 1.0])
def test_every_term_of_a_gradient_shows(fn, smoothing):
    rows, classes, width = 12, 5, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn(classes, width, generator=g, device="cuda") / width**0.5
    x = torch.randn(rows, width, generator=g, device="cuda")
    b = torch.randn(classes, generator=g, device="cuda") * 0.5
    y = torch.arange(rows, device="cuda") % classes
    y[5] = -100
    m = torch.rand(rows, generator=g, device="cuda") + 0.5

    def loss(x, w, b):
        return (fn.linear_cross_entropy(x, w, y, bias=b, smoothing=smoothing)[0].double() * m.double()).sum().item()

    _, lse = fn.linear_cross_entropy(x, w, y, bias=b, smoothing=smoothing)
    dx, dw, db = fn.linear_cross_entropy_backward(m, x, w, y, lse, bias=b, smoothing=smoothing)
    # a logit: (width + 4) u of its products; a loss: two logits', the sum of the
    # exponentials and its logarithm (5 + 8 + 4), the mean of the logits (5 + 2)
    # of numbers below 8
    size = (x.abs() @ w.abs().t()).amax(1) + b.abs().max() + STEP * x.abs().sum(1) + 1
    each = U * (2 * (width + 4) * size + 17 + 8 * size)
    roundings = ((m * each).sum() / STEP).item()
    assert roundings < 0.01
    moment = 3**0.5 / 18 * STEP**2 / 6
    of_b = moment * m.sum().item() * torch.ones_like(b)
    of_w = moment * (m @ (x.abs() + STEP) ** 3)[None].expand(classes, width)
    spread = w.amax(0) - w.amin(0)
    of_x = moment * m[:, None] * (spread + STEP)[None] ** 3
    # what the gradient itself is rounded by, in rows of size 8 at most
    own = 64 * U * m.sum().item() * 8
    for which, (grad, off) in enumerate(((dx, of_x), (dw, of_w), (db, of_b))):
        leaves = (x, w, b)
        for k in range(grad.numel()):
            ends, places = [], []
            for sign in (1, -1):
                args = [v.clone() for v in leaves]
                args[which].view(-1)[k] += sign * STEP
                places.append(args[which].view(-1)[k].item())  # as fp32 holds it
                ends.append(loss(*args))
            slope = (ends[0] - ends[1]) / (places[0] - places[1])
            tol = 1.01 * (off.reshape(-1)[k].item() + roundings) + own
            assert abs(slope - grad.view(-1)[k].item()) <= tol, (which, k)
    counts = (y >= 0).float() * m
    # the terms that a wrong formula could lack, against what was allowed
    largest = max(v.max().item() for v in (of_x, of_w, of_b)) * 1.01 + roundings * 1.01 + own
    assert largest < 0.02
    if smoothing > 0:
        assert smoothing / classes * counts.sum().item() > 10 * largest
    if smoothing < 1:
        assert (1 - smoothing) * counts[y == 0].sum().item() > 10 * largest
