"""Losses whose logits are exact, so that nothing but the formula's own roundings
is left: a head of zero features, whose logits are its bias.

With u = 2^-24, top the largest logit and e_v = exp(z_v - top): the sum of V
numbers e_v, which is 1 or more, is off by (V + EXP) u of itself for the additions
and an exponential's few u, and by V u / 2 for what |z_v - top| adds to those
(|z_v - top| u e_v <= u / e); its logarithm by that and 2 u of its own; top - z_y
and the sum with it by u of each.  No term is as large as the logits."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EXP = 8
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


def zero_head(rows, classes, t):
    return torch.zeros(rows, 16, dtype=t, device="cuda"), torch.zeros(classes, 16, dtype=t, device="cuda")


# one tile that has all classes, and several
@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,classes", [(1, 5), (5, 5), (40, 60), (3, 700), (100, 700), (300, 2000)])
def test_a_loss_keeps_the_digits_that_its_logits_size_would_take(fn, rows, classes, t):
    x, w = zero_head(rows, classes, t)
    g = torch.Generator(device="cuda").manual_seed(classes)
    spread = torch.randn(classes, generator=g, device="cuda").mul(4).round().div(4) - 9
    spread[classes // 3] = 0.0  # the largest: its loss is small
    y = torch.randint(0, classes, (rows,), generator=g, device="cuda")
    y[::2] = classes // 3
    for shift in (0.0, 20.0, 1000.0, -3000.0, 2.0 ** 18):
        z = spread + shift  # exact
        losses, lse = fn.linear_cross_entropy(x, w, y, bias=z)
        ref = torch.logsumexp(z.double(), 0) - z.double()
        total = torch.exp(spread.double()).sum()
        tol = (1.5 * classes + EXP) * U + 2 * U * total.log() + U * (2 * spread.double().abs() + ref)
        assert ((losses.double() - ref[y]).abs() <= tol[y]).all(), shift
        assert ((lse.double() - torch.logsumexp(z.double(), 0)).abs() <= (1.5 * classes + EXP) * U + U * (abs(shift) + 16)).all()


@pytest.mark.parametrize("rows,classes", [(5, 5), (3, 700), (300, 2000)])
def test_a_smoothed_loss_too(fn, rows, classes):
    """The mean of the logits has roundings of its own, of V u of their size: of
    up to 2^8 here, the share 0.25 of which is allowed."""
    x, w = zero_head(rows, classes, torch.float32)
    g = torch.Generator(device="cuda").manual_seed(classes)
    spread = torch.randn(classes, generator=g, device="cuda").mul(4).round().div(4) - 9
    spread[classes // 3] = 0.0
    y = torch.randint(0, classes, (rows,), generator=g, device="cuda")
    for shift in (0.0, 200.0):
        z = spread + shift
        losses, _ = fn.linear_cross_entropy(x, w, y, bias=z, smoothing=0.25)
        zd = z.double()
        ref = torch.logsumexp(zd, 0) - 0.75 * zd - 0.25 * zd.mean()
        total = torch.exp(spread.double()).sum()
        tol = (1.5 * classes + EXP) * U + 2 * U * total.log() + 4 * U * (spread.double().abs() + spread.double().abs().mean() + ref.abs())
        tol = tol + 0.25 * (classes + 2) * U * zd.abs().mean()
        assert ((losses.double() - ref[y]).abs() <= tol[y]).all(), shift


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,classes", [(5, 5), (40, 60), (300, 2000)])
def test_a_class_left_out_of_a_loss_that_is_all_smoothing(fn, rows, classes, t):
    """With smoothing 1 the target's own logit has no part in the loss: whether the
    target is left out or another class, every row's loss is infinite, not NaN, and
    the gradients are p - 1 / V."""
    x, w = zero_head(rows, classes, t)
    b = torch.zeros(classes, device="cuda")
    y = torch.arange(rows, device="cuda") % classes
    losses, lse = fn.linear_cross_entropy(x, w, y, bias=b, smoothing=1.0)
    want = torch.log(torch.tensor(float(classes), dtype=torch.float64)).item()
    assert ((losses.double() - want).abs() <= (1.5 * classes + EXP) * U + 4 * U * want).all()
    b[0] = -float("inf")
    y[-1] = -1  # ignored
    losses, lse = fn.linear_cross_entropy(x, w, y, bias=b, smoothing=1.0)
    assert (losses[:-1] == float("inf")).all() and losses[-1] == 0
    _, _, db = fn.linear_cross_entropy_backward(torch.ones(rows, device="cuda"), x, w, y, lse, bias=b, smoothing=1.0)
    p = torch.full((classes,), 1 / (classes - 1), dtype=torch.float64, device="cuda")
    p[0] = 0
    tol = (rows - 1) * U * ((1.5 * classes + EXP + 4 * want) * p + (rows + 8) / classes)
    assert ((db.double() - (rows - 1) * (p - 1 / classes)).abs() <= tol).all()


@pytest.mark.parametrize("rows,classes,out", [(5, 10, 3), (40, 60, 8), (3, 700, 100), (300, 2000, 1999)])
def test_classes_masked_by_the_lowest_number(fn, rows, classes, out):
    """Several logits of the lowest finite number: their mean is one, though their sum
    is not.  The mean is off by (V + 4) u of the logits' mean size, a loss by that
    share of it and its own few u."""
    x, w = zero_head(rows, classes, torch.float32)
    b = torch.linspace(-1, 1, classes, device="cuda")
    b[:out] = torch.finfo(torch.float32).min
    y = out + torch.arange(rows, device="cuda") % (classes - out)
    for smoothing in (0.0, 0.125):
        losses, lse = fn.linear_cross_entropy(x, w, y, bias=b, smoothing=smoothing)
        bd = b.double()
        ref = torch.logsumexp(bd, 0) - (1 - smoothing) * bd[y] - smoothing * bd.mean()
        tol = (1.5 * classes + EXP + 16) * U + smoothing * (classes + 4) * U * bd.abs().mean() + 8 * U * ref.abs()
        assert torch.isfinite(losses).all() and ((losses.double() - ref).abs() <= tol).all()
        grads = fn.linear_cross_entropy_backward(torch.ones(rows, device="cuda"), x, w, y, lse, bias=b, smoothing=smoothing)
        assert all(torch.isfinite(v).all() for v in grads)
        want = rows * smoothing / classes
        assert ((grads[2][:out].double() + want).abs() <= (rows + 8) * U * want).all()
