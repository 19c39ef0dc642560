"""The linear head's softmax cross entropy and its gradients against their
formulas in 64 bits.

Tolerances.  u = 2^-24 is one fp32 rounding, half = finfo(t).eps / 2 the
rounding to the operands' type.  A logit is a sum of `width` products in fp32,
in any order: off by at most (width + 4) u times the sum of the products'
magnitudes, which is `dz` below.  An exponential is off by a few u relative,
those of its argument's roundings (|z - lse| u) included: EXP u covers |z - lse|
up to 40.  A sum of n numbers is off by at most n u of their magnitudes' sum.
"""
from __future__ import annotations

import pytest
import torch

from conftest import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EXP = 64
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


def half(t) -> float:
    return torch.finfo(t).eps / 2


def tiny(t) -> float:
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def head(seed, rows, classes, width, t, with_bias=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(classes, width, generator=g, device="cuda") / width ** 0.5
    y = torch.randint(0, classes, (rows,), generator=g, device="cuda")
    x = torch.randn(rows, width, generator=g, device="cuda") + 2 * w[y]
    b = torch.randn(classes, generator=g, device="cuda") * 0.5 if with_bias else None
    if rows > 4:
        y[2], y[4] = -100, classes  # ignored, either way
    return x.to(t), w.to(t), y, b


def check_close(got, want, tol, what):
    got, want, tol = got.double(), want.double(), tol.double()
    off = (got - want).abs()
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert bool((off <= tol).all()), f"{what}: {worst:.3g} of its tolerance"


def logits(x, w, b):
    z = x.double() @ w.double().t()
    dz = (x.size(1) + 4) * U * (x.double().abs() @ w.double().abs().t())
    if b is not None:
        z += b.double()
        dz += U * z.abs()
    return z, dz


def check_forward(fn, x, w, y, b, smoothing, **kw):
    losses, lse = fn.linear_cross_entropy(x, w, y, bias=b, smoothing=smoothing, **kw)
    z, dz = logits(x, w, b)
    ref = torch.logsumexp(z, 1)
    p = torch.exp(z - ref[:, None])
    # lse moves by the mean of the logits' errors under p
    off = (p * dz).sum(1) + (EXP + 24 + w.size(0) / 16) * U + 2 * U * ref.abs()
    check_close(lse, ref, off, "lse")
    ok = (y >= 0) & (y < w.size(0))
    at = y.clamp(0, w.size(0) - 1)[:, None]
    want = ref - (1 - smoothing) * z.gather(1, at)[:, 0] - smoothing * z.mean(1)
    tol = off + dz.gather(1, at)[:, 0] + 4 * U * (z.gather(1, at)[:, 0].abs() + ref.abs())
    if smoothing:
        tol = tol + smoothing * (dz.mean(1) + w.size(0) * U * z.abs().mean(1)) + 4 * U * z.mean(1).abs()
    check_close(losses, torch.where(ok, want, 0.0), torch.where(ok, tol, 1e-300), "losses")
    return losses, lse


def gradient(x, w, y, b, lse, dlosses, smoothing):
    """g in 64 bits and what its roundings come to before that to the type."""
    z, dz = logits(x, w, b)
    p = torch.exp(z - lse.double()[:, None])
    ok = ((y >= 0) & (y < w.size(0)))
    g = p - smoothing / w.size(0)
    at = y.clamp(0, w.size(0) - 1)[:, None]
    g.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=torch.float64) * (1 - smoothing))
    d = torch.where(ok, dlosses.double(), 0.0)[:, None]
    off = p * (dz + EXP * U) + 4 * U * (p + smoothing / w.size(0))
    off.scatter_add_(1, at, torch.full_like(at, 4 * U, dtype=torch.float64))
    return g * d, off * d.abs()


def check_backward(fn, x, w, y, b, smoothing, dlosses, lse, **kw):
    t = x.dtype
    dx, dw, db = fn.linear_cross_entropy_backward(dlosses, x, w, y, lse, bias=b, smoothing=smoothing, **kw)
    g, off = gradient(x, w, y, b, lse, dlosses, smoothing)
    gb = off + U * g.abs()
    # g rounded to the type (in fp16 scaled so that the largest dloss has 2^13 at
    # least, where its subnormal numbers begin at 2^-14)
    rounded = off + (half(t) + 2 * U) * g.abs() * (1 + half(t))
    if t == torch.float16:
        rounded = rounded + tiny(t) * 2.0 ** -13 * dlosses.abs().max().double()
    ga = g.abs() + rounded
    if dx is not None:
        want = g @ w.double()
        tol = rounded @ w.double().abs() + (w.size(0) + 8) * U * (ga @ w.double().abs())
        check_close(dx, want, tol * (1 + half(t)) + half(t) * want.abs() + tiny(t), "dx")
    if dw is not None:
        want = g.t().contiguous() @ x.double()
        tol = rounded.t().contiguous() @ x.double().abs() + (x.size(0) + 8) * U * (ga.t().contiguous() @ x.double().abs())
        check_close(dw, want, tol * (1 + half(t)) + half(t) * want.abs() + tiny(t), "dweight")
    if db is not None:
        check_close(db, g.sum(0), gb.sum(0) + (x.size(0) + 8) * U * g.abs().sum(0) + 1e-30, "dbias")
    return dx, dw, db


SIZES = [(1, 1, 1), (1, 10, 8), (3, 7, 5), (1, 1000, 64), (16, 64, 64), (17, 65, 72), (65, 63, 64), (64, 1000, 768),
         (200, 1003, 130), (129, 257, 100), (300, 300, 33), (513, 2000, 96), (64, 5000, 64), (5000, 60, 64),
         (31, 4099, 520), (256, 256, 1), (1030, 1025, 264), (2, 3, 4096), (1500, 4001, 1000), (2048, 2048, 1025)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,classes,width", SIZES)
def test_losses_and_gradients_match_their_formulas(fn, rows, classes, width, t):
    for smoothing, with_bias in ((0.0, False), (0.1, True)):
        x, w, y, b = head(rows + classes, rows, classes, width, t, with_bias)
        _, lse = check_forward(fn, x, w, y, b, smoothing)
        g = torch.Generator(device="cuda").manual_seed(1)
        d = torch.randn(rows, generator=g, device="cuda") * (100 if t == torch.float16 else 1)
        check_backward(fn, x, w, y, b, smoothing, d, lse)


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,classes,width", [(2050, 40001, 64), (3000, 30000, 33)])
def test_classes_in_pieces(fn, rows, classes, width, t):
    """More gradients of logits than a piece holds, operands in place and not."""
    x, w, y, b = head(rows, rows, classes, width, t)
    _, lse = check_forward(fn, x, w, y, b, 0.1)
    check_backward(fn, x, w, y, b, 0.1, torch.full((rows,), 1 / rows, device="cuda"), lse)
