"""More than 2^31 gradients of logits in one piece: rows whose gradients begin
beyond 32-bit offsets in elements, in every part of fp32 operands.

dlosses are zero in all rows but some at both ends and in between, so that the
sums over the rows add up exact zeros and as many terms as there are others."""
from __future__ import annotations

import pytest
import torch

from test_gpu_cross_entropy import EXP, U, check_close, gradient, half, head, logits, tiny

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16, torch.float32], ids=str)
def test_more_gradients_than_32_bits_count(fn, t):
    rows, classes, width = 2**23 + 70001, 300, 8  # a piece has 256 classes at least
    x, w, y, b = head(1, rows, classes, width, t)
    losses, lse = fn.linear_cross_entropy(x, w, y, bias=b)
    for first in range(0, rows, 2**19):
        part = slice(first, first + 2**19)
        z, dz = logits(x[part], w, b)
        ref = torch.logsumexp(z, 1)
        off = dz.amax(1) + (EXP + 24 + classes / 16) * U + 2 * U * ref.abs()
        check_close(lse[part], ref, off, "lse")
        yp = y[part]
        ok = (yp >= 0) & (yp < classes)
        at = yp.clamp(0, classes - 1)[:, None]
        want = ref - z.gather(1, at)[:, 0]
        tol = 2 * off + 4 * U * z.gather(1, at)[:, 0].abs()
        check_close(losses[part], torch.where(ok, want, 0.0), torch.where(ok, tol, 1e-300), "losses")
    some = torch.cat([torch.arange(1000), torch.arange(4000, rows, 4099), torch.arange(rows - 1500, rows)]).unique().cuda()
    d = torch.zeros(rows, device="cuda")
    d[some] = torch.rand(some.numel(), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") + 0.5
    d[some[::2]] *= -1
    dx, dw, db = fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b)
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[some] = False
    assert (dx[others] == 0).all()
    xs, ys, n = x[some], y[some], some.numel()
    g, off = gradient(xs, w, ys, b, lse[some], d[some], 0.0)
    rounded = off + (half(t) + 2 * U) * g.abs() * (1 + half(t))
    if t == torch.float16:
        rounded = rounded + tiny(t) * 2.0**-13 * d.abs().max().double()
    ga = g.abs() + rounded
    want = g @ w.double()
    tol = rounded @ w.double().abs() + (classes + 8) * U * (ga @ w.double().abs())
    check_close(dx[some], want, tol * (1 + half(t)) + half(t) * want.abs() + tiny(t), "dx")
    want = g.t().contiguous() @ xs.double()
    tol = rounded.t().contiguous() @ xs.double().abs() + (n + 8) * U * (ga.t().contiguous() @ xs.double().abs())
    check_close(dw, want, tol * (1 + half(t)) + half(t) * want.abs() + tiny(t), "dweight")
    check_close(db, g.sum(0), (off + U * g.abs()).sum(0) + (n + 8) * U * g.abs().sum(0), "dbias")
