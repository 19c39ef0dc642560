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


def test_large_fp32_products_in_pieces(fn):
    """Operands in three parts, whose pieces are added up."""
    x, w, y, b = head(5, 5000, 10001, 1021, torch.float32)
    _, lse = check_forward(fn, x, w, y, b, 0.1)
    check_backward(fn, x, w, y, b, 0.1, torch.full((5000,), 1 / 5000, device="cuda"), lse)


def test_a_constant_loss_gradient_may_be_expanded(fn):
    x, w, y, b = head(1, 300, 500, 128, torch.bfloat16)
    losses, lse = fn.linear_cross_entropy(x, w, y, bias=b)
    one = torch.full((), 1 / 300, device="cuda")
    for p, q in zip(fn.linear_cross_entropy_backward(one.expand(300), x, w, y, lse, bias=b),
                    fn.linear_cross_entropy_backward(one.repeat(300), x, w, y, lse, bias=b)):
        assert torch.equal(p, q)
    with pytest.raises(ValueError, match="dlosses"):
        fn.linear_cross_entropy_backward(one.repeat(600)[::2], x, w, y, lse, bias=b)


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_what_is_not_wanted_is_not_computed(fn, t):
    for rows, classes, width in ((40, 70, 64), (3000, 30000, 64)):
        x, w, y, b = head(7, rows, classes, width, t)
        _, lse = fn.linear_cross_entropy(x, w, y, bias=b)
        d = torch.full((rows,), 0.5, device="cuda")
        dx, dw, db = fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b)
        only = fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b, want_dweight=False)
        assert torch.equal(only[0], dx) or (only[0].double() - dx.double()).abs().max() <= half(t) * 4 * dx.abs().max()
        assert only[1] is None and torch.equal(only[2], db)
        only = fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b, want_dx=False)
        assert only[0] is None and torch.equal(only[2], db)
        assert (only[1].double() - dw.double()).abs().max() <= half(t) * 4 * dw.abs().max()


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,classes,width", [(20, 100, 40), (300, 1000, 256), (1500, 4001, 1000)])
def test_classes_that_are_left_out(fn, t, rows, classes, width):
    """Bias -infinity: probability 0, gradient of the bias 0 but for the rows that
    want the class; rows that want it lose infinitely; all classes left out: NaN."""
    x, w, y, b = head(3, rows, classes, width, t)
    b[::3] = -float("inf")
    losses, lse = fn.linear_cross_entropy(x, w, y, bias=b)
    keep = torch.arange(classes, device="cuda") % 3 != 0
    z, dz = logits(x, w, b.nan_to_num(neginf=0.0))
    ref = torch.logsumexp(z[:, keep], 1)
    check_close(lse, ref, dz.amax(1) + (EXP + 24 + classes / 16) * U + 2 * U * ref.abs(), "lse")
    ok = (y >= 0) & (y < classes)
    out = ok & (y % 3 == 0)
    assert torch.isinf(losses[out]).all() and (losses[out] > 0).all()
    assert torch.isfinite(losses[ok & ~out]).all() and (losses[~ok] == 0).all()
    d = torch.where(out, 0.0, 1.0)
    dx, dw, db = fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    assert (db[~keep] == 0).all() and (dw[~keep] == 0).all() and (dx[out] == 0).all()
    g, off = gradient(x, w[keep], torch.where(ok & ~out, y - y // 3 - 1, -1), b[keep], lse, d, 0.0)
    check_close(db[keep], g.sum(0), (off + U * g.abs()).sum(0) + (rows + 8) * U * g.abs().sum(0) + 1e-30, "dbias")
    losses, lse = fn.linear_cross_entropy(x, w, y, bias=torch.full_like(b, -float("inf")))
    assert losses[ok].isnan().all() and (losses[~ok] == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,classes,width", [(20, 100, 40), (300, 1000, 256), (1500, 4001, 1000)])
def test_a_bad_row_stays_alone(fn, t, rows, classes, width):
    """A row of NaN features has NaN losses and gradients; an ignored one has none,
    and its gradient is zero.  The other rows do not notice."""
    x, w, y, b = head(5, rows, classes, width, t)
    want = fn.linear_cross_entropy(x, w, y, bias=b)
    bad = x.clone()
    bad[0] = float("nan")
    bad[2] = float("nan")  # ignored
    losses, lse = fn.linear_cross_entropy(bad, w, y, bias=b)
    assert losses[0].isnan() and losses[2] == 0 and lse[0].isnan()
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[0] = others[2] = False
    assert torch.equal(losses[others], want[0][others]) and torch.equal(lse[others], want[1][others])
    d = torch.full((rows,), 0.25, device="cuda")
    dx, _, _ = fn.linear_cross_entropy_backward(d, bad, w, y, lse, bias=b)
    ref, _, _ = fn.linear_cross_entropy_backward(d, x, w, y, want[1], bias=b)
    assert dx[0].isnan().all() and (dx[2] == 0).all() and torch.equal(dx[others], ref[others])
    # a NaN or an infinity among the losses' gradients likewise
    d2 = d.clone()
    d2[0], d2[1] = float("nan"), float("inf")
    dx, _, _ = fn.linear_cross_entropy_backward(d2, x, w, y, want[1], bias=b)
    assert dx[0].isnan().all() and not torch.isfinite(dx[1]).any()
    assert torch.equal(dx[2:], ref[2:])
    # and gradients of zero are zero
    dx, dw, db = fn.linear_cross_entropy_backward(d * 0, x, w, y, want[1], bias=b)
    assert (dx == 0).all() and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_small_and_large_loss_gradients(fn, t):
    """The results are linear in dlosses over the type's whole range."""
    x, w, y, b = head(9, 100, 300, 64, t)
    _, lse = fn.linear_cross_entropy(x, w, y, bias=b)
    one = torch.ones(100, device="cuda")
    dx, dw, db = fn.linear_cross_entropy_backward(one, x, w, y, lse, bias=b)
    for k in (-20, 3) if t == torch.float16 else (-60, 40):
        a, c, e = fn.linear_cross_entropy_backward(one * 2.0 ** k, x, w, y, lse, bias=b)
        scale = 2.0 ** k
        check_close(a, dx.double() * scale, half(t) * 2.01 * dx.abs().double() * scale + tiny(t) * (1 + scale), "dx")
        check_close(c, dw.double() * scale, half(t) * 2.01 * dw.abs().double() * scale + tiny(t) * (1 + scale), "dweight")
        check_close(e, db.double() * scale, 4 * U * db.abs().double() * scale + 1e-40, "dbias")


def test_gradients_are_those_of_differences(fn):
    """Central differences of the summed losses in fp32, as in the formula: a step
    of 2^-6 leaves a third-order error below 2^-12 of the logits' slopes, the
    losses' roundings 12 rows x 2^-22 / 2^-5."""
    rows, classes, width = 12, 37, 24
    x, w, y, b = head(2, rows, classes, width, torch.float32)
    m = torch.randn(rows, generator=torch.Generator().manual_seed(1)).cuda()

    def loss(x, w, b):
        return (fn.linear_cross_entropy(x, w, y, bias=b, smoothing=0.1)[0].double() * m.double()).sum()

    _, lse = fn.linear_cross_entropy(x, w, y, bias=b, smoothing=0.1)
    grads = fn.linear_cross_entropy_backward(m, x, w, y, lse, bias=b, smoothing=0.1)
    step = 2.0 ** -6
    for which, grad in enumerate(grads):
        flat = (x, w, b)[which].flatten()
        for k in range(0, flat.numel(), 11):
            ends = []
            for sign in (1, -1):
                moved = flat.clone()
                moved[k] += sign * step
                args = [x, w, b]
                args[which] = moved.view_as(args[which])
                ends.append(loss(*args).item())
            slope = (ends[0] - ends[1]) / (2 * step)
            assert abs(slope - grad.flatten()[k].item()) <= 2.0 ** -9 * 6, (which, k)


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,classes,width", [(9, 77, 40), (70, 1003, 130), (16, 40000, 64), (700, 3000, 512), (2050, 40001, 64)])
def test_strides_places_and_guards(fn, t, rows, classes, width):
    """Operands that start anywhere give what aligned ones give, up to the order
    of their sums' roundings; nothing is written beside the outputs."""
    x, w, y, b = head(rows, rows, classes, width, t)
    losses, lse = fn.linear_cross_entropy(x, w, y, bias=b)
    d = torch.full((rows,), 1 / rows, device="cuda")
    ref = fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b)
    wide_x = torch.full((rows, width + 13), 7.0, dtype=t, device="cuda")
    wide_w = torch.full((classes, width + 9), 7.0, dtype=t, device="cuda")
    xs, ws = wide_x[:, 5:5 + width], wide_w[:, 3:3 + width]
    xs.copy_(x)
    ws.copy_(w)
    got, got_lse = check_forward(fn, xs, ws, y, b, 0.0)
    dxs = torch.full((rows, width + 5), 7.0, dtype=t, device="cuda")
    dws = torch.full((classes, width + 7), 7.0, dtype=t, device="cuda")
    dx, dw, db = check_backward(fn, xs, ws, y, b, 0.0, d, lse, dx=dxs[:, 1:1 + width], dweight=dws[:, 4:4 + width])
    assert (dxs[:, :1] == 7).all() and (dxs[:, 1 + width:] == 7).all()
    assert (dws[:, :4] == 7).all() and (dws[:, 4 + width:] == 7).all()
    assert (wide_x[:, :5] == 7).all() and (wide_x[:, 5 + width:] == 7).all() and torch.equal(xs, x)
    # aligned views: the same bits as their copies
    if width * t.itemsize % 16 == 0:
        pad = 16 // t.itemsize
        wide = torch.full((rows, width + 2 * pad), 7.0, dtype=t, device="cuda")
        wide[:, pad:pad + width] = x
        same = fn.linear_cross_entropy(wide[:, pad:pad + width], w, y, bias=b)
        assert torch.equal(same[0], losses) and torch.equal(same[1], lse)
    # one row of features for all
    one = x[:1].expand(rows, width)
    a = fn.linear_cross_entropy(one, w, y, bias=b)
    assert torch.equal(a[1], fn.linear_cross_entropy(one.contiguous(), w, y, bias=b)[1])
    # leading dimensions
    if rows % 2 == 0:
        l3, s3 = fn.linear_cross_entropy(x.view(2, rows // 2, width), w, y.view(2, rows // 2), bias=b)
        assert l3.shape == (2, rows // 2) and torch.equal(l3.flatten(), losses)
        g3 = fn.linear_cross_entropy_backward(d.view(2, -1), x.view(2, rows // 2, width), w, y.view(2, -1), s3, bias=b)
        assert g3[0].shape == (2, rows // 2, width) and torch.equal(g3[0].flatten(0, 1), ref[0])


def test_no_rows(fn):
    for t in TYPES:
        x, w = torch.empty(0, 40, dtype=t, device="cuda"), torch.ones(7, 40, dtype=t, device="cuda")
        y, b = torch.empty(0, dtype=torch.int64, device="cuda"), torch.zeros(7, device="cuda")
        losses, lse = fn.linear_cross_entropy(x, w, y, bias=b)
        assert losses.shape == lse.shape == (0,)
        dw = torch.full((7, 40), 3.0, dtype=t, device="cuda")
        dx, dw, db = fn.linear_cross_entropy_backward(losses, x, w, y, lse, bias=b, dweight=dw, dbias=torch.ones(7, device="cuda"))
        assert dx.shape == (0, 40) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16], ids=str)
def test_offsets_beyond_32_bits(fn, t):
    """Rows four megabytes apart, so that the last ones lie beyond 2^32 bytes, as
    operands and as outputs; and 2^31 gradients of logits."""
    e = t.itemsize
    stride, classes, rows, width = 2**22 // e, 1100, 1050, 64
    x, w, y, b = head(4, rows, classes, width, t)
    big = torch.zeros(max(rows, classes) * stride, dtype=t, device="cuda")
    losses, lse = fn.linear_cross_entropy(x, w, y, bias=b)
    d = torch.full((rows,), 1 / rows, device="cuda")
    dx, dw, db = fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b)
    far = big.as_strided((classes, width), (stride, 1))
    far.copy_(w)
    got = fn.linear_cross_entropy(x, far, y, bias=b)
    assert torch.equal(got[0], losses)
    got = fn.linear_cross_entropy_backward(d, x, far, y, lse, bias=b)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    far = big.as_strided((rows, width), (stride, 1))
    far.copy_(x)
    assert torch.equal(fn.linear_cross_entropy(far, w, y, bias=b)[1], lse)
    got = fn.linear_cross_entropy_backward(d, far, w, y, lse, bias=b)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    out = big.as_strided((classes, width), (stride, 1))
    fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b, dweight=out)
    assert torch.equal(out, dw)


def test_many_rows_and_many_classes(fn):
    """2^33 logits: rows beyond the work-groups' search for the largest dloss,
    classes beyond one piece."""
    rows, classes, width = 70000, 123000, 8
    x, w, y, b = head(6, rows, classes, width, torch.bfloat16)
    losses, lse = fn.linear_cross_entropy(x, w, y, bias=b)
    at = torch.tensor([0, 1, 3, 35000, 69999], device="cuda")
    z, dz = logits(x[at], w, b)
    ref = torch.logsumexp(z, 1)
    tol = dz.amax(1) + (EXP + 24 + classes / 16) * U + 2 * U * ref.abs()
    check_close(lse[at], ref, tol, "lse")
    want = ref - z.gather(1, y[at][:, None])[:, 0]
    check_close(losses[at], want, 2 * tol, "losses")
    d = torch.full((rows,), 1 / rows, device="cuda")
    dx, dw, db = fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b)
    g, off = gradient(x[at], w, y[at], b, lse[at], d[at], 0.0)
    want = g @ w.double()
    rounded = off + (half(torch.bfloat16) + 2 * U) * g.abs() * 1.01
    tol = rounded @ w.double().abs() + (classes + 8) * U * (g.abs() @ w.double().abs())
    check_close(dx[at], want, tol * 1.01 + half(torch.bfloat16) * want.abs() + 1e-30, "dx")
    at = torch.tensor([0, 61111, 122999], device="cuda")
    z, dz = logits(x, w[at], b[at])
    p = torch.exp(z - lse.double()[:, None])
    ok = ((y >= 0) & (y < classes))[:, None]
    g = torch.where(ok, (p - (y[:, None] == at[None]).double()) / rows, 0.0)
    off = p / rows * (dz + (EXP + 4) * U) + U / rows
    check_close(db[at], g.sum(0), off.sum(0) + (rows + 8) * U * g.abs().sum(0), "dbias")
    rounded = off + half(torch.bfloat16) * 1.01 * g.abs()
    want = g.t() @ x.double()
    tol = rounded.t() @ x.double().abs() + (rows + 8) * U * (g.abs().t() @ x.double().abs())
    check_close(dw[at], want, tol * 1.01 + half(torch.bfloat16) * want.abs(), "dweight")


@pytest.mark.parametrize("rows,classes,width,t", [(1, 1000, 256, torch.bfloat16), (300, 1000, 256, torch.half), (600, 3001, 333, torch.float32),
                                                  (2050, 40001, 64, torch.bfloat16)])
def test_graphs_replayed_between_eager_calls(fn, rows, classes, width, t):
    x, w, y, b = head(1, rows, classes, width, t)
    other, _, y2, _ = head(2, rows, classes, width, t)
    d = torch.full((rows,), 1 / rows, device="cuda")

    def step(x, y):
        losses, lse = fn.linear_cross_entropy(x, w, y, bias=b, smoothing=0.1)
        return (losses, lse, *fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b, smoothing=0.1))

    wants = [[v.clone() for v in step(*a)] for a in ((x, y), (other, y2))]
    fixed, fixed_y = x.clone(), y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(fixed, fixed_y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(fixed, fixed_y)
    for k in range(4):
        fixed.copy_(other if k % 2 else x)
        fixed_y.copy_(y2 if k % 2 else y)
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(got, wants[k % 2]):
            assert torch.equal(a, c), k
        step(other, y2)


def test_results_are_the_same_every_time(fn):
    for rows, classes, width, t in ((500, 5000, 512, torch.bfloat16), (1500, 4001, 1000, torch.float32), (16, 40000, 256, torch.half)):
        x, w, y, b = head(8, rows, classes, width, t)
        d = torch.full((rows,), 1 / rows, device="cuda")
        first = None
        for _ in range(5):
            losses, lse = fn.linear_cross_entropy(x, w, y, bias=b)
            got = [losses, lse, *fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b)]
            first = first or [v.clone() for v in got]
            assert all(torch.equal(p, q) for p, q in zip(got, first))


def test_a_workspace_may_be_given_and_is_checked(fn):
    x, w, y, b = head(1, 200, 3000, 72, torch.half)
    want = fn.linear_cross_entropy(x, w, y, bias=b)
    d = torch.full((200,), 0.01, device="cuda")
    ref = fn.linear_cross_entropy_backward(d, x, w, y, want[1], bias=b)
    ws, back = fn.linear_cross_entropy_workspace(x, w), fn.linear_cross_entropy_workspace(x, w, True)
    for size, space in ((ws.numel(), ws), (back.numel(), back)):
        guard = torch.full((size + 4096,), 9, dtype=torch.uint8, device="cuda")
        inside = guard[:size]
        if space is ws:
            got = fn.linear_cross_entropy(x, w, y, bias=b, workspace=inside)
            assert all(torch.equal(p, q) for p, q in zip(got, want))
        else:
            got = fn.linear_cross_entropy_backward(d, x, w, y, want[1], bias=b, workspace=inside)
            assert all(torch.equal(p, q) for p, q in zip(got, ref))
        assert (guard[size:] == 9).all()
        with pytest.raises(fn.FnError, match="workspace"):
            if space is ws:
                fn.linear_cross_entropy(x, w, y, bias=b, workspace=inside[:-16])
            else:
                fn.linear_cross_entropy_backward(d, x, w, y, want[1], bias=b, workspace=inside[:-16])
        with pytest.raises(ValueError, match="contiguous"):
            fn.linear_cross_entropy(x, w, y, bias=b, workspace=guard[::2])
    with pytest.raises(fn.FnError, match="overlap"):
        fn.linear_cross_entropy_backward(d, x, w, y, want[1], bias=b, dx=x)


def test_wrong_arguments_are_refused(fn):
    x, w, y, b = head(1, 20, 30, 40, torch.half)
    for bad in (dict(x=x.float()), dict(w=w[:, :39]), dict(y=y.int()), dict(y=y[:19]), dict(b=b.half()), dict(b=b[:29]),
                dict(w=w.cpu()), dict(y=y.cpu()), dict(w=w[0])):
        a = dict(x=x, w=w, y=y, b=b, **{})
        a.update(bad)
        with pytest.raises(ValueError):
            fn.linear_cross_entropy(a["x"], a["w"], a["y"], bias=a["b"])
    _, lse = fn.linear_cross_entropy(x, w, y, bias=b)
    d = torch.ones(20, device="cuda")
    for kw in (dict(dx=x, want_dx=False), dict(dweight=w, want_dweight=False), dict(dbias=b, bias=None)):
        with pytest.raises(ValueError):
            fn.linear_cross_entropy_backward(d, x, w, y, lse, **dict(dict(bias=b), **kw))
