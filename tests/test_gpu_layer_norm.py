"""Dropout and layer norm with its gradients against their formulas in 64 bits.

Tolerances.  u = 2^-24 is one fp32 rounding, half = finfo(t).eps / 2 the
rounding to the output's type.  A row's sum of D terms is a chain of at most
depth(D) additions (a lane's own terms, 6 steps across the wavefront, up to 16
wavefronts); each is off by u relative to the sum of the terms' magnitudes.  The
mask is compared for equality: it is made of integers alone.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from conftest import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]
EPS = 1e-5
SEED = 0x9E3779B97F4A7C15


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


def depth(width: int) -> int:
    """Additions on the longest path to a row's sum."""
    own = 64 if width <= 32768 else 8 * -(-width // 8192)
    return own + 6 + 16


def half(t) -> float:
    return torch.finfo(t).eps / 2


def tiny(t) -> float:
    """Half a step of the type's subnormal numbers."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def rows(seed, n, width, t, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, width, generator=g) * torch.exp(torch.randn(n, 1, generator=g))
    return (x + mean * torch.randn(n, 1, generator=g)).to(t).cuda()


def vector(seed, width, t, mean=1.0):
    g = torch.Generator().manual_seed(seed)
    return (mean + 0.3 * torch.randn(width, generator=g)).to(t).cuda()


def check_close(got, want, tol, what):
    got, want, tol = got.double().cpu(), want.double().cpu(), tol.double().cpu()
    off = (got - want).abs()
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert bool((off <= tol).all()), f"{what}: {worst:.3g} of its tolerance"


def share(p) -> int:
    return int(np.rint(np.float64(np.float32(p)) * 65536))


def kept(seed, first_row, n, width, p) -> torch.Tensor:
    """Truth values from Philox4x32-10 in Python's integers, one block at a time
    for few blocks, in numpy's 64-bit words for many."""
    blocks = -(-width // 8)
    low = np.uint64(0xFFFFFFFF)
    row = (np.arange(n, dtype=np.uint64) + np.uint64(first_row))[:, None].repeat(blocks, 1)
    c = [np.arange(blocks, dtype=np.uint64)[None].repeat(n, 0), np.full_like(row, 1 << 31), row & low,
         row >> np.uint64(32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    fields = np.stack([h for w in c for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], -1)
    return torch.from_numpy(fields.reshape(n, -1)[:, :width] >= share(p)).cuda()


def dropped(x, p, first_row=0, seed=SEED):
    """Dropout of a matrix in 64 bits (lost elements are 0 whatever they hold)."""
    if p == 0:
        return x.double()
    scale = 65536 / (65536 - share(p)) if share(p) < 65536 else 0.0
    return torch.where(kept(seed, first_row, *x.shape, p), x.double() * scale, 0.0)


WIDTHS = [1, 2, 7, 8, 9, 15, 16, 17, 63, 65, 100, 257, 512, 513, 768, 1000, 1025, 1537, 2048, 2049, 2560,
          2561, 4095, 4096, 5003, 6145, 8192, 8193, 12344, 16384, 16385, 32768, 32769, 40001]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("width", WIDTHS)
def test_dropout_matches_its_formula(fn, width, t):
    for n, p, first in ((1, 0.1, 0), (5, 0.5, 2**32 - 2), (3, 1.0, 7), (3, 0.0, 7), (2, 1e-6, 0)):
        x, r = rows(width + n, n, width, t), rows(width + n + 1, n, width, t)
        d = dropped(x, p, first)
        out = fn.dropout(x, p, SEED, first)
        # the scale's rounding, the product's and the output's
        check_close(out, d, d.abs() * (half(t) + 2 * U) + tiny(t), "dropout")
        assert torch.equal(out == 0, (d == 0) | (x == 0))
        out = fn.dropout(x, p, SEED, first, residual=r)
        want = d + r.double()
        check_close(out, want, want.abs() * (half(t) + U) + d.abs() * 2 * U + tiny(t), "with residual")
        # the gradient is the same call: <dropout(x), y> = <x, dropout(y)>
        assert torch.equal(fn.dropout(torch.ones_like(x), p, SEED, first) == 0, ~kept(SEED, first, n, width, p))


def test_dropout_of_parts_is_that_of_the_whole(fn):
    x = rows(1, 301, 777, torch.bfloat16)
    whole = fn.dropout(x, 0.3, SEED, 2**40)
    part = torch.cat([fn.dropout(x[a:b], 0.3, SEED, 2**40 + a) for a, b in ((0, 1), (1, 128), (128, 301))])
    assert torch.equal(whole, part)
    assert not torch.equal(whole, fn.dropout(x, 0.3, SEED + 1, 2**40))
    assert not torch.equal(whole, fn.dropout(x, 0.3, SEED, 2**40 + 1))
    assert torch.equal(whole, fn.dropout(x.view(7, 43, 777), 0.3, SEED, 2**40).view(301, 777))


def test_dropout_counts(fn):
    """Lost elements are binomial: 6 standard deviations, and neighbours (in a
    row, in a column, in the two halves of a word) are lost independently."""
    for p in (0.1, 0.5):
        q = share(p) / 65536
        lost = (fn.dropout(torch.ones(4096, 4096, device="cuda"), p, 11) == 0).double()
        n = lost.numel()
        assert abs(lost.sum().item() - n * q) <= 6 * (n * q * (1 - q)) ** 0.5
        for pair in (lost[:, 1:] * lost[:, :-1], lost[1:] * lost[:-1], lost[:, 8:] * lost[:, :-8]):
            m, qq = pair.numel(), q * q
            # a pair shares an element with at most two others
            assert abs(pair.sum().item() - m * qq) <= 6 * (3 * m * qq) ** 0.5


def test_lost_elements_may_hold_anything(fn):
    x = torch.ones(40, 123, device="cuda")
    keep = kept(SEED, 0, 40, 123, 0.5)
    x[~keep] = float("nan")
    x[0][~keep[0]] = float("inf")
    out = fn.dropout(x, 0.5, SEED)
    assert torch.equal(out, keep.float() * 2)
    x[keep] = float("nan")
    assert torch.equal(fn.dropout(x, 0.5, SEED).isnan(), keep)


def norm_reference(h, w, b):
    """mean, rstd, the norm of rows h in 64 bits."""
    hd = h.double()
    mean = hd.mean(1)
    d = hd - mean[:, None]
    rstd = 1 / torch.sqrt(d.square().mean(1) + EPS)
    y = d * rstd[:, None]
    if w is not None:
        y = y * w.double()
    return mean, rstd, y if b is None else y + b.double()


def norm_errors(h, width):
    """What the roundings of a row's statistics come to: of the mean; of rstd,
    relative; of h - mean, absolute."""
    hd = h.double()
    off_mean = (depth(width) + 1) * U * hd.abs().mean(1)
    # the deviations are off by off_mean, which adds its square to their mean
    # square (their own sum is zero), and by a rounding each
    var = (hd - hd.mean(1, keepdim=True)).square().mean(1)
    rel_var = ((depth(width) + 4) * U * var + off_mean ** 2 + 2 * off_mean * U * hd.abs().amax(1)) / (var + EPS)
    return off_mean, rel_var / 2 + 4 * U


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_matches_its_formula(fn, width, t):
    for n, p, with_residual, affine in ((1, 0.0, False, 2), (3, 0.0, True, 1), (9, 0.2, True, 2), (4, 0.5, False, 0)):
        x = rows(width * 3 + n, n, width, t, mean=3.0)
        r = rows(width * 5 + n, n, width, t) if with_residual else None
        w = vector(width, width, t) if affine else None
        b = vector(width + 1, width, t, 0.0) if affine == 2 else None
        out, mean, rstd, h = fn.layer_norm(x, w, b, EPS, residual=r, p=p, seed=SEED, first_row=5)
        if p == 0 and r is None:
            assert h is x
        else:
            want = dropped(x, p, 5) + (r.double() if with_residual else 0)
            check_close(h, want, want.abs() * (half(t) + U) + dropped(x, p, 5).abs() * 2 * U + tiny(t), "h")
            if p > 0:
                assert torch.equal(h, fn.dropout(x, p, SEED, 5, residual=r))
            else:
                assert torch.equal(h, (x.float() + r.float()).to(t))
        ref_mean, ref_rstd, y = norm_reference(h, w, b)
        off_mean, rel_rstd = norm_errors(h, width)
        check_close(mean, ref_mean, off_mean + 1e-30, "mean")
        check_close(rstd, ref_rstd, ref_rstd * rel_rstd, "rstd")
        n_ = (y - (b.double() if b is not None else 0)).abs()
        wd = w.double().abs() if w is not None else 1.0
        tol = n_ * (rel_rstd[:, None] + 4 * U) + off_mean[:, None] * ref_rstd[:, None] * wd + y.abs() * half(t) * (1 + half(t)) + U * y.abs() + tiny(t)
        check_close(out, y, tol, "out")


def backward_reference(dout, h, w, mean, rstd, dsum):
    d, r = dout.double(), rstd.double()[:, None]
    n = (h.double() - mean.double()[:, None]) * r
    g = d * w.double() if w is not None else d
    dh = r * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    if dsum is not None:
        dh = dh + dsum.double()
    return dh, (d * n).sum(0), d.sum(0), n, g


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("width", WIDTHS)
def test_gradients_match_their_formula(fn, width, t):
    for n, p, with_dsum, with_weight in ((1, 0.0, False, True), (3, 0.2, True, True), (41, 0.0, True, False), (300 if width <= 1024 else 20, 0.5, False, True)):
        h, dout = rows(width + n, n, width, t, 2.0), rows(width + n + 1, n, width, t)
        dsum = rows(width + n + 2, n, width, t) if with_dsum else None
        w = vector(width, width, t) if with_weight else None
        _, mean, rstd, _ = fn.layer_norm(h, w, None, EPS)
        dh, dx, dw, db = fn.layer_norm_backward(dout, h, w, mean, rstd, dsum=dsum, p=p, seed=SEED, first_row=9)
        ref, ref_w, ref_b, nn, g = backward_reference(dout, h, w, mean, rstd, dsum)
        r = rstd.double()[:, None]
        # n: a difference and a product; g: a product; the two means are sums of
        # depth(width) additions; then a product, two differences, a product and a sum
        D = depth(width)
        # h - mean: one rounding of the difference
        off_n = 2 * U * nn.abs()
        gm, gnm = g.abs().mean(1, keepdim=True), (g * nn).abs().mean(1, keepdim=True)
        off = r * (4 * U * g.abs() + (D + 4) * U * gm + (D + 6) * U * gnm * nn.abs() + 3 * U * (nn * (g * nn).mean(1, keepdim=True)).abs()
                   + off_n * (g * nn).mean(1, keepdim=True).abs())
        off = off + U * (ref.abs() + (dsum.double().abs() if dsum is not None else 0))
        check_close(dh, ref, off * (1 + half(t)) + ref.abs() * half(t) + tiny(t), "dh")
        if p > 0:
            scale = 65536 / (65536 - share(p))
            want = dropped(ref, p, 9)
            check_close(dx, want, scale * off * (1 + half(t)) + want.abs() * (half(t) + 2 * U) + tiny(t), "dx")
            assert torch.equal(dx == 0, (want == 0) | (dx == 0))
        else:
            assert dx is dh
        # a column's sum: every row's term off by 3 u, at most n + 10 additions in a chain
        d = dout.double().abs()
        check_close(dw, ref_w, (n + 14) * U * (d * nn.abs()).sum(0) + 1e-30, "dweight")
        check_close(db, ref_b, (n + 10) * U * d.sum(0) + 1e-30, "dbias")


def test_gradients_are_those_of_differences(fn):
    """Central differences of a loss of the output, in fp32: a step of 2^-6
    leaves a third-order error of about 2^-12 of the derivative's scale, and the
    loss's roundings (64 terms of size 1, u each) 64 u / 2^-6 = 2^-12."""
    n, width = 3, 64
    x, w, b = rows(1, n, width, torch.float32), vector(2, width, torch.float32), vector(3, width, torch.float32, 0.0)
    r, m = rows(4, n, width, torch.float32), rows(5, n, width, torch.float32)

    def loss(x, r, w, b):
        out, _, _, h = fn.layer_norm(x, w, b, EPS, residual=r, p=0.3, seed=SEED, first_row=3)
        return (out.double() * m.double()).sum() + 0.5 * h.double().square().sum()

    out, mean, rstd, h = fn.layer_norm(x, w, b, EPS, residual=r, p=0.3, seed=SEED, first_row=3)
    dh, dx, dw, db = fn.layer_norm_backward(m, h, w, mean, rstd, dsum=h, p=0.3, seed=SEED, first_row=3)
    step = 2.0 ** -6
    for which, grad in ((0, dx), (1, dh), (2, dw), (3, db)):
        args = [x, r, w, b]
        flat = args[which].flatten()
        scale = grad.abs().max().item() + m.abs().max().item()
        for k in range(0, flat.numel(), 7):
            up, down = flat.clone(), flat.clone()
            up[k] += step
            down[k] -= step
            lo, hi = list(args), list(args)
            hi[which], lo[which] = up.view_as(args[which]), down.view_as(args[which])
            slope = (loss(*hi) - loss(*lo)).item() / (2 * step)
            assert abs(slope - grad.flatten()[k].item()) <= 2.0 ** -8 * scale, (which, k)


def test_rows_without_a_norm_are_nan(fn):
    for t in TYPES:
        for width in (5, 96, 3000, 40001):
            x = rows(1, 6, width, t)
            x[1, width // 2] = float("nan")
            x[2, 0] = float("inf")
            x[3, width - 1] = -float("inf")
            x[4] = 0.25
            if t != torch.float16:
                x[5] = torch.linspace(-1, 1, width).to(t).cuda() * 1e30 * (3e8 if t == torch.bfloat16 else 1e8)
            out, mean, rstd, _ = fn.layer_norm(x, None, None, EPS)
            for k in (1, 2, 3):
                assert out[k].isnan().all() and rstd[k].isnan()
            assert torch.equal(out[4], torch.zeros_like(out[4])) and abs(rstd[4].item() * EPS ** 0.5 - 1) <= 4 * U
            assert mean[4] == 0.25
            if t != torch.float16:
                assert out[5].isnan().all() and rstd[5].isnan()
            assert not out[0].isnan().any()


@pytest.mark.parametrize("width", [6, 100, 768, 2243, 5003, 12344, 40001])
def test_strides_places_and_guards(fn, width):
    """Column ranges of wider buffers at odd strides, outputs in the place of
    inputs, nothing written beside them."""
    for t in TYPES:
        n = 37
        wide = rows(3, n, width + 13, t)
        x, r = wide[:, 5:5 + width], rows(4, n, width, t)
        w, b = vector(1, width, t), vector(2, width, t, 0.0)
        want = fn.layer_norm(x.contiguous(), w, b, EPS, residual=r, p=0.1, seed=SEED)
        out = torch.full((n, width + 9), 7.0, dtype=t, device="cuda")
        s = torch.full((n, width + 3), 7.0, dtype=t, device="cuda")
        fn.layer_norm(x, w, b, EPS, residual=r, p=0.1, seed=SEED, out=out[:, 2:2 + width], sum_out=s[:, 1:1 + width])
        assert torch.equal(out[:, 2:2 + width], want[0]) and torch.equal(s[:, 1:1 + width], want[3])
        assert (out[:, :2] == 7).all() and (out[:, 2 + width:] == 7).all()
        assert (s[:, :1] == 7).all() and (s[:, 1 + width:] == 7).all()
        a, c = x.contiguous().clone(), r.clone()
        got = fn.layer_norm(a, w, b, EPS, residual=c, p=0.1, seed=SEED, out=a, sum_out=c)
        assert torch.equal(a, want[0]) and torch.equal(c, want[3])
        # one residual row for all
        one = r[:1].expand(n, width)
        assert torch.equal(fn.dropout(x, 0.1, SEED, residual=one), fn.dropout(x, 0.1, SEED, residual=one.contiguous()))
        d = x.contiguous().clone()
        assert torch.equal(fn.dropout(d, 0.1, SEED, residual=r, out=d), want[3])
        d = r.clone()
        assert torch.equal(fn.dropout(x, 0.1, SEED, residual=d, out=d), want[3])
        # gradients
        out, mean, rstd, h = want
        ref = fn.layer_norm_backward(r, h, w, mean, rstd, dsum=x.contiguous(), p=0.1, seed=SEED)
        g1, g2 = torch.full((2, n, width + 9), 7.0, dtype=t, device="cuda")
        got = fn.layer_norm_backward(r, h, w, mean, rstd, dsum=x, p=0.1, seed=SEED, dh=g1[:, 3:3 + width], dx=g2[:, 4:4 + width])
        for p, q in zip(got, ref):
            assert torch.equal(p, q)
        for g, k in ((g1, 3), (g2, 4)):
            assert (g[:, :k] == 7).all() and (g[:, k + width:] == 7).all()
        a, c = r.clone(), h.clone()
        got = fn.layer_norm_backward(a, c, w, mean, rstd, dsum=x, p=0.1, seed=SEED, dh=c, dx=a)
        for p, q in zip(got, ref):
            assert torch.equal(p, q)


def test_no_rows(fn):
    x = torch.empty(0, 64, device="cuda")
    assert fn.dropout(x, 0.1, 1).shape == (0, 64)
    out, mean, rstd, h = fn.layer_norm(x, None, None, p=0.1)
    assert out.shape == h.shape == (0, 64) and mean.shape == (0,)
    dh, dx, dw, db = fn.layer_norm_backward(x, x, None, mean, rstd, p=0.1)
    assert dh.shape == (0, 64) and (dw == 0).all() and (db == 0).all() and dw.shape == (64,)


@pytest.mark.parametrize("rows_,width", [(1_300_000, 12), (70_000, 40), (3, 2**20 + 3), (2, 2**26 + 5)])
def test_many_rows_and_wide_ones(fn, rows_, width):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows_, width, generator=g, device="cuda").half()
    at = torch.tensor(sorted({0, 1, rows_ // 2, rows_ - 1}))
    out, mean, rstd, h = fn.layer_norm(x, None, None, EPS, p=0.25, seed=SEED, first_row=1)
    for k in at.tolist():
        keep = kept(SEED, 1 + k, 1, width, 0.25)
        assert torch.equal(h[k:k + 1] == 0, ~keep | (x[k:k + 1] == 0))
    assert torch.equal(h, fn.dropout(x, 0.25, SEED, 1))
    _, ref_rstd, y = norm_reference(h[at], None, None)
    off_mean, rel = norm_errors(h[at], width)
    check_close(out[at], y, y.abs() * (rel[:, None] + 4 * U + half(torch.float16)) + (off_mean * ref_rstd)[:, None] + tiny(torch.float16), "out")
    dh, dx, dw, db = fn.layer_norm_backward(x, h, None, mean, rstd)
    ref_b = x.double().sum(0)
    check_close(db, ref_b, (rows_ / 64 + 600) * U * x.double().abs().sum(0), "dbias")


def test_offsets_beyond_32_bits(fn):
    """A buffer of 5 GiB: rows a quarter of a gigabyte apart, beyond 2^32 bytes
    and 2^31 elements."""
    stride, width, n = 2**27 + 8, 1000, 20
    big = torch.zeros(n * stride, dtype=torch.half, device="cuda")
    x = big.as_strided((n, width), (stride, 1))
    x.copy_(rows(1, n, width, torch.half))
    want = fn.layer_norm(x.contiguous(), None, None, EPS, p=0.1, seed=SEED)
    out, mean, rstd, h = fn.layer_norm(x, None, None, EPS, p=0.1, seed=SEED, out=x)
    assert torch.equal(out, want[0]) and torch.equal(h, want[3])
    x.copy_(h)
    ref = fn.layer_norm_backward(want[0], h, None, mean, rstd)
    got = fn.layer_norm_backward(want[0], x, None, mean, rstd, dh=x)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[2], ref[2])


def test_graphs_replayed_between_eager_calls(fn):
    """Forward and backward captured once, replayed on other data, with eager
    calls and their own workspaces between."""
    t, n, width = torch.bfloat16, 700, 768
    x, r, m = (rows(k, n, width, t) for k in (1, 2, 3))
    w, b = vector(1, width, t), vector(2, width, t, 0.0)

    def step(x):
        out, mean, rstd, h = fn.layer_norm(x, w, b, EPS, residual=r, p=0.1, seed=SEED)
        return (out, *fn.layer_norm_backward(m, h, w, mean, rstd, dsum=out, p=0.1, seed=SEED))

    wants = [[v.clone() for v in step(y)] for y in (x, r)]
    fixed = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(fixed)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(fixed)
    for k in range(4):
        fixed.copy_(r if k % 2 else x)
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(got, wants[k % 2]):
            assert torch.equal(a, c), k
        step(m)


def test_a_block_trains_through_a_function(fn):
    """dropout + residual + norm as a torch.autograd.Function, against autograd
    in 64 bits.  Each gradient is a sum of products of numbers up to `size`, a
    row's sums chains of under 100 additions: 128 u of it."""
    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, weight, bias, p, seed):
            out, mean, rstd, h = fn.layer_norm(x, weight, bias, EPS, residual=residual, p=p, seed=seed)
            ctx.save_for_backward(h, weight, mean, rstd)
            ctx.drop = (p, seed)
            return out, h

        @staticmethod
        def backward(ctx, dout, dsum):
            h, weight, mean, rstd = ctx.saved_tensors
            p, seed = ctx.drop
            dh, dx, dw, db = fn.layer_norm_backward(dout, h, weight, mean, rstd, dsum=dsum, p=p, seed=seed)
            return dx, dh, dw, db, None, None

    n, width = 9, 200
    x, r, m = (rows(k, n, width, torch.float32) for k in (1, 2, 3))
    w, b = vector(4, width, torch.float32), vector(5, width, torch.float32, 0.0)
    leaves = [v.clone().requires_grad_() for v in (x, r, w, b)]
    out, h = Block.apply(*leaves, 0.2, SEED)
    (out * m).sum().add((h * h).sum()).backward()
    ref = [v.double().requires_grad_() for v in (x, r, w, b)]
    hd = torch.where(kept(SEED, 0, n, width, 0.2), ref[0] * (65536 / (65536 - share(0.2))), 0.0) + ref[1]
    d = hd - hd.mean(1, keepdim=True)
    yd = d / torch.sqrt(d.square().mean(1, keepdim=True) + EPS) * ref[2] + ref[3]
    (yd * m.double()).sum().add((hd * hd).sum()).backward()
    for got, want in zip(leaves, ref):
        size = want.grad.abs().max() + (x.abs() * m.abs()).max()
        assert (got.grad.double() - want.grad).abs().max() <= 128 * U * size
