"""RMS norm, its gradients and row quantisation against their formulas in 64
bits (through the C ABI and the tensor helpers).

Tolerances.  u = 2^-24 is one fp32 rounding, half = finfo(t).eps / 2 the
rounding to the output's type.  A row's sum of D terms is a chain of at most
depth(D) additions (a lane's own terms, 6 steps across the wavefront, up to 16
wavefronts), each off by u relative to a sum of positive terms; rstd halves
that.  Codes are compared for equality: they depend on no sum.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from conftest import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]
EPS = 1e-6


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


def depth(width: int) -> int:
    """Additions on the longest path to a row's sum."""
    own = 32 if width <= 32768 else 8 * -(-width // 8192)
    return own + 6 + 16


def half(t) -> float:
    return torch.finfo(t).eps / 2 if t != torch.float32 else U


def tiny(t) -> float:
    """Half a step of the type's subnormal numbers."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def rows(seed, n, width, t, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, width, generator=g) * torch.exp(spread * torch.randn(n, 1, generator=g))
    return x.to(t).cuda()


def weights(seed, width, t):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(width, generator=g)).to(t).cuda()


def codes_of(t32: torch.Tensor):
    """Codes and A of rows by the documented fp32 steps, in numpy (IEEE)."""
    t = t32.cpu().numpy()
    assert t.dtype == np.float32
    top = np.max(np.abs(t), axis=1)
    scale = np.where(top < np.float32(2.0 ** -100), np.float32(2.0 ** 100), np.float32(1))
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        inv = np.where(top > 0, np.float32(127) * (np.float32(1) / (top * scale)),
                       np.float32(0)).astype(np.float32)
        q = np.rint(((t * scale[:, None]).astype(np.float32) * inv[:, None]).astype(np.float32))
    bad = ~np.isfinite(top)
    q[bad] = 0
    return torch.from_numpy(q.astype(np.int8)), torch.from_numpy(top.astype(np.float64))


def check_close(got, want, tol, what):
    got, want, tol = got.double().cpu(), want.double().cpu(), tol.double().cpu()
    off = (got - want).abs()
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert bool((off <= tol).all()), f"{what}: {worst:.3g} of its tolerance"


def reference(x, residual, weight):
    """h (exact rounding), and in 64 bits: t = h w, rstd, the norm."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    hd = h.double()
    rstd = 1 / torch.sqrt(hd.square().mean(1) + EPS)
    return h, rstd, hd * rstd[:, None] * weight.double()


WIDTHS = [1, 2, 7, 8, 9, 15, 63, 64, 65, 257, 511, 512, 513, 768, 1000, 1023, 1024, 1025, 2047,
          2048, 2049, 2560, 2561, 4095, 4096, 4097, 5003, 8191, 8192, 8193, 16383, 16384, 16385, 32767, 32768,
          32769, 40001, 65544]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_matches_its_formula(fn, width, t):
    for n in (1, 3, 9):
        for with_residual in (False, True):
            x = rows(width * 3 + n, n, width, t)
            r = rows(width * 5 + n, n, width, t) if with_residual else None
            w = weights(width, width, t)
            h, rstd, y = reference(x, r, w)
            out, got_rstd, got_h = fn.rms_norm(x, w, EPS, residual=r)
            codes, scales, got_h8 = fn.rms_norm_q8(x, w, EPS, residual=r)
            assert torch.equal(got_h, h) and torch.equal(got_h8, h)
            rel = (depth(width) / 2 + 6) * U
            check_close(got_rstd, rstd, rstd * rel, "rstd")
            check_close(out, y, y.abs() * (half(t) + rel + 2 * U) + tiny(t), "out")
            want, top = codes_of(h.float() * w.float())
            assert torch.equal(codes.cpu(), want)
            check_close(scales, top * rstd.cpu() / 127, top * rstd.cpu() / 127 * (rel + 3 * U),
                        "scales")


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("width", WIDTHS)
def test_quantized_rows_match_their_formula(fn, width, t):
    for n in (1, 6):
        x = rows(width + n, n, width, t)
        codes, scales = fn.quantize_rows(x)
        want, top = codes_of(x.float())
        assert torch.equal(codes.cpu(), want)
        check_close(scales, top / 127, top / 127 * U + tiny(torch.float32), "scales")
        # and as a quantiser: every element within half a step of its value
        off = (codes.double().cpu() * (top / 127)[:, None] - x.double().cpu()).abs()
        assert bool((off <= (top / 127)[:, None] * (0.5 + 127 * 3 * U)).all())


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("width", [5, 768, 1500, 4096, 33000])
def test_rows_without_a_norm_and_empty_rows(fn, width, t):
    """Rows of zeros, NaN, infinities, the type's lowest value throughout,
    squares that overflow, numbers too small for 1 / A, ties and near-ties."""
    n = 12
    x = rows(7, n, width, t, spread=0.0)
    fin = torch.finfo(t)
    x[1] = 0
    x[2, width // 2] = float("nan")
    x[3, width - 1] = float("inf")
    x[4, 0] = -float("inf")
    x[5] = fin.min
    x[6] = 0
    x[6, width - 1] = fin.smallest_normal * fin.eps  # the smallest subnormal
    x[7] = fin.smallest_normal
    x[8] = 0
    x[8, 0] = 1.0
    x[9] = 254.0
    x[9, : width // 2] = 1.0  # 127 / 254: a half
    x[9, width // 2:width - 1] = -3.0  # -1.5
    w = torch.ones(width, dtype=t, device="cuda")
    codes, scales = fn.quantize_rows(x)
    want, top = codes_of(x.float())
    bad = [2, 3, 4]
    good = [r for r in range(n) if r not in bad]
    assert torch.equal(codes.cpu(), want)
    assert bool(torch.isnan(scales[bad]).all()) and not codes[bad].any()
    check_close(scales[good], top[good] / 127, top[good] / 127 * U + tiny(torch.float32), "scales")
    assert scales[1] == 0 and not codes[1].any()

    codes, scales, _ = fn.rms_norm_q8(x, w, EPS)
    out, rstd, _ = fn.rms_norm(x, w, EPS)
    assert torch.isnan(out[bad]).all() and torch.isnan(rstd[bad]).all()
    assert torch.isnan(scales[bad]).all() and not codes[bad].any()
    assert not out[1].any() and scales[1] == 0 and not codes[1].any()
    xd = x.double()
    ms = xd.square().mean(1)
    if t != torch.float16:  # the squares of the lowest value overflow fp32
        assert torch.isnan(out[5]).all() and torch.isnan(rstd[5]) and torch.isnan(scales[5])
        assert not codes[5].any()
        good.remove(5)
    y = xd / torch.sqrt(ms + EPS)[:, None]
    rel = (depth(width) / 2 + 8) * U
    # squares below fp32's smallest are lost beside eps = 1e-6, as they should be
    check_close(out[good], y[good], y[good].abs() * (half(t) + rel) + tiny(t), "out")
    assert torch.equal(codes[good].cpu(), want[good])


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_weights_that_are_nan_infinite_or_zero(fn, t):
    x = rows(3, 4, 600, t, spread=0.0)
    w = weights(3, 600, t)
    w[17] = float("nan")
    codes, scales, _ = fn.rms_norm_q8(x, w, EPS)
    assert torch.isnan(scales).all() and not codes.any()
    w[17] = float("inf")
    codes, scales, _ = fn.rms_norm_q8(x, w, EPS)
    assert torch.isnan(scales).all() and not codes.any()
    codes, scales, _ = fn.rms_norm_q8(x, torch.zeros_like(w), EPS)
    assert not scales.any() and not codes.any()


def padded(x, left, right, fill):
    """x as a column range of a wider buffer."""
    big = torch.full((x.size(0), left + x.size(1) + right), fill, dtype=x.dtype, device=x.device)
    big[:, left:left + x.size(1)] = x
    return big, big[:, left:left + x.size(1)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("width", [1, 8, 100, 768, 1021, 2048, 2243, 2560, 5003, 20000, 33001])
def test_strided_rows_and_guard_columns(fn, width, t):
    """Inputs and outputs as column ranges at odd offsets: the same results,
    and nothing beside them is written."""
    n = 5
    x0, r0, w = rows(1, n, width, t), rows(2, n, width, t), weights(3, width, t)
    out0, rstd0, h0 = fn.rms_norm(x0, w, EPS, residual=r0)
    codes0, scales0, _ = fn.rms_norm_q8(x0, w, EPS, residual=r0)
    for left, right in ((1, 0), (3, 2), (8, 8), (0, 5)):
        _, x = padded(x0, left, right, float("nan"))
        _, r = padded(r0, right, left, float("nan"))
        sb, s = padded(torch.zeros_like(x0), left + 1, right, 7.0)
        ob, o = padded(torch.zeros_like(x0), left, right + 1, 7.0)
        cb, c = padded(torch.zeros_like(codes0), left, right, 77)
        out, rstd, h = fn.rms_norm(x, w, EPS, residual=r, sum_out=s, out=o)
        assert torch.equal(out, out0) and torch.equal(h, h0) and torch.equal(rstd, rstd0)
        codes, scales, h = fn.rms_norm_q8(x, w, EPS, residual=r, sum_out=s, codes=c)
        assert torch.equal(codes, codes0) and torch.equal(scales, scales0) and torch.equal(h, h0)
        for big, l, value in ((sb, left + 1, 7.0), (ob, left, 7.0), (cb, left, 77)):
            assert (big[:, :l] == value).all() and (big[:, l + width:] == value).all()
        c2b, c2 = padded(torch.zeros_like(codes0), left, right, 77)
        codes, scales = fn.quantize_rows(x, codes=c2)
        ref_codes, ref_scales = fn.quantize_rows(x0)
        assert torch.equal(codes, ref_codes) and torch.equal(scales, ref_scales)
        assert (c2b[:, :left] == 77).all() and (c2b[:, left + width:] == 77).all()


@pytest.mark.parametrize("width", [100, 4096, 33000])
def test_outputs_in_the_place_of_inputs(fn, width):
    t = torch.bfloat16
    x0, r0, w = rows(1, 6, width, t), rows(2, 6, width, t), weights(3, width, t)
    out0, _, h0 = fn.rms_norm(x0, w, EPS, residual=r0)
    codes0, scales0, _ = fn.rms_norm_q8(x0, w, EPS, residual=r0)
    x, r = x0.clone(), r0.clone()
    out, _, h = fn.rms_norm(x, w, EPS, residual=r, sum_out=r, out=x)
    assert out is x and h is r and torch.equal(x, out0) and torch.equal(r, h0)
    x, r = x0.clone(), r0.clone()
    out, _, h = fn.rms_norm(x, w, EPS, residual=r, sum_out=x, out=r)
    assert torch.equal(r, out0) and torch.equal(x, h0)
    x, r = x0.clone(), r0.clone()
    codes, scales, h = fn.rms_norm_q8(x, w, EPS, residual=r, sum_out=r)
    assert torch.equal(codes, codes0) and torch.equal(scales, scales0) and torch.equal(r, h0)
    x = x0.clone()
    plain, _, _ = fn.rms_norm(x0, w, EPS)
    fn.rms_norm(x, w, EPS, out=x)
    assert torch.equal(x, plain)


def test_one_residual_row_for_all_and_leading_dimensions(fn):
    t = torch.float16
    x, w = rows(1, 24, 700, t), weights(3, 700, t)
    r = rows(2, 1, 700, t)
    want = fn.rms_norm_q8(x, w, EPS, residual=r.expand(24, 700).contiguous())
    got = fn.rms_norm_q8(x.view(2, 3, 4, 700), w, EPS, residual=r.expand(2, 3, 4, 700))
    for a, b in zip(got, want):
        assert torch.equal(a.reshape(b.shape), b)
    assert got[0].shape == (2, 3, 4, 700) and got[1].shape == (2, 3, 4)
    one = fn.rms_norm(x[0], w, EPS)
    assert one[0].shape == (700,) and one[1].shape == ()
    assert torch.equal(one[0], fn.rms_norm(x, w, EPS)[0][0])


def test_many_rows(fn):
    """More rows than one grid holds at a time (and than 2^20 work-groups)."""
    t = torch.float16
    for n, width in ((4_300_000, 3), (1_100_000, 1100)):
        x, w = torch.randn(n, width, device="cuda").to(t), weights(3, width, t)
        codes, scales = fn.quantize_rows(x)
        top = x.float().abs().amax(1)
        inv = 127.0 * (1.0 / top.double()).float()
        assert torch.equal(codes, torch.round(x.float() * inv[:, None]).to(torch.int8))
        out, rstd, _ = fn.rms_norm(x, w, EPS)
        want = 1 / torch.sqrt(x.double().square().mean(1) + EPS)
        assert ((rstd.double() - want).abs() <= want * (depth(width) / 2 + 6) * U).all()
        y = x.double() * want[:, None] * w.double()
        assert ((out.double() - y).abs() <= y.abs() * (half(t) + 60 * U) + tiny(t)).all()


def test_rows_far_apart(fn):
    """Row offsets beyond 2^32 elements."""
    t, width, n = torch.bfloat16, 2050, 3
    far = 2_200_000_123
    buf = torch.empty(2 * far + width, dtype=t, device="cuda")
    x = buf.as_strided((n, width), (far, 1))
    x0 = rows(4, n, width, t)
    x.copy_(x0)
    w = weights(5, width, t)
    for got, want in zip(fn.rms_norm_q8(x, w, EPS)[:2], fn.rms_norm_q8(x0, w, EPS)[:2]):
        assert torch.equal(got, want)
    want, _, _ = fn.rms_norm(x0, w, EPS)
    fn.rms_norm(x, w, EPS, out=x)
    assert torch.equal(x, want)


# ------------------------------------------------------------------ backward

def backward_reference(dout, h, w, rstd, dsum):
    d, h, w, r = dout.double(), h.double(), w.double(), rstd.double()[:, None]
    n, g = h * r, d * w
    mean = (g * n).mean(1, keepdim=True)
    dx = r * (g - n * mean) + (0 if dsum is None else dsum.double())
    size = 8 * ((r * g).abs() + (r * n * mean).abs())
    if dsum is not None:
        size = size + 2 * dsum.double().abs()
    size = size + (depth(h.size(1)) + 8) * (r * n).abs() * (g * n).abs().mean(1, keepdim=True)
    return dx, size * U, (d * n).sum(0), (d * n).abs().sum(0)


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("width", WIDTHS)
def test_gradients_match_their_formula(fn, width, t):
    for n, with_sum in ((1, True), (7, False), (600, True)):
        if n * width > 2_000_000:
            n = 40
        h, w = rows(width + n, n, width, t), weights(width, width, t)
        dout = rows(width + n + 1, n, width, t, spread=0.2)
        dsum = rows(width + n + 2, n, width, t, spread=0.2) if with_sum else None
        rstd = (1 / torch.sqrt(h.double().square().mean(1) + EPS)).float()
        dx, dweight = fn.rms_norm_backward(dout, h, w, rstd, dsum=dsum)
        want, size, dw, dw_size = backward_reference(dout, h, w, rstd, dsum)
        check_close(dx, want, want.abs() * half(t) + size + tiny(t), "dx")
        # a column: the rows of one lane, up to three more lanes, 64 parts of
        # the partial sums; the product's two roundings
        chain = n + 3 + 32 + 64 + 3
        check_close(dweight, dw, dw_size * chain * U + tiny(torch.float32), "dweight")


def test_gradients_match_autograd_and_differences(fn):
    """Against torch's derivative of the forward formula in 64 bits, and
    against central differences of it."""
    n, width, step = 3, 11, 1e-5
    g = torch.Generator().manual_seed(2)
    x, r, w, dout, dsum = (torch.randn(*s, generator=g) for s in
                           ((n, width), (n, width), (width,), (n, width), (n, width)))

    def loss(x, r, w):
        h = x + r
        return (h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * w * dout.double()).sum() \
            + (h * dsum.double()).sum()

    leaves = [v.double().requires_grad_() for v in (x, r, w)]
    grads = torch.autograd.grad(loss(*leaves), leaves)
    out, rstd, h = fn.rms_norm(x.cuda(), w.cuda(), EPS, residual=r.cuda())
    dx, dweight = fn.rms_norm_backward(dout.cuda(), h, w.cuda(), rstd, dsum=dsum.cuda())
    # h itself is rounded to fp32 here: a relative change of u in each element
    size = 100 * U * (1 + grads[0].abs().max())
    for got, want in ((dx, grads[0]), (dx, grads[1]), (dweight, grads[2])):
        assert (got.double().cpu() - want).abs().max() <= size
    with torch.no_grad():
        for k, (leaf, got) in enumerate(zip(leaves, (dx, dx, dweight))):
            flat = leaf.view(-1)
            for i in range(flat.numel()):
                keep = flat[i].item()
                flat[i] = keep + step
                up = loss(*leaves)
                flat[i] = keep - step
                down = loss(*leaves)
                flat[i] = keep
                slope = ((up - down) / (2 * step)).item()
                # the third derivative's share is step^2, the loss's own rounding 2^-52 / step
                assert abs(got.reshape(-1)[i].item() - slope) <= size.item() + 1e-7, (k, i)


@pytest.mark.parametrize("width", [60, 768, 3001, 33000])
def test_gradient_in_place_strided_and_repeatable(fn, width):
    t, n = torch.float16, 700 if width < 4000 else 20
    h, w = rows(1, n, width, t), weights(2, width, t)
    dout, dsum = rows(3, n, width, t, 0.1), rows(4, n, width, t, 0.1)
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + EPS)).float()
    dx0, dw0 = fn.rms_norm_backward(dout, h, w, rstd, dsum=dsum)
    for _ in range(3):
        dx, dw = fn.rms_norm_backward(dout, h, w, rstd, dsum=dsum)
        assert torch.equal(dx, dx0) and torch.equal(dw, dw0)
    for k in range(3):
        args = [dout.clone(), h.clone(), dsum.clone()]
        dx, dw = fn.rms_norm_backward(args[0], args[1], w, rstd, dsum=args[2], dx=args[k])
        assert torch.equal(args[k], dx0) and torch.equal(dw, dw0)
    _, hs = padded(h, 3, 1, float("nan"))
    _, ds = padded(dout, 1, 1, float("nan"))
    _, ss = padded(dsum, 0, 3, float("nan"))
    big, o = padded(torch.zeros_like(h), 5, 2, 9.0)
    guard = torch.full((width + 8,), 9.0, device="cuda")
    dx, dw = fn.rms_norm_backward(ds, hs, w, rstd, dsum=ss, dx=o, dweight=guard[4:-4])
    assert torch.equal(dx, dx0) and torch.equal(dw, dw0)
    assert (big[:, :5] == 9).all() and (big[:, 5 + width:] == 9).all()
    assert (guard[:4] == 9).all() and (guard[-4:] == 9).all()


def test_gradient_of_no_rows_is_zero(fn):
    for width in (1, 100, 40000):
        h = torch.empty(0, width, dtype=torch.bfloat16, device="cuda")
        dw = torch.full((width,), 5.0, device="cuda")
        w = torch.ones(width, dtype=torch.bfloat16, device="cuda")
        dx, got = fn.rms_norm_backward(h, h, w, torch.empty(0, device="cuda"), dweight=dw)
        assert dx.shape == (0, width) and not got.any()


def test_rows_in_a_graph_and_on_another_stream(fn):
    """Captured once and replayed, with eager work between the replays, and
    issued on a stream of its own: the eager results."""
    t, n, width = torch.bfloat16, 300, 1000
    x, r, w = rows(1, n, width, t), rows(2, n, width, t), weights(3, width, t)
    dout = rows(4, n, width, t)
    codes = torch.empty(n, width, dtype=torch.int8, device="cuda")
    scales, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    h, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(width, device="cuda")
    ws = fn.rms_norm_backward_workspace(n, width)

    def work(stream=None):
        fn.rms_norm_q8(x, w, EPS, residual=r, sum_out=h, codes=codes, scales=scales, rstd=rstd,
                       stream=stream)
        fn.rms_norm_backward(dout, h, w, rstd, dx=dx, dweight=dw, workspace=ws, stream=stream)

    def results():
        torch.cuda.synchronize()
        return [v.clone() for v in (h, codes, scales, rstd, dx, dw)]

    work()
    want = results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        work()
    for k in range(5):
        for v in (h, codes, scales, rstd, dx, dw):
            v.zero_()
        graph.replay()
        for a, b in zip(results(), want):
            assert torch.equal(a, b), k
        fn.quantize_rows(x)  # eager work between replays
    for v in (h, codes, scales, rstd, dx, dw):
        v.zero_()
    torch.cuda.synchronize()
    work(stream=side)
    side.synchronize()
    for a, b in zip(results(), want):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ refusals

def test_refusals_on_device_buffers(fn):
    """Overlaps, short buffers, host memory, wrong dtypes and shapes: refused
    before anything is launched (nothing is written)."""
    t = torch.float16
    buf = torch.zeros(100, 64, dtype=t, device="cuda")
    w = torch.ones(64, dtype=t, device="cuda")
    x, r = rows(1, 10, 64, t), rows(2, 10, 64, t)

    def refused(word, call, *args, **kw):
        with pytest.raises(fn.FnError) as e:
            call(*args, **kw)
        assert e.value.code == -1 and word in str(e.value), str(e.value)

    refused("overlap", fn.rms_norm, buf[:10], w, out=buf[1:11])
    refused("overlap", fn.rms_norm, x, w, residual=r, sum_out=buf[:10], out=buf[:10])
    refused("overlap", fn.rms_norm, x, w, residual=r, sum_out=buf[:10], out=buf[9:19])
    refused("overlap", fn.rms_norm_q8, buf[:10], w, codes=buf.view(torch.int8)[:10, :64])
    refused("overlap", fn.rms_norm, x, buf[3], out=buf[:10])
    wide = torch.zeros(10, 128, dtype=t, device="cuda")
    refused("overlap", fn.rms_norm, wide[:, :64], w, out=wide[:, 63:127])
    refused("overlap", fn.rms_norm, wide[:, 64:], w, out=wide[:, 1:65])
    fn.rms_norm(wide[:, :64], w, out=wide[:, 64:])  # side by side: allowed
    fn.rms_norm(wide[:, 64:], w, out=wide[:, :64])
    refused("overlap", fn.rms_norm_backward, buf[:10], x, w, torch.ones(10, device="cuda"),
            dx=buf[5:15])
    small = torch.zeros(2, dtype=torch.float32, device="cuda")
    many = torch.zeros(3000, 64, dtype=t, device="cuda")
    refused("workspace", fn.rms_norm_backward, many, many, w, torch.ones(3000, device="cuda"),
            workspace=small)
    refused("x_dev", fn.fn_rms_norm, torch.zeros(10, 64, dtype=t), 64, None, 0, w, 10, 64, 1e-6, 1,
            None, 0, buf, 64, None)
    refused("available", fn.fn_quantize_rows, x, 64, 1 << 22, 64, 1,
            torch.empty(10, 64, dtype=torch.int8, device="cuda"), 64, small)
    for bad in (lambda: fn.rms_norm(x, w.float()), lambda: fn.rms_norm(x, w[:63]),
                lambda: fn.rms_norm(x, w, residual=r.float()),
                lambda: fn.rms_norm(x, w, sum_out=r), lambda: fn.rms_norm(x.double(), w.double()),
                lambda: fn.rms_norm(x.t(), torch.ones(10, dtype=t, device="cuda")),
                lambda: fn.rms_norm(x, w, out=buf[:9]),
                lambda: fn.quantize_rows(x, scales=torch.empty(20, device="cuda")[::2])):
        with pytest.raises(ValueError):
            bad()
    assert not buf.any()


MORE_WIDTHS = [3, 4, 5, 6, 10, 12, 16, 17, 24, 28, 31, 32, 33, 100, 127, 128, 129, 200, 255, 256,
               600, 769, 900, 1500, 1536, 1537, 3000, 6143, 6144, 6145, 10001, 12344, 12345, 20001]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("width", MORE_WIDTHS)
def test_rows_of_every_shape_of_threads(fn, width, t):
    """The widths at which the threads per row change, and between: more rows
    than a work-group takes, an odd number of them."""
    n = 259 if width < 4000 else 21
    x, r, w = rows(width, n, width, t), rows(width + 1, n, width, t), weights(width, width, t)
    h, rstd, y = reference(x, r, w)
    rel = (depth(width) / 2 + 6) * U
    out, got_rstd, got_h = fn.rms_norm(x, w, EPS, residual=r)
    assert torch.equal(got_h, h)
    check_close(got_rstd, rstd, rstd * rel, "rstd")
    check_close(out, y, y.abs() * (half(t) + rel + 2 * U) + tiny(t), "out")
    codes, scales, _ = fn.rms_norm_q8(x, w, EPS, residual=r)
    want, top = codes_of(h.float() * w.float())
    assert torch.equal(codes.cpu(), want)
    check_close(scales, top * rstd.cpu() / 127, top * rstd.cpu() / 127 * (rel + 3 * U), "scales")
    codes, scales = fn.quantize_rows(x)
    want, top = codes_of(x.float())
    assert torch.equal(codes.cpu(), want)
    check_close(scales, top / 127, top / 127 * U + tiny(torch.float32), "scales")
    dout = rows(width + 2, n, width, t, spread=0.2)
    dx, dweight = fn.rms_norm_backward(dout, h, w, rstd.float(), dsum=x)
    want, size, dw, dw_size = backward_reference(dout, h, w, rstd.float(), x)
    check_close(dx, want, want.abs() * half(t) + size + tiny(t), "dx")
    check_close(dweight, dw, dw_size * (n + 3 + 32 + 64 + 3) * U + tiny(torch.float32), "dweight")


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("n,width", [(6100, 2811), (5999, 2811), (6000, 3585)])
def test_gradients_of_rows_for_many_work_groups(fn, n, width, t):
    """Where the number of work-groups changes with the rows and the width."""
    h, w = rows(1, n, width, t), weights(2, width, t)
    dout = rows(3, n, width, t, spread=0.2)
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + EPS)).float()
    dx, dweight = fn.rms_norm_backward(dout, h, w, rstd)
    want, size, dw, dw_size = backward_reference(dout, h, w, rstd, None)
    check_close(dx, want, want.abs() * half(t) + size + tiny(t), "dx")
    # the rows of one thread, then 512 partial sums
    chain = n // 256 + 1 + 512 + 3
    check_close(dweight, dw, dw_size * chain * U + tiny(torch.float32), "dweight")
