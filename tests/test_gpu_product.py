"""The product of 8-bit codes against 64-bit integers.

The sum is exact; what follows is three fp32 operations and one rounding to
the output's type, so the result is compared bit for bit with the same steps
in numpy, and with the 64-bit value within 4 u |sum sa sb| + u |y| + half |y|
(u = 2^-24: the sum's conversion, two products, the bias's addition)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from conftest import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


def operands(seed, m, n, k, lowest=-128):
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(lowest, 128, (m, k), generator=g, dtype=torch.int8)
    b = torch.randint(lowest, 128, (n, k), generator=g, dtype=torch.int8)
    sa = torch.exp(torch.randn(m, generator=g)) * 0.01
    sb = torch.exp(torch.randn(n, generator=g)) * 0.01
    bias = torch.randn(n, generator=g)
    return a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), bias.cuda()


def sums(a, b):
    """The exact integer sums (64-bit floating point holds them all)."""
    return torch.matmul(a.double(), b.double().t().contiguous())


def expected(total, sa, sb, bias, t):
    """The documented fp32 steps, elementwise (no fused operation in numpy)."""
    y = total.cpu().numpy().astype(np.float32)
    y = y * sa.cpu().numpy()[:, None]
    y = y * sb.cpu().numpy()[None, :]
    if bias is not None:
        y = y + bias.cpu().numpy()[None, :]
    assert y.dtype == np.float32
    return torch.from_numpy(y).to(t)


def check(got, total, sa, sb, bias, t):
    want = expected(total, sa, sb, bias, t)
    assert torch.equal(got.cpu(), want)
    scaled = total * sa.double()[:, None] * sb.double()[None, :]
    y = scaled if bias is None else scaled + bias.double()
    half = U if t == torch.float32 else torch.finfo(t).eps / 2
    tol = 4 * U * scaled.abs() + (U + half) * y.abs() + torch.finfo(t).smallest_normal * 2 * half
    assert bool(((got.double() - y).abs() <= tol).all())


SIZES = [(1, 1, 1), (1, 16, 16), (2, 3, 5), (1, 100, 64), (3, 5, 7), (5, 1, 33), (16, 16, 64),
         (17, 33, 65), (15, 31, 63), (32, 32, 32), (33, 48, 128), (64, 64, 64), (65, 63, 96),
         (1, 513, 1000), (7, 1000, 1021), (48, 520, 512), (100, 300, 256), (127, 129, 272),
         (128, 128, 128), (129, 257, 300), (200, 520, 1024), (256, 256, 192), (257, 511, 320),
         (300, 1000, 768), (1, 2048, 4096), (16, 1024, 2048), (31, 777, 2048), (64, 768, 1536),
         (520, 260, 16), (1000, 8, 4096), (700, 900, 80), (513, 1025, 640)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_is_exact(fn, m, n, k, t):
    a, sa, b, sb, bias = operands(m * 7 + n * 3 + k, m, n, k)
    total = sums(a, b)
    for bi in (None, bias):
        out = torch.full((m, n), 3.0, dtype=t, device="cuda")
        check(fn.matmul_q8(a, sa, b, sb, bias=bi, out=out), total, sa, sb, bi, t)


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("m,n,k", [(2048, 1024, 512), (1030, 4100, 1056), (3000, 768, 768),
                                   (2049, 2047, 1040), (5000, 129, 2000), (130, 5000, 999)])
def test_larger_products(fn, m, n, k, t):
    a, sa, b, sb, bias = operands(m + n + k, m, n, k)
    total = sums(a, b)
    check(fn.matmul_q8(a, sa, b, sb, bias=bias, out_dtype={
        torch.float32: fn.FN_OUT_FP32, torch.float16: fn.FN_OUT_FP16,
        torch.bfloat16: fn.FN_OUT_BF16}[t]), total, sa, sb, bias, t)


@pytest.mark.parametrize("m,n", [(1, 3), (20, 70), (300, 140)])
def test_longest_sums_of_extreme_codes(fn, m, n):
    """|sum| up to 128 * 128 * 131071, just inside 32 bits."""
    k = 131071
    a = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    b = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    b[n // 2] = 127
    a[m - 1, ::2] = 127
    sa, sb = torch.full((m,), 0.5, device="cuda"), torch.full((n,), 2.0, device="cuda")
    check(fn.matmul_q8(a, sa, b, sb, out_dtype=fn.FN_OUT_FP32), sums(a, b), sa, sb, None,
          torch.float32)
    with pytest.raises(fn.FnError) as e:
        fn.matmul_q8(torch.zeros(1, k + 1, dtype=torch.int8, device="cuda"), sa[:1],
                     torch.zeros(1, k + 1, dtype=torch.int8, device="cuda"), sb[:1])
    assert e.value.code == -2


@pytest.mark.parametrize("m,n,k", [(1, 70, 100), (40, 300, 256), (150, 200, 512), (600, 520, 160),
                                   (300, 260, 1021)])
def test_strided_operands_and_guard_columns(fn, m, n, k):
    """Rows as column ranges of wider buffers, at every kind of offset; what
    lies beside them is neither used nor written."""
    a0, sa, b0, sb, bias = operands(m + n, m, n, k)
    for t in (torch.float16, torch.float32):
        total = sums(a0, b0)
        for left, right in ((1, 0), (16, 16), (4, 12), (0, 3), (32, 0)):
            a = torch.full((m, left + k + right), 99, dtype=torch.int8, device="cuda")
            b = torch.full((n, right + k + left), 99, dtype=torch.int8, device="cuda")
            o = torch.full((m, left + n + right), 7.0, dtype=t, device="cuda")
            av, bv, ov = a[:, left:left + k], b[:, right:right + k], o[:, left:left + n]
            av.copy_(a0)
            bv.copy_(b0)
            check(fn.matmul_q8(av, sa, bv, sb, bias=bias, out=ov), total, sa, sb, bias, t)
            assert (o[:, :left] == 7).all() and (o[:, left + n:] == 7).all()


@pytest.mark.parametrize("m,n,k", [(1, 64, 128), (40, 300, 256), (600, 520, 160)])
def test_buffers_that_end_with_their_matrix(fn, m, n, k):
    """Operands at the very end of their allocations, guard bands around the
    output: nothing outside is written."""
    a0, sa, b0, sb, _ = operands(m + n, m, n, k)
    total = sums(a0, b0)
    for off in (0, 1, 16):
        a = torch.empty(off + m * k, dtype=torch.int8, device="cuda")[off:].view(m, k)
        b = torch.empty(off + n * k, dtype=torch.int8, device="cuda")[off:].view(n, k)
        a.copy_(a0)
        b.copy_(b0)
        o = torch.full((m * n + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = o[2048:-2048].view(m, n)
        check(fn.matmul_q8(a, sa, b, sb, out=out), total, sa, sb, None, torch.bfloat16)
        assert (o[:2048] == 7).all() and (o[-2048:] == 7).all()


def test_empty_products(fn):
    a, sa, b, sb, bias = operands(1, 5, 40, 64)
    assert fn.matmul_q8(a[:0], sa[:0], b, sb).shape == (0, 40)
    assert fn.matmul_q8(a, sa, b[:0], sb[:0]).shape == (5, 0)
    for m in (5, 300):
        a = torch.empty(m, 0, dtype=torch.int8, device="cuda")
        sa = torch.ones(m, device="cuda")
        out = fn.matmul_q8(a, sa, b[:, :0], sb, bias=bias, out_dtype=fn.FN_OUT_FP32)
        assert torch.equal(out, bias.expand(m, 40))
        assert not fn.matmul_q8(a, sa, b[:, :0], sb).any()


def test_scales_and_bias_that_are_not_numbers(fn):
    """A NaN or infinite scale reaches its own row or channel alone."""
    a, sa, b, sb, bias = operands(3, 70, 90, 256)
    want = fn.matmul_q8(a, sa, b, sb, bias=bias, out_dtype=fn.FN_OUT_FP32)
    sa[4], sb[7], bias[9] = float("nan"), float("nan"), float("inf")
    got = fn.matmul_q8(a, sa, b, sb, bias=bias, out_dtype=fn.FN_OUT_FP32)
    assert torch.isnan(got[4]).all() and torch.isnan(got[:, 7]).all()
    keep_r, keep_c = torch.arange(70) != 4, torch.arange(90) != 7
    inner = got[keep_r][:, keep_c]
    w = want[keep_r][:, keep_c].clone()
    w[:, 8] = float("inf")  # channel 9 once channel 7 is left out
    assert torch.equal(inner, w)


def test_leading_dimensions_graph_and_stream(fn):
    a, sa, b, sb, bias = operands(3, 60, 200, 256)
    want = fn.matmul_q8(a, sa, b, sb, bias=bias)
    got = fn.matmul_q8(a.view(3, 4, 5, 256), sa.view(3, 4, 5), b, sb, bias=bias)
    assert got.shape == (3, 4, 5, 200) and torch.equal(got.view(60, 200), want)
    assert torch.equal(fn.matmul_q8(a[0], sa[0], b, sb, bias=bias), want[0])
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    fn.matmul_q8(a, sa, b, sb, bias=bias, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn.matmul_q8(a, sa, b, sb, bias=bias, out=out)
    for _ in range(5):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        fn.matmul_q8(a, sa, b, sb)


def test_norm_then_product_is_the_linear_layer(fn):
    """rms_norm_q8 -> matmul_q8 against the unquantised layer: each side's
    codes are off by at most half a step, so |y - want| <= the sum over k of
    (|x_k| step_w + |w_k| step_x + step_x step_w / 2) / 2."""
    t = torch.float16
    g = torch.Generator().manual_seed(1)
    x = torch.randn(37, 768, generator=g).to(t).cuda()
    w = (torch.randn(300, 768, generator=g) / 28).to(t).cuda()
    nw = torch.ones(768, dtype=t, device="cuda")
    qx, sx, _ = fn.rms_norm_q8(x, nw)
    qw, sw = fn.quantize_rows(w)
    y = fn.matmul_q8(qx, sx, qw, sw, out_dtype=fn.FN_OUT_FP32)
    n = x.double() / torch.sqrt(x.double().square().mean(1, keepdim=True) + 1e-6)
    want = n @ w.double().t().contiguous()
    step_x, step_w = sx.double()[:, None], sw.double()[None, :]
    bound = 0.5 * (n.abs().sum(1)[:, None] * step_w + step_x * w.double().abs().sum(1)[None, :]
                   + 768 * step_x * step_w / 2) * 1.001
    assert bool(((y.double() - want).abs() <= bound).all())


def test_refusals_on_device_buffers(fn):
    a, sa, b, sb, bias = operands(1, 8, 32, 64)
    o = torch.zeros(8, 32, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fn.FnError, match="overlap"):
        fn.matmul_q8(o.view(torch.int8), sa, b, sb, out=o)
    with pytest.raises(fn.FnError, match="available"):
        fn.fn_matmul_q8(a, 64, sa, b, 64, sb, None, 8, 1 << 20, 64, 0, o, 1 << 20)
    with pytest.raises(fn.FnError, match="b_scales_dev"):
        fn.fn_matmul_q8(a, 64, sa, b, 64, None, None, 8, 32, 64, fn.FN_OUT_BF16, o, 32)
    for bad in (lambda: fn.matmul_q8(a, sa, b[:, :63], sb), lambda: fn.matmul_q8(a.float(), sa, b, sb),
                lambda: fn.matmul_q8(a, sa[:7], b, sb), lambda: fn.matmul_q8(a, sa, b, sb.half()),
                lambda: fn.matmul_q8(a, sa, b, sb, bias=bias.half()),
                lambda: fn.matmul_q8(a, sa, b, sb, out_dtype=2),
                lambda: fn.matmul_q8(a, sa, b.t().contiguous().t(), sb),
                lambda: fn.matmul_q8(a, sa, b, sb, out=o[:7])):
        with pytest.raises(ValueError):
            bad()
    assert not o.any()
