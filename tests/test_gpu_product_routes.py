"""The 8-bit product on every kernel that its sizes choose between, with edges
that no tile divides, and beyond 4 GiB.  Expected values and tolerance as in
test_gpu_product.py: bit for bit with the documented fp32 steps."""
from __future__ import annotations

import pytest
import torch

from test_gpu_product import TYPES, check, expected, operands, sums

pytestmark = pytest.mark.gpu

# (m, n, k): on a device of 256 compute units, rows at multiples of 16 bytes
# where k is one
ROUTES = {
    "few tokens, groups of 16 channels": (13, 4091, 400),
    "few tokens, groups of 64 channels": (9, 8501, 272),
    "few tokens, groups of 64 channels, whole": (16, 16384, 256),
    "32 x 32 groups": (61, 4001, 1040),
    "128 x 64 tiles, the second row in part": (150, 6001, 400),
    "64 x 64 tiles": (100, 4001, 400),
    "128 x 64 tiles": (500, 4090, 272),
    "128 x 128 tiles": (4090, 2040, 400),
    "256 x 256 tiles": (4090, 4070, 400),
    "256 x 256 tiles, whole": (4096, 4096, 128),
    "256 x 256 tiles, one stage in part": (4095, 4095, 48),
    "whole rounds of 256 x 256 tiles, and the rest": (16677, 1024, 1296),
    "whole rounds of 256 x 256 tiles, and a few tokens": (8195, 2047, 2048),
    "any row, few tokens": (11, 5001, 1033),
    "any row, 32 x 16 groups": (100, 1001, 2049),
    "any row, 64 x 64 tiles": (700, 1001, 333),
    "any row, 128 x 64 tiles": (2001, 1003, 517),
    "any row, 256 x 128 tiles": (3901, 4003, 301),
    "any row, a few codes": (3001, 2003, 7),
}


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("route", list(ROUTES))
def test_every_route(fn, route, t):
    m, n, k = ROUTES[route]
    a, sa, b, sb, bias = operands(m + n + k, m, n, k)
    total = sums(a, b)
    guard = torch.full((m * n + 4096,), 7.0, dtype=t, device="cuda")
    out = guard[2048:-2048].view(m, n)
    check(fn.matmul_q8(a, sa, b, sb, bias=bias, out=out), total, sa, sb, bias, t)
    assert (guard[:2048] == 7).all() and (guard[-2048:] == 7).all()


@pytest.mark.parametrize("route", list(ROUTES))
def test_the_same_bits_every_time(fn, route):
    """Twenty calls in a row, nothing between them: stages of one tile never
    mix with the next one's."""
    m, n, k = ROUTES[route]
    a, sa, b, sb, bias = operands(1, m, n, k)
    outs = [fn.matmul_q8(a, sa, b, sb, bias=bias) for _ in range(20)]
    want = expected(sums(a, b), sa, sb, bias, torch.bfloat16)
    assert torch.equal(outs[0].cpu(), want)
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("m,stride", [(600, 8_000_000), (600, 8_000_003), (150, 40_000_000),
                                      (16, 300_000_000)])
def test_operand_rows_far_apart(fn, m, stride):
    """Row offsets beyond 2^32 bytes, at strides that the tile kernels take and
    at strides that only the others can."""
    n, k = 200, 272
    a, sa, b, sb, bias = operands(m, m, n, k)
    big = torch.empty((m - 1) * stride + k, dtype=torch.int8, device="cuda")
    far = big.as_strided((m, k), (stride, 1))
    far.copy_(a)
    check(fn.matmul_q8(far, sa, b, sb, bias=bias), sums(a, b), sa, sb, bias, torch.bfloat16)
    # the same matrix as the channels
    check(fn.matmul_q8(b, sb, far, sa), sums(b, a), sb, sa, None, torch.bfloat16)


@pytest.mark.parametrize("m,n,k", [(70_000, 33_000, 32), (70_001, 33_001, 15), (12, 300_000_000, 16)])
def test_outputs_beyond_4_gib(fn, m, n, k):
    a, sa, b, sb, _ = operands(5, m, min(n, 40_000), k)
    if n > b.size(0):
        b, sb = b.repeat(n // b.size(0) + 1, 1)[:n], sb.repeat(n // sb.size(0) + 1)[:n]
    out = fn.matmul_q8(a, sa, b, sb)
    assert out.numel() * out.element_size() > 2 ** 32
    rows = torch.tensor([0, 1, m // 2, m - 1], device="cuda")
    cols = torch.cat([torch.arange(0, 300, device="cuda"),
                      torch.arange(n // 2, n // 2 + 300, device="cuda"),
                      torch.arange(n - 300, n, device="cuda")])
    got = out[rows][:, cols]
    want = expected(sums(a[rows], b[cols]), sa[rows], sb[cols], None, torch.bfloat16)
    assert torch.equal(got.cpu(), want)
    # every 997th row whole, on the device, by the same fp32 steps
    some = torch.arange(0, m, 997, device="cuda") if m > 1000 else rows[:1]
    for r in some.split(4):
        y = sums(a[r], b).float() * sa[r][:, None] * sb[None, :]
        assert torch.equal(out[r], y.to(torch.bfloat16))


@pytest.mark.parametrize("m,n", [(1000, 600), (1500, 1700), (2100, 2000), (4090, 2040)])
@pytest.mark.parametrize("k,a_stride,a_from,b_stride,b_from",
                         [(16, 16, 0, 16, 0), (112, 144, 16, 112, 0), (128, 128, 112, 256, 16),
                          (144, 144, 0, 400, 128), (400, 464, 48, 400, 0), (1040, 1040, 0, 1040, 0),
                          (1152, 1168, 0, 1152, 64), (1264, 1280, 0, 1264, 32)])
def test_rows_off_the_cache_lines(fn, m, n, k, a_stride, a_from, b_stride, b_from):
    """Rows of whole 16-byte pieces that start at other places than multiples
    of 128 bytes, each operand at its own."""
    a, sa, b, sb, bias = operands(m + n + k, m, n, k)

    def placed(v, stride, start):
        # nothing but the operand's own codes may reach the sums
        flat = torch.full((start + v.size(0) * stride,), 77, dtype=torch.int8, device="cuda")
        at = flat[start:].view(v.size(0), stride)[:, :k]
        at.copy_(v)
        return at

    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    fn.matmul_q8(placed(a, a_stride, a_from), sa, placed(b, b_stride, b_from), sb, bias=bias,
                 out=out)
    check(out, sums(a, b), sa, sb, bias, torch.bfloat16)
