"""What the 16-bit gradients of the linear cross entropy are scaled by: the
largest finite |dloss| among the rows that count, found by every work-group for
up to 8,192 rows and in a launch of its own for more."""
from __future__ import annotations

import pytest
import torch

from test_gpu_cross_entropy import check_backward, head

pytestmark = pytest.mark.gpu

HALVES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


@pytest.mark.parametrize("t", [torch.float32, *HALVES], ids=str)
@pytest.mark.parametrize("rows", [300, 8192, 8193, 20011])
def test_an_ignored_row_has_no_say_in_the_scale(fn, rows, t):
    """Whatever stands among dlosses where rows are ignored, the gradients are the
    bits that zeros there give."""
    x, w, y, b = head(rows, rows, 70, 40, t)
    ignored = torch.arange(rows, device="cuda") % 7 == 0
    ignored[-1] = True
    y = torch.where(ignored, torch.where(torch.arange(rows, device="cuda") % 2 == 0, -100, 70), y)
    ignored |= (y < 0) | (y >= 70)
    _, lse = fn.linear_cross_entropy(x, w, y, bias=b)
    d = torch.rand(rows, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") + 0.5
    want = fn.linear_cross_entropy_backward(torch.where(ignored, 0.0, d), x, w, y, lse, bias=b)
    assert (want[0][ignored] == 0).all() and (want[0][~ignored] != 0).any(1).all()
    for junk in (2.0**40, 1e30, -3e38, float("inf"), float("nan")):
        got = fn.linear_cross_entropy_backward(torch.where(ignored, junk, d), x, w, y, lse, bias=b)
        for p, q in zip(got, want):
            assert torch.equal(p, q), junk
    # nobody counts
    none = torch.full_like(y, -1)
    for p in fn.linear_cross_entropy_backward(d * 1e30, x, w, none, lse, bias=b):
        assert (p == 0).all()
    # one number for all, with and without its own place in every row
    one = torch.full((), 0.3, device="cuda")
    for p, q in zip(fn.linear_cross_entropy_backward(one.expand(rows), x, w, y, lse, bias=b),
                    fn.linear_cross_entropy_backward(one.repeat(rows), x, w, y, lse, bias=b)):
        assert torch.equal(p, q)


@pytest.mark.parametrize("t", HALVES, ids=str)
@pytest.mark.parametrize("rows", [1000, 8192, 8193, 20011])
def test_the_largest_is_found_wherever_it_stands(fn, rows, t):
    """One row's dloss is 1,024 times the others': in fp16 a search that missed it
    would scale its gradients to 2^24, which is infinite."""
    x, w, y, b = head(rows, rows, 33, 24, t)
    y = y.clamp(0, 32)
    _, lse = fn.linear_cross_entropy(x, w, y, bias=b)
    d = torch.rand(rows, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") + 0.5
    for at in (0, 65, 700, rows // 2, rows - 2, rows - 1):
        big = d.clone()
        big[at] = -1024.0 if at % 2 else 1024.0
        check_backward(fn, x, w, y, b, 0.1, big, lse)
