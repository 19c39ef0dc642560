"""Gradients of rows so wide that the sum of the partial rows takes more than
one launch (2^32 threads, of which HIP starts fewer at a time).

Tolerances: u = 2^-24.  With one row, dweight is dout (h rstd), two fp32
roundings, and its sums add nothing but zeros: compared bit for bit.  A
row's mean of D terms is a chain of 8 ceil(D / 8192) additions in a thread, 6
across the wavefront and 16 across the wavefronts."""
from __future__ import annotations

import pytest
import torch

from conftest import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


@pytest.mark.parametrize("width", [2**28 - 8, 2**28 + 77])
def test_gradients_of_one_row_wider_than_a_launch(fn, width):
    t = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(width)
    dout, h, w = (torch.randn(1, width, generator=g, device="cuda", dtype=t) for _ in range(3))
    rstd = torch.full((1,), 0.75, device="cuda")
    guard = torch.full((width + 64,), 9.0, device="cuda")
    dx, dweight = fn.rms_norm_backward(dout, h, w[0], rstd, dweight=guard[32:-32])
    n = h.float() * rstd
    assert torch.equal(dweight, (dout.float() * n)[0])
    assert (guard[:32] == 9).all() and (guard[-32:] == 9).all()
    gr = dout.float() * w.float()
    mean, size = 0.0, 0.0
    for a, b in zip(gr[0].split(1 << 24), n[0].split(1 << 24)):
        terms = a.double() * b.double()
        mean, size = mean + terms.sum().item() / width, size + terms.abs().sum().item() / width
    chain = 8 * -(-width // 8192) + 6 + 16
    for at in range(0, width, 1 << 24):
        sl = slice(at, at + (1 << 24))
        r, gd, nd = rstd.double(), gr[0, sl].double(), n[0, sl].double()
        want = r * (gd - nd * mean)
        tol = want.abs() * 2.0 ** -8 + 8 * U * (r * gd).abs() + (chain + 8) * U * r * nd.abs() * size
        assert ((dx[0, sl].double() - want).abs() <= tol).all(), at


def test_gradient_of_no_rows_wider_than_a_launch(fn):
    width = 2**28 + 77
    dweight = torch.full((width,), 5.0, device="cuda")
    none = torch.empty(0, width, dtype=torch.bfloat16, device="cuda")
    # no rows: the weight is not read
    w = torch.empty(1, dtype=torch.bfloat16, device="cuda").expand(width)
    assert fn.fn_rms_norm_backward(none, width, none, width, w, none, None, 0, 0, width,
                                   fn.FN_OUT_BF16, none, width, dweight, None, 0) == 0
    assert not dweight.any()
