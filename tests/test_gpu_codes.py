"""Codes against the exact 127 t / A in 64 bits, not the steps by which the
kernels come to them.

Bound: RN32(1 / A), times 127, times t: three roundings of at most u = 2^-24
each, of a value of at most 127, so a code is the nearest to 127 t / A unless
that lies within 127 * 3 u (and a little for their products) of half way
between two codes, and then it is one of the two.  For fp32 rows the norm's
t = h w and A are rounded themselves: two more."""
from __future__ import annotations

import pytest
import torch

from conftest import ROOT  # noqa: F401
from test_gpu_rows import EPS, TYPES, U, rows, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


def check_codes(codes, t, roundings):
    exact = 127 * t / t.abs().amax(1, keepdim=True).clamp(min=1e-300)
    off = (codes.double() - exact).abs()
    assert bool((off <= 0.5 + 127 * (roundings + 0.01) * U).all()), off.max().item()
    # away from half way it is the nearest, and nothing else
    clear = ((exact - exact.floor()) - 0.5).abs() > 127 * (roundings + 0.01) * U
    assert torch.equal(codes[clear], exact.round().to(torch.int8)[clear])
    assert clear.double().mean() > 0.9


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("n,width", [(400, 5), (400, 768), (300, 1021), (40, 4096), (41, 5003), (20, 12344),
                                     (5, 33001)])
def test_codes_are_the_nearest(fn, n, width, t):
    x, r, w = rows(1, n, width, t), rows(2, n, width, t), weights(3, width, t)
    codes, _ = fn.quantize_rows(x)
    check_codes(codes, x.double(), 3)
    codes, _, h = fn.rms_norm_q8(x, w, EPS, residual=r)
    check_codes(codes, h.double() * w.double(), 5 if t == torch.float32 else 3)


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16], ids=str)
def test_values_half_way_get_one_of_the_two(fn, t):
    """Rows whose largest value is 254: every odd number is half way."""
    x = torch.arange(-254, 255, dtype=torch.float32).to(t).repeat(3, 1).cuda()
    codes, scales = fn.quantize_rows(x)
    assert (codes[:, 0] == -127).all() and (codes[:, -1] == 127).all()
    assert bool(((codes.double() - x.double() / 2).abs() <= 0.5).all())
    assert bool((codes.double() - x.double() / 2)[:, ::2].abs().max() == 0)
    assert bool(((scales.double() - 2).abs() <= 2 * U).all())
