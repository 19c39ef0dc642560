"""Gradients of rows of odd width beyond 2,560 elements at odd and at even row
strides.  16-bit rows at an odd stride of dout are worked on from another
first element where their number is odd: dx then differs by the rounding of
the row's mean at most, dweight not at all.

Tolerance: u = 2^-24; mean(g n) of D terms is a chain of at most `chain`
additions, so two orders of it differ by 2 chain u mean|g n|, and dx by rstd |n|
times that, before either is rounded to its type (half a step each)."""
from __future__ import annotations

import pytest
import torch

from conftest import ROOT  # noqa: F401
from test_gpu_rows import EPS, TYPES, U, backward_reference, check_close, half, rows, tiny, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


def chain(width: int) -> int:
    """Additions on the longest path to a row's sum: a thread's own chunks of
    eight, 6 steps across the wavefront, and the wavefronts."""
    threads = 256 if width <= 6144 else 512
    return 8 * -(-width // (8 * threads)) + 6 + threads // 64


def at_stride(x, stride):
    big = torch.full((x.size(0), stride), float("nan"), dtype=x.dtype, device=x.device)
    big[:, :x.size(1)] = x
    return big[:, :x.size(1)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("n,width", [(2, 2561), (3, 2561), (600, 2561), (601, 3001), (301, 4095),
                                     (600, 4097), (523, 5003), (600, 8191), (300, 8193), (600, 12345),
                                     (257, 16383)])
def test_gradients_at_odd_and_even_strides(fn, n, width, t):
    h, w = rows(width, n, width, t), weights(width, width, t)
    dout, dsum = rows(width + 1, n, width, t, 0.2), rows(width + 2, n, width, t, 0.2)
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + EPS)).float()
    want, size, dw, dw_size = backward_reference(dout, h, w, rstd, dsum)
    r, nd = rstd.double()[:, None], h.double() * rstd.double()[:, None]
    gn = (dout.double() * w.double() * nd).abs().mean(1, keepdim=True)
    order = 2 * chain(width) * U * (r * nd).abs() * gn
    dx0, dw0 = fn.rms_norm_backward(dout, h, w, rstd, dsum=dsum)
    for strides in ((1, 1, 1), (1, 0, 2), (3, 3, 3), (0, 1, 1), (2, 5, 0)):
        args = [at_stride(v, width + s) for v, s in zip((dout, h, dsum), strides)]
        out = at_stride(torch.zeros_like(h), width + strides[0])
        dx, dweight = fn.rms_norm_backward(args[0], args[1], w, rstd, dsum=args[2], dx=out)
        check_close(dx, want, want.abs() * half(t) + size + order + tiny(t), "dx")
        assert torch.equal(dweight, dw0)
        # the even rows, and all at a stride as odd as the width, are the same bits
        same = slice(None) if strides[0] % 2 == 0 or t == torch.float32 else slice(0, None, 2)
        assert torch.equal(dx[same], dx0[same])
        off = (dx.double() - dx0.double()).abs()
        assert bool((off <= 2 * half(t) * (want.abs() + order + size) + order + 2 * tiny(t)).all())
