"""More rows than there are work-groups, where a work-group has one row at a
time: the loop over rows, the halves of the reduction's LDS in turn, chunks
shifted for odd rows, the next row under way in the backward pass, and sums of
dweight over several rows.

The forward kernels have at most 2^20 work-groups (one row each from 2,561
elements on), the backward ones 256, or 512.  (test_many_rows in
test_gpu_rows.py stays below both: four and 256 of its rows share a
work-group.)  Tolerances as in test_gpu_rows.py, with the chains of additions
that the sizes give (depth() there has too few for 16-bit rows of 8,193 to
16,384 elements: 64 of a thread's own, not 32)."""
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


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("width", [2563, 2564])
def test_more_rows_than_work_groups(fn, width, t):
    n, step = (1 << 20) + 777, 1 << 16
    g = torch.Generator(device="cuda").manual_seed(width)
    x = torch.empty(n, width, dtype=t, device="cuda")
    for at in range(0, n, step):
        part = x[at:at + step]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    w = weights(3, width, t)
    # 16 of a thread's own, 6 steps across the wavefront, 4 wavefronts
    rel = (26 / 2 + 6) * U
    codes, scales = fn.quantize_rows(x)
    codes8, scales8, _ = fn.rms_norm_q8(x, w, EPS)
    out, rstd, _ = fn.rms_norm(x, w, EPS)

    def codes_of(v):
        top = v.abs().amax(1)
        inverse = 127.0 * (1.0 / top.double()).float()
        return torch.round(v * inverse[:, None]).to(torch.int8), top.double() / 127

    for at in range(0, n, step):
        sl = slice(at, at + step)
        v = x[sl].float()
        want, scale = codes_of(v)
        assert torch.equal(codes[sl], want), at
        assert ((scales[sl].double() - scale).abs() <= scale * U).all()
        r = 1 / torch.sqrt(x[sl].double().square().mean(1) + EPS)
        assert ((rstd[sl].double() - r).abs() <= r * rel).all()
        want, scale = codes_of(v * w.float())
        assert torch.equal(codes8[sl], want), at
        assert ((scales8[sl].double() - scale * r).abs() <= scale * r * (rel + 3 * U)).all()
        y = x[sl].double() * r[:, None] * w.double()
        assert ((out[sl].double() - y).abs() <= y.abs() * (half(t) + rel + 2 * U) + tiny(t)).all(), at


# width: (rows that a work-group has at a time, work-groups at most, slices)
SHAPES = {100: (16, 512), 768: (8, 512), 1500: (4, 256), 2560: (4, 256), 4097: (1, 256),
          5003: (1, 256), 6144: (1, 256), 8191: (1, 256), 12345: (1, 256), 16384: (1, 256),
          16385: (1, 64), 40001: (1, 64)}


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("n", [2, 1100])
@pytest.mark.parametrize("width", list(SHAPES))
def test_weight_gradients_over_several_rows_of_a_work_group(fn, width, n, t):
    n = min(n, 600) if width > 8192 else n
    h, w = rows(width, n, width, t), weights(width, width, t)
    dout, dsum = rows(width + 1, n, width, t, 0.2), rows(width + 2, n, width, t, 0.2)
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + EPS)).float()
    dx, dweight = fn.rms_norm_backward(dout, h, w, rstd, dsum=dsum)
    want, size, dw, dw_size = backward_reference(dout, h, w, rstd, dsum)
    # a row's mean: up to 40 of a thread's own in registers, 8 for each 8,192
    # elements beyond 16,384
    own = 40 if width <= 16384 else 8 * -(-width // 8192)
    r, gn = rstd.double()[:, None], (dout.double() * w.double() * h.double() * rstd.double()[:, None])
    size = size + (own + 22) * U * (r * h.double() * r).abs() * gn.abs().mean(1, keepdim=True)
    check_close(dx, want, want.abs() * half(t) + size + tiny(t), "dx")
    # a column: a thread's rows, the rows of a work-group, the partial sums (64
    # at a time, 4 of these, 4 steps), and the product's two roundings
    at_once, most = SHAPES[width]
    groups = min(-(-n // at_once), most)
    if groups <= 2 and at_once * 2 >= n and width <= 16384:
        groups = 1
    chain = -(-n // (groups * at_once)) + (at_once - 1).bit_length() + -(-groups // 64) + 4 + 4 + 2
    check_close(dweight, dw, dw_size * chain * U + tiny(torch.float32), "dweight")
