"""Many wide fp32 rows, which the row kernels read past the caches by a rule on
their number, width and place: the bits are those of the same rows a few at a
time, and dweight is its formula's.

A column's sum of n terms in groups of rows is off by at most (n + 14) u of the
terms' magnitudes: a term has three roundings, a chain no more than n additions."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


# rows x width of 2^23 elements or more in every shape of threads from 256 on, full and
# not, on whole lines and off them; and one row fewer than that
SIZES = [(2048, 4096), (2047, 4096), (2500, 3584), (2600, 3528), (2050, 4095), (1640, 5120), (1641, 5119), (1366, 6144),
         (1024, 8192), (1023, 8192), (1200, 7001), (512, 16384), (511, 16384), (600, 14336), (600, 14335), (700, 12288),
         (256, 32768), (255, 32768), (300, 28001)]


def rows(seed, n, width, pad):
    """n x width; with a pad, columns of a wider buffer that start off the lines."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, width + pad, generator=g, device="cuda")[:, pad:]


@pytest.mark.parametrize("pad", [0, 1, 32])
@pytest.mark.parametrize("n,width", SIZES)
def test_many_rows_are_those_of_a_few(fn, n, width, pad):
    x, r, dout, dsum = (rows(k, n, width, pad) for k in range(4))
    w = torch.rand(width, device="cuda") + 0.5
    out, rstd, _ = fn.rms_norm(x, w, EPS)
    out_r, rstd_r, h = fn.rms_norm(x, w, EPS, residual=r)
    codes, scales = fn.quantize_rows(x)
    norm_codes, norm_scales, _ = fn.rms_norm_q8(x, w, EPS)
    dx, dw = fn.rms_norm_backward(dout, h, w, rstd_r)
    dx_s, dw_s = fn.rms_norm_backward(dout, h, w, rstd_r, dsum=dsum)
    assert torch.equal(dw_s, dw)
    assert torch.equal(h, x + r)
    for a in (0, 1, n // 2, n - 7):
        part = slice(a, a + 7)
        few, few_rstd, _ = fn.rms_norm(x[part], w, EPS)
        assert torch.equal(out[part], few) and torch.equal(rstd[part], few_rstd)
        few, few_rstd, _ = fn.rms_norm(x[part], w, EPS, residual=r[part])
        assert torch.equal(out_r[part], few) and torch.equal(rstd_r[part], few_rstd)
        few, few_scales = fn.quantize_rows(x[part])
        assert torch.equal(codes[part], few) and torch.equal(scales[part], few_scales)
        few, few_scales, _ = fn.rms_norm_q8(x[part], w, EPS)
        assert torch.equal(norm_codes[part], few) and torch.equal(norm_scales[part], few_scales)
        for d, s in ((dx, None), (dx_s, dsum)):
            few, _ = fn.rms_norm_backward(dout[part], h[part], w, rstd_r[part], dsum=None if s is None else s[part])
            assert torch.equal(d[part], few)
    terms = dout.double() * (h.double() * rstd_r.double()[:, None])
    off = (dw.double() - terms.sum(0)).abs()
    assert (off <= (n + 14) * U * terms.abs().sum(0)).all()
    # in the place of inputs
    a, c = x.clone(), r.clone()
    got = fn.rms_norm(a, w, EPS, residual=c, out=a, sum_out=c)
    assert torch.equal(a, out_r) and torch.equal(c, h) and torch.equal(got[1], rstd_r)
    a = dout.clone()
    assert torch.equal(fn.rms_norm_backward(a, h, w, rstd_r, dsum=dsum, dx=a)[0], dx_s)
