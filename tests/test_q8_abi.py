"""Refusals of the 8-bit linear layer's entry points on the CPU: every invalid
argument gives its documented code and a message that names it, before
anything is launched; calls without rows need no buffers."""
from __future__ import annotations

import ctypes

import pytest

from conftest import ROOT  # noqa: F401


@pytest.fixture(scope="module")
def b():
    from augmentation_amd import binding
    return binding


NORM = dict(x=None, x_stride=64, residual=None, residual_stride=0, weight=None, rows=4, width=64,
            eps=1e-6, dtype=1, sum=None, sum_stride=0)


def norm(b, q8, **kw):
    a = dict(NORM, out=None, out_stride=64, scales=None, rstd=None, **{})
    a.update(kw)
    head = [a[k] for k in NORM]
    if q8:
        return b._lib.fn_rms_norm_q8(*head, a["out"], a["out_stride"], a["scales"], a["rstd"], None)
    return b._lib.fn_rms_norm(*head, a["out"], a["out_stride"], a["rstd"], None)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kw,code,word", [
    (dict(rows=-1), -1, "rows"), (dict(width=0), -1, "width"), (dict(width=-5), -1, "width"),
    (dict(width=2**30 + 1), -2, "width"), (dict(rows=2**40 + 1), -2, "rows"),
    (dict(dtype=2), -1, "dtype"), (dict(dtype=4), -1, "dtype"), (dict(dtype=-1), -1, "dtype"),
    (dict(eps=0.0), -1, "eps"), (dict(eps=-1.0), -1, "eps"), (dict(eps=float("nan")), -1, "eps"),
    (dict(eps=float("inf")), -1, "eps"),
    (dict(residual=4096), -1, "together"), (dict(sum=4096), -1, "together"),
    (dict(x_stride=-64), -1, "negative"), (dict(out_stride=63), -1, "shorter"),
    (dict(residual=4096, sum=8192, sum_stride=63), -1, "shorter"),
    (dict(residual=4096, sum=8192, sum_stride=64, residual_stride=-1), -1, "negative"),
    (dict(x_stride=2**62), -2, "x_dev"), (dict(rows=2**39, x_stride=2**30), -2, "x_dev"),
    (dict(), -1, "x_dev is NULL"), (dict(x=4097), -1, "aligned"),
])
def test_norm_refusals(b, q8, kw, code, word):
    assert norm(b, q8, **kw) == code
    assert word in b.fn_last_error()


@pytest.mark.parametrize("q8", [False, True])
def test_norm_of_no_rows(b, q8):
    assert norm(b, q8, rows=0) == 0
    assert b.fn_last_error() == ""
    assert norm(b, q8, rows=0, out_stride=0, x_stride=0, width=2**30) == 0


@pytest.mark.parametrize("kw,code,word", [
    (dict(rows=-1), -1, "rows"), (dict(width=0), -1, "width"), (dict(width=2**30 + 1), -2, "width"),
    (dict(dtype=2), -1, "dtype"), (dict(x_stride=-1), -1, "negative"),
    (dict(codes_stride=3), -1, "shorter"), (dict(), -1, "x_dev is NULL"),
    (dict(codes_stride=2**62), -2, "codes_dev"), (dict(x=4098), -1, "aligned"),
])
def test_quantize_refusals(b, kw, code, word):
    a = dict(x=None, x_stride=64, rows=4, width=64, dtype=0, codes=None, codes_stride=64,
             scales=None)
    a.update(kw)
    assert b._lib.fn_quantize_rows(*a.values(), None) == code
    assert word in b.fn_last_error()
    a["rows"] = 0
    if code == -1 and word == "x_dev is NULL":
        assert b._lib.fn_quantize_rows(*a.values(), None) == 0


BACK = dict(dout=None, dout_stride=64, h=None, h_stride=64, weight=None, rstd=None, dsum=None,
            dsum_stride=0, rows=4, width=64, dtype=1, dx=None, dx_stride=64, dweight=None,
            workspace=None, workspace_bytes=1 << 20)


@pytest.mark.parametrize("kw,code,word", [
    (dict(rows=-1), -1, "rows"), (dict(width=0), -1, "width"), (dict(dtype=7), -1, "dtype"),
    (dict(rows=4000, workspace_bytes=0), -1, "workspace"), (dict(h_stride=-2), -1, "negative"),
    (dict(dx_stride=1), -1, "shorter"), (dict(dsum=4096, dsum_stride=-1), -1, "negative"),
    (dict(), -1, "dout_dev is NULL"), (dict(rows=0), -1, "dweight_dev is NULL"),
])
def test_backward_refusals(b, kw, code, word):
    a = dict(BACK, **kw)
    assert b._lib.fn_rms_norm_backward(*a.values(), None) == code
    assert word in b.fn_last_error()


def test_backward_workspace_sizes(b):
    n = ctypes.c_int64(-1)
    assert b._lib.fn_rms_norm_backward_workspace(4, 64, None) == -1
    assert b._lib.fn_rms_norm_backward_workspace(-1, 64, ctypes.byref(n)) == -1
    assert b._lib.fn_rms_norm_backward_workspace(4, 2**30 + 1, ctypes.byref(n)) == -2
    assert b.fn_rms_norm_backward_workspace(0, 64) == 0
    last = 0
    for rows in (1, 5, 100, 10_000, 10_000_000):
        size = b.fn_rms_norm_backward_workspace(rows, 768)
        # whole rows of partial sums, more of them for more rows, up to a
        # limit; none where one work-group's sums are the gradient
        assert size >= last and size % (768 * 4) == 0 and size <= 4096 * 768 * 4
        assert (size == 0) == (rows <= 5)
        last = size
    # wide rows add one fp32 number for each row
    wide = b.fn_rms_norm_backward_workspace(1000, 50_000)
    assert wide % 4 == 0 and 50_000 * 4 + 4000 <= wide <= 64 * 50_000 * 4 + 4000


MUL = dict(a=None, a_stride=64, sa=None, b=None, b_stride=64, sb=None, bias=None, M=4, N=8, K=64,
           out_dtype=0, out=None, out_stride=8)


@pytest.mark.parametrize("kw,code,word", [
    (dict(M=-1), -1, "M, N and K"), (dict(N=-1), -1, "M, N and K"), (dict(K=-1), -1, "M, N and K"),
    (dict(K=131072), -2, "131071"), (dict(M=2**40 + 1), -2, "M or N"),
    (dict(N=2**40 + 1, out_stride=2**41), -2, "M or N"),
    (dict(out_dtype=2), -1, "out_dtype"), (dict(a_stride=-1), -1, "negative"),
    (dict(b_stride=-1), -1, "negative"), (dict(out_stride=7), -1, "shorter"),
    (dict(), -1, "a_dev is NULL"), (dict(K=0), -1, "a_scales_dev is NULL"),
    (dict(K=0, sa=4098), -1, "aligned"),
])
def test_product_refusals(b, kw, code, word):
    a = dict(MUL, **kw)
    assert b._lib.fn_matmul_q8(*a.values(), None) == code
    assert word in b.fn_last_error()


def test_empty_products_need_no_buffers(b):
    for kw in (dict(M=0), dict(N=0, out_stride=0), dict(M=0, K=0)):
        assert b._lib.fn_matmul_q8(*dict(MUL, **kw).values(), None) == 0, b.fn_last_error()


def test_helpers_refuse_host_tensors_and_wrong_shapes(b):
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        b.quantize_rows(x)
    with pytest.raises(ValueError):
        b.rms_norm(x, torch.ones(8))
    with pytest.raises(ValueError):
        b.rms_norm_q8(x, torch.ones(8))
    with pytest.raises(ValueError):
        b.rms_norm_backward(x, x, torch.ones(8), torch.ones(4))
    with pytest.raises(ValueError):
        b.matmul_q8(x.to(torch.int8), torch.ones(4), x.to(torch.int8), torch.ones(4))


def test_row_stride_of_views(b):
    import torch
    t = torch.zeros(4, 6, 10)
    assert b._row_stride(t, "t") == 10
    assert b._row_stride(t[:, :, 2:7], "t") == 10
    assert b._row_stride(t[:, 0], "t") == 60
    assert b._row_stride(t[0, 0], "t") == 10
    assert b._row_stride(torch.zeros(1, 10).expand(24, 10), "t") == 0
    assert b._row_stride(torch.zeros(1, 10).expand(4, 6, 10), "t") == 0
    assert b._row_stride(torch.zeros(0, 10), "t") == 10
    assert b._row_stride(t[:, :, :1], "t") == 10
    for bad in (t[:, :3], t.transpose(0, 1), t[:, :, ::2], t.transpose(1, 2)):
        with pytest.raises(ValueError):
            b._row_stride(bad, "t")
