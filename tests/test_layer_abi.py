"""Refusals of dropout and layer norm on the CPU: every invalid argument gives
its documented code and a message that names it, before anything is launched;
calls without rows need no buffers; helpers refuse what they cannot keep."""
from __future__ import annotations

import ctypes

import pytest
import torch
from torch.autograd import forward_ad

from conftest import ROOT  # noqa: F401


@pytest.fixture(scope="module")
def b():
    from augmentation_amd import binding
    return binding


NAN = float("nan")
COMMON = [
    (dict(rows=-1), -1, "rows"), (dict(width=0), -1, "width"), (dict(width=2**30 + 1), -2, "width"),
    (dict(rows=2**40 + 1), -2, "rows"), (dict(dtype=2), -1, "dtype"), (dict(dtype=9), -1, "dtype"),
    (dict(p=-0.1), -1, "dropout_p"), (dict(p=1.5), -1, "dropout_p"), (dict(p=NAN), -1, "dropout_p"),
    (dict(first_row=-1), -1, "first_row"), (dict(first_row=2**63 - 2), -2, "first_row"),
]

DROP = dict(x=None, x_stride=64, residual=None, residual_stride=0, rows=4, width=64, p=0.1, seed=1,
            first_row=0, dtype=1, out=None, out_stride=64)


@pytest.mark.parametrize("kw,code,word", COMMON + [
    (dict(x_stride=-1), -1, "negative"), (dict(out_stride=63), -1, "shorter"),
    (dict(residual=4096, residual_stride=-1), -1, "negative"), (dict(x_stride=2**62), -2, "x_dev"),
    (dict(), -1, "x_dev is NULL"), (dict(x=4097), -1, "aligned"),
])
def test_dropout_refusals(b, kw, code, word):
    assert b._lib.fn_dropout(*dict(DROP, **kw).values(), None) == code
    assert word in b.fn_last_error()


NORM = dict(x=None, x_stride=64, residual=None, residual_stride=0, weight=None, bias=None, rows=4,
            width=64, eps=1e-5, p=0.0, seed=1, first_row=0, dtype=1, sum=None, sum_stride=0, out=None,
            out_stride=64, mean=None, rstd=None)


@pytest.mark.parametrize("kw,code,word", COMMON + [
    (dict(eps=0.0), -1, "eps"), (dict(eps=NAN), -1, "eps"), (dict(eps=float("inf")), -1, "eps"),
    (dict(residual=4096), -1, "sum_dev"), (dict(p=0.5), -1, "sum_dev"), (dict(sum=4096), -1, "sum_dev"),
    (dict(p=0.5, sum=4096, sum_stride=63), -1, "shorter"), (dict(out_stride=1), -1, "shorter"),
    (dict(x_stride=-64), -1, "negative"), (dict(), -1, "x_dev is NULL"), (dict(x=4098, dtype=0), -1, "aligned"),
])
def test_norm_refusals(b, kw, code, word):
    assert b._lib.fn_layer_norm(*dict(NORM, **kw).values(), None) == code
    assert word in b.fn_last_error()


BACK = dict(dout=None, dout_stride=64, h=None, h_stride=64, weight=None, mean=None, rstd=None, dsum=None,
            dsum_stride=0, rows=4, width=64, p=0.0, seed=1, first_row=0, dtype=1, dh=None, dh_stride=64,
            dx=None, dx_stride=0, dweight=None, dbias=None, workspace=None, workspace_bytes=1 << 30)


@pytest.mark.parametrize("kw,code,word", COMMON + [
    (dict(rows=4000, workspace_bytes=0), -1, "workspace"), (dict(p=0.5), -1, "dx_dev"),
    (dict(dx=4096), -1, "dx_dev"), (dict(p=0.5, dx=4096, dx_stride=3), -1, "shorter"),
    (dict(h_stride=-2), -1, "negative"), (dict(dh_stride=1), -1, "shorter"),
    (dict(), -1, "dout_dev is NULL"),
])
def test_backward_refusals(b, kw, code, word):
    assert b._lib.fn_layer_norm_backward(*dict(BACK, **kw).values(), None) == code
    assert word in b.fn_last_error()


def test_calls_without_rows(b):
    assert b._lib.fn_dropout(*dict(DROP, rows=0).values(), None) == 0
    assert b._lib.fn_layer_norm(*dict(NORM, rows=0).values(), None) == 0
    assert b._lib.fn_layer_norm(*dict(NORM, rows=0, p=0.5).values(), None) == 0
    assert b._lib.fn_layer_norm_backward(*dict(BACK, rows=0).values(), None) == 0
    assert b.fn_last_error() == ""


def test_workspace_sizes(b):
    n = ctypes.c_int64(-1)
    assert b._lib.fn_layer_norm_backward_workspace(4, 64, None) == -1
    assert b._lib.fn_layer_norm_backward_workspace(-1, 64, ctypes.byref(n)) == -1
    assert b._lib.fn_layer_norm_backward_workspace(4, 2**30 + 1, ctypes.byref(n)) == -2
    assert b.fn_layer_norm_backward_workspace(0, 64) == 0
    last = 0
    for rows in (1, 5, 100, 10_000, 10_000_000):
        size = b.fn_layer_norm_backward_workspace(rows, 768)
        assert size >= last and size % 16 == 0 and size <= 4096 * 768 * 8
        assert (size == 0) == (rows <= 5)
        last = size
    wide = b.fn_layer_norm_backward_workspace(1000, 50_000)
    assert wide % 16 == 0 and 50_000 * 8 + 8000 <= wide <= 64 * 50_000 * 8 + 8016


def calls(b):
    """(name, function, its float arguments)."""
    x, w, s = torch.ones(4, 8), torch.ones(8), torch.ones(4)
    return [
        ("dropout", lambda **k: b.dropout(p=0.1, seed=1, **k), dict(x=x, residual=x, out=x)),
        ("layer_norm", lambda **k: b.layer_norm(**k),
         dict(x=x, weight=w, bias=w, residual=x, out=x, sum_out=x, mean=s, rstd=s)),
        ("layer_norm_backward", lambda **k: b.layer_norm_backward(p=0.1, **k),
         dict(dout=x, h=x, weight=w, mean=s, rstd=s, dsum=x, dh=x, dx=x, dweight=w, dbias=w)),
    ]


CASES = [(name, arg) for name, _, args in calls(None) for arg in args]


@pytest.mark.parametrize("name,arg", CASES)
def test_lost_gradients_and_tangents_are_refused(b, name, arg):
    _, call, args = next(c for c in calls(b) if c[0] == name)
    leaf = dict(args, **{arg: args[arg].clone().requires_grad_()})
    with pytest.raises(ValueError, match="requires a gradient"):
        call(**leaf)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        call(**leaf)
    with forward_ad.dual_level():
        dual = dict(args, **{arg: forward_ad.make_dual(args[arg], torch.ones_like(args[arg]))})
        with pytest.raises(ValueError, match="tangent"):
            call(**dual)
        with pytest.raises(ValueError, match="CUDA"):
            call(**args)
