"""Refusals of the linear cross entropy on the CPU: every invalid argument gives
its documented code and a message that names it, before anything is launched;
the workspace's sizes; helpers refuse what they cannot keep."""
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
SIZES = [
    (dict(rows=-1), -1, "rows"), (dict(classes=0), -1, "classes"), (dict(classes=-3), -1, "classes"),
    (dict(width=0), -1, "width"), (dict(width=-1), -1, "width"), (dict(dtype=2), -1, "dtype"),
    (dict(dtype=-1), -1, "dtype"), (dict(rows=2**28 + 1), -2, "rows"), (dict(classes=2**28 + 1), -2, "classes"),
    (dict(width=2**20 + 1), -2, "width"), (dict(rows=2**20, classes=2**17), -2, "2^36"),
    (dict(rows=2**20, width=2**17), -2, "2^36"), (dict(classes=2**20, width=2**17), -2, "2^36"),
]
COMMON = SIZES + [
    (dict(smoothing=-0.1), -1, "smoothing"), (dict(smoothing=1.1), -1, "smoothing"), (dict(smoothing=NAN), -1, "smoothing"),
    (dict(workspace_bytes=0), -1, "workspace"), (dict(x_stride=-1), -1, "negative"), (dict(w_stride=-1), -1, "negative"),
    (dict(x_stride=2**62), -2, "x_dev"),
]

LOSS = dict(x=None, x_stride=64, weight=None, w_stride=64, bias=None, targets=None, rows=4, classes=10,
            width=64, smoothing=0.0, dtype=1, losses=None, lse=None, workspace=None, workspace_bytes=1 << 30)


@pytest.mark.parametrize("kw,code,word", COMMON + [(dict(), -1, "x_dev is NULL"), (dict(x=4097), -1, "aligned")])
def test_loss_refusals(b, kw, code, word):
    assert b._lib.fn_linear_cross_entropy(*dict(LOSS, **kw).values(), None) == code
    assert word in b.fn_last_error()


BACK = dict(dlosses=None, dlosses_stride=1, x=None, x_stride=64, weight=None, w_stride=64, bias=None,
            targets=None, lse=None, rows=4, classes=10, width=64, smoothing=0.0, dtype=1, dx=None,
            dx_stride=64, dweight=None, dw_stride=64, dbias=None, workspace=None, workspace_bytes=1 << 30)


@pytest.mark.parametrize("kw,code,word", COMMON + [
    (dict(), -1, "dlosses_dev is NULL"), (dict(dlosses_stride=-1), -1, "dlosses_stride"),
    (dict(dlosses_stride=2), -1, "dlosses_stride"), (dict(dx=4096, dx_stride=63), -1, "shorter"),
    (dict(dweight=4096, dw_stride=3), -1, "shorter"),
])
def test_backward_refusals(b, kw, code, word):
    assert b._lib.fn_linear_cross_entropy_backward(*dict(BACK, **kw).values(), None) == code
    assert word in b.fn_last_error()


def test_a_loss_of_no_rows(b):
    assert b._lib.fn_linear_cross_entropy(*dict(LOSS, rows=0).values(), None) == 0
    assert b.fn_last_error() == ""


@pytest.mark.parametrize("kw,code,word", SIZES)
def test_workspace_refusals(b, kw, code, word):
    a = dict(dict(rows=4, classes=10, width=64, dtype=1), **kw)
    n = ctypes.c_int64(-1)
    assert b._lib.fn_linear_cross_entropy_workspace(*a.values(), 1, 1, 0, ctypes.byref(n)) == code
    assert word in b.fn_last_error()
    assert b._lib.fn_linear_cross_entropy_workspace(4, 10, 64, 1, 1, 1, 0, None) == -1


def test_workspace_sizes(b):
    size = b.fn_linear_cross_entropy_workspace
    for backward in (0, 1):
        for dtype, e in ((0, 4), (1, 2), (3, 2)):
            for rows, classes, width in ((1, 10, 8), (256, 1000, 768), (8192, 50000, 4096), (0, 5, 3), (70000, 40, 33)):
                inside = size(rows, classes, width, dtype, 1, 1, backward)
                copied = size(rows, classes, width, dtype, 0, 0, backward)
                assert inside % 16 == 0 and 0 < inside <= copied
                # never the logits of many classes: statistics of tiles, or pieces of
                # the gradients, and sums of the products and copies of the operands
                if rows * classes * e > 2**28:
                    operands = 6 * (rows + classes) * (width + 8) + 2**23
                    sums = 64 * rows * (width + 4) * 4 if backward else 0
                    assert inside < rows * classes * e or sums + operands > rows * classes * e
    assert size(8192, 50000, 4096, 3, 1, 1, 0) < 8192 * 50000 * 2 / 30


def test_a_workspace_for_copies_is_enough_in_place(b):
    size = b.fn_linear_cross_entropy_workspace
    for rows in (0, 1, 16, 17, 300, 5000, 2**17):
        for classes in (1, 64, 1000, 2**17, 2**18):
            for width in (8, 512, 4096, 2**16):
                for dtype in (0, 1):
                    for backward in (0, 1):
                        a = (rows, classes, width, dtype)
                        both, x, w, none = (size(*a, i, j, backward) for i, j in
                                            ((1, 1), (1, 0), (0, 1), (0, 0)))
                        assert both <= min(x, w) and max(x, w) <= none


def calls(b):
    """(name, function, its float arguments)."""
    x, w, s, c = torch.ones(4, 8), torch.ones(5, 8), torch.ones(4), torch.ones(5)
    y = torch.zeros(4, dtype=torch.int64)
    return [
        ("loss", lambda **k: b.linear_cross_entropy(targets=y, **k), dict(x=x, weight=w, bias=c, losses=s, lse=s)),
        ("backward", lambda **k: b.linear_cross_entropy_backward(targets=y, **k),
         dict(dlosses=s, x=x, weight=w, lse=s, bias=c, dx=x, dweight=w, dbias=c)),
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
