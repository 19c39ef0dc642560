"""The helpers of the 8-bit linear layer differentiate nothing: an argument
whose gradient or tangent would be lost is refused, on the CPU, before any
device is looked for; without gradients the same arguments pass this check."""
from __future__ import annotations

import pytest
import torch
from torch.autograd import forward_ad

from conftest import ROOT  # noqa: F401


@pytest.fixture(scope="module")
def b():
    from augmentation_amd import binding
    return binding


def calls(b):
    """(name, function, the float arguments it takes, the others)."""
    x, w, s = torch.ones(4, 8), torch.ones(8), torch.ones(4)
    codes = torch.ones(4, 8, dtype=torch.int8)
    return [
        ("rms_norm", lambda **k: b.rms_norm(**k),
         dict(x=x, weight=w, residual=x, sum_out=x, out=x, rstd=s), {}),
        ("rms_norm_q8", lambda **k: b.rms_norm_q8(**k),
         dict(x=x, weight=w, residual=x, sum_out=x, scales=s, rstd=s), dict(codes=codes)),
        ("quantize_rows", lambda **k: b.quantize_rows(**k), dict(x=x, scales=s), dict(codes=codes)),
        ("rms_norm_backward", lambda **k: b.rms_norm_backward(**k),
         dict(dout=x, h=x, weight=w, rstd=s, dsum=x, dx=x, dweight=w), {}),
        ("matmul_q8", lambda **k: b.matmul_q8(**k),
         dict(a_scales=s, b_scales=s, bias=s, out=torch.ones(4, 4)), dict(a=codes, b=codes)),
    ]


CASES = [(name, arg) for name, _, args, _ in calls(None) for arg in args]


@pytest.mark.parametrize("name,arg", CASES)
def test_an_argument_that_requires_a_gradient_is_refused(b, name, arg):
    _, call, args, others = next(c for c in calls(b) if c[0] == name)
    args = dict(args, **others, **{arg: args[arg].clone().requires_grad_()})
    with pytest.raises(ValueError, match="requires a gradient"):
        call(**args)
    # host tensors are refused for what they are once nothing is recorded
    with torch.no_grad(), pytest.raises(ValueError) as e:
        call(**args)
    assert "gradient" not in str(e.value) and "CUDA" in str(e.value)
    args[arg] = args[arg].detach()
    with pytest.raises(ValueError, match="CUDA"):
        call(**args)


@pytest.mark.parametrize("name,arg", CASES)
def test_an_argument_with_a_tangent_is_refused(b, name, arg):
    _, call, args, others = next(c for c in calls(b) if c[0] == name)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(args[arg], torch.ones_like(args[arg]))
        with pytest.raises(ValueError, match="tangent"):
            call(**dict(args, **others, **{arg: dual}))
        with pytest.raises(ValueError, match="CUDA"):
            call(**args, **others)


def test_within_an_autograd_function_nothing_is_refused(b):
    """The way to train through the helpers: torch records nothing there."""
    seen = []

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            with pytest.raises(ValueError, match="CUDA"):
                b.rms_norm(x, w)
            seen.append(True)
            return x * w

    x, w = torch.ones(4, 8, requires_grad=True), torch.ones(8, requires_grad=True)
    Norm.apply(x, w)
    assert seen
