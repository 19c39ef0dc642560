"""Training through the norm's helpers inside a torch.autograd.Function, and
their refusal of arguments whose gradients would be lost, on device tensors.

Tolerance of the gradients in fp32: each is a sum of a few products of numbers
of size up to `size`; the row's sums are chains of under 100 additions, so
128 u (u = 2^-24) of the largest magnitude in play covers them."""
from __future__ import annotations

import pytest
import torch

from conftest import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


def norm_function(fn):
    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, weight):
            out, rstd, h = fn.rms_norm(x, weight, EPS, residual=residual)
            ctx.save_for_backward(h, weight, rstd)
            return out, h

        @staticmethod
        def backward(ctx, dout, dsum):
            h, weight, rstd = ctx.saved_tensors
            dx, dweight = fn.rms_norm_backward(dout, h, weight, rstd, dsum=dsum)
            return dx, dx, dweight.to(weight.dtype)

    return Norm.apply


def test_a_layer_trains_through_a_function(fn):
    g = torch.Generator().manual_seed(1)
    x, r, w, m = (torch.randn(*s, generator=g).cuda() for s in ((9, 200), (9, 200), (200,), (200,)))
    leaves = [v.clone().requires_grad_() for v in (x, r, w)]
    out, h = norm_function(fn)(*leaves)
    (out * m).sum().add((h * h).sum()).backward()
    ref = [v.double().requires_grad_() for v in (x, r, w)]
    hd = ref[0] + ref[1]
    yd = hd / torch.sqrt(hd.square().mean(1, keepdim=True) + EPS) * ref[2]
    (yd * m.double()).sum().add((hd * hd).sum()).backward()
    for got, want in zip(leaves, ref):
        size = want.grad.abs().max() + (x.abs() * m.abs()).max()
        assert (got.grad.double() - want.grad).abs().max() <= 128 * U * size


def test_lost_gradients_are_refused_on_the_device(fn):
    x = torch.ones(4, 64, device="cuda")
    w = torch.ones(64, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="requires a gradient"):
        fn.rms_norm(x, w)
    codes, scales = fn.quantize_rows(x)
    with pytest.raises(ValueError, match="requires a gradient"):
        fn.matmul_q8(codes, scales, codes, scales, bias=torch.zeros(4, device="cuda", requires_grad=True))
    with torch.no_grad():
        out, _, _ = fn.rms_norm(x, w)
    assert not out.requires_grad and torch.equal(out, fn.rms_norm(x, w.detach())[0])


def test_written_tensors_count_a_version(fn):
    """Every tensor that a call writes, and no other: a backward pass that saved
    one of them before raises rather than use what has taken its place."""
    def made(*shape, t=torch.float32):
        return torch.ones(*shape, dtype=t, device="cuda")

    x, r, w, out, h, dsum = (made(700, 64) if k != 2 else made(64) for k in range(6))
    rstd, scales, codes, dw = made(700), made(700), made(700, 64, t=torch.int8), made(64)
    ws = fn.rms_norm_backward_workspace(700, 64)
    product = made(700, 700)
    everything = [x, r, w, out, h, dsum, rstd, scales, codes, dw, ws, product]

    def writes(call, *written):
        before = [v._version for v in everything]
        call()
        for v, old in zip(everything, before):
            assert v._version == old + any(v is o for o in written)

    writes(lambda: fn.rms_norm(x, w, residual=r, sum_out=h, out=out, rstd=rstd), h, out, rstd)
    writes(lambda: fn.rms_norm(x, w, residual=r, sum_out=r, out=x), r, x)
    writes(lambda: fn.rms_norm(x, w, out=x), x)
    writes(lambda: fn.rms_norm(x, w))
    writes(lambda: fn.rms_norm_q8(x, w, residual=r, sum_out=h, codes=codes, scales=scales, rstd=rstd),
           h, codes, scales, rstd)
    writes(lambda: fn.quantize_rows(x, codes=codes, scales=scales), codes, scales)
    writes(lambda: fn.rms_norm_backward(out, h, w, rstd, dsum=dsum, dx=dsum, dweight=dw, workspace=ws),
           dsum, dw, ws)
    writes(lambda: fn.matmul_q8(codes, scales, codes, scales, out=product), product)
    with torch.inference_mode():
        assert fn.quantize_rows(made(3, 8))[0].shape == (3, 8)

    leaf = made(700, 64).requires_grad_()
    y = leaf * h  # saves h
    with torch.no_grad():
        fn.rms_norm(x, w, residual=h, sum_out=h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
