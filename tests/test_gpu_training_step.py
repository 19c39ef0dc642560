"""Dropout, layer norm and the linear cross entropy together, as a training step
uses them, and what the helpers have in common: streams, threads, versions.

Tolerance of the step's gradients in fp16: a gradient passes three roundings to
fp16 on its way (the head's dx, the mean's, the norm's), each at most 2^-11 of a
value, and the features' own roundings change p by as much: 2^-8 of the
gradient's norm covers their sum."""
from __future__ import annotations

import sys

import pytest
import torch

from conftest import ROOT
from test_gpu_layer_norm import kept, share

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, ROOT)
    from examples import train_head
    return train_head


@pytest.mark.parametrize("images,width,classes", [(3, 128, 10), (16, 384, 1000)])
def test_the_example_runs_and_its_gradients_are_those_of_64_bits(example, images, width, classes):
    losses, head, features, labels = example.run(images, width, 1, classes, 2)
    assert all(torch.isfinite(x) for x in losses)
    tokens = features.size(1)
    loss = head.loss(features, labels, seed=7)
    (loss * example.LOSS_SCALE).backward()
    position, nw, nb, w, b = (p.detach().double().requires_grad_() for p in head.parameters())
    keep = kept(7, 0, images * tokens, width, example.DROPOUT).view(images, tokens, width)
    x = torch.where(keep, features.double() * (65536 / (65536 - share(example.DROPOUT))), 0.0)
    h = x + position
    d = h - h.mean(-1, keepdim=True)
    n = d / torch.sqrt(d.square().mean(-1, keepdim=True) + example.EPS) * nw + nb
    ref = torch.nn.functional.cross_entropy(n.mean(1) @ w.t() + b, labels, label_smoothing=example.SMOOTHING)
    assert abs(loss.item() - ref.item()) <= 2.0 ** -8 * ref.item()
    (ref * example.LOSS_SCALE).backward()
    for got, want in zip(head.parameters(), (position, nw, nb, w, b)):
        off = (got.grad.double() - want.grad).norm()
        assert off <= 2.0 ** -8 * want.grad.norm() + 2.0 ** -24 * want.grad.numel() ** 0.5, got.shape


def helpers(fn):
    """name -> a call that allocates everything it returns."""
    g = torch.Generator().manual_seed(1)
    t = torch.bfloat16
    x, r, d = (torch.randn(3000, 1000, generator=g).to(t).cuda() for _ in range(3))
    w, b = (torch.randn(1000, generator=g).to(t).cuda() for _ in range(2))
    out, mean, rstd, h = fn.layer_norm(x, w, b, residual=r, p=0.1, seed=3)
    weight = (torch.randn(700, 1000, generator=g) / 30).to(t).cuda()
    y = torch.randint(0, 700, (3000,), generator=g).cuda()
    bias = torch.randn(700, generator=g).cuda()
    losses, lse = fn.linear_cross_entropy(x, weight, y, bias=bias)
    return {
        "dropout": lambda s: (fn.dropout(x, 0.1, 3, residual=r, stream=s),),
        "layer_norm": lambda s: fn.layer_norm(x, w, b, residual=r, p=0.1, seed=3, stream=s),
        "layer_norm_backward": lambda s: fn.layer_norm_backward(d, h, w, mean, rstd, p=0.1, seed=3, stream=s),
        "linear_cross_entropy": lambda s: fn.linear_cross_entropy(x, weight, y, bias=bias, stream=s),
        "linear_cross_entropy_backward": lambda s: fn.linear_cross_entropy_backward(lse, x, weight, y, lse, bias=bias, stream=s),
    }


NAMES = ["dropout", "layer_norm", "layer_norm_backward", "linear_cross_entropy", "linear_cross_entropy_backward"]


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_no_memory_that_the_current_stream_still_writes(fn, name, handle):
    call = helpers(fn)[name]
    want = [v.clone() for v in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the results' sizes (and the workspaces'), freed with their last
    # use still to come on the current stream
    torch.cuda._sleep(20_000_000)
    stale = [torch.empty_like(v) for v in want] + [torch.empty(1 << k, dtype=torch.uint8, device="cuda") for k in (20, 23, 25)]
    at = {v.data_ptr() for v in stale}
    for v in stale:
        v.fill_(77)
    del stale, v
    got = call(side.cuda_stream if handle else side)
    assert not at & {v.data_ptr() for v in got}
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_streams_and_two_threads_at_once(fn):
    import threading

    calls = helpers(fn)
    want = {k: [v.clone() for v in f(None)] for k, f in calls.items()}
    torch.cuda.synchronize()
    wrong = []

    def work(names):
        s = torch.cuda.Stream()
        for _ in range(20):
            got = [(k, calls[k](s)) for k in names]
            s.synchronize()
            wrong.extend(k for k, vs in got for a, b in zip(vs, want[k]) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(n,)) for n in (NAMES, NAMES[::-1])]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


def test_written_tensors_count_a_version(fn):
    def made(*shape, t=torch.float32):
        return torch.ones(*shape, dtype=t, device="cuda")

    x, r, out, s, dh, dx, dsum = (made(60, 64) for _ in range(7))
    w, b, dw, db = (made(64) for _ in range(4))
    mean, rstd, losses, lse = (made(60) for _ in range(4))
    weight, dweight, bias, dbias = made(9, 64), made(9, 64), made(9), made(9)
    y = torch.zeros(60, dtype=torch.int64, device="cuda")
    ws, lws = fn.layer_norm_backward_workspace(60, 64), fn.linear_cross_entropy_workspace(x, weight, True)
    everything = [x, r, out, s, dh, dx, dsum, w, b, dw, db, mean, rstd, losses, lse, weight, dweight, bias, dbias, y, ws, lws]

    def writes(call, *written):
        before = [v._version for v in everything]
        call()
        for v, old in zip(everything, before):
            assert v._version == old + any(v is o for o in written)

    writes(lambda: fn.dropout(x, 0.1, 1, residual=r, out=out), out)
    writes(lambda: fn.dropout(x, 0.1, 1))
    writes(lambda: fn.layer_norm(x, w, b, residual=r, p=0.1, out=out, sum_out=s, mean=mean, rstd=rstd), out, s, mean, rstd)
    writes(lambda: fn.layer_norm(x, out=out), out)
    writes(lambda: fn.layer_norm_backward(out, s, w, mean, rstd, dsum=dsum, p=0.1, dh=dh, dx=dx, dweight=dw, dbias=db, workspace=ws),
           dh, dx, dw, db, ws)
    writes(lambda: fn.layer_norm_backward(out, s, w, mean, rstd, dh=dh), dh)
    writes(lambda: fn.linear_cross_entropy(x, weight, y, bias=bias, losses=losses, lse=lse, workspace=lws), losses, lse, lws)
    writes(lambda: fn.linear_cross_entropy_backward(losses, x, weight, y, lse, bias=bias, dx=dx, dweight=dweight, dbias=dbias, workspace=lws),
           dx, dweight, dbias, lws)
    writes(lambda: fn.linear_cross_entropy_backward(losses, x, weight, y, lse, dx=dx, want_dweight=False), dx)
