"""Tensors that the helpers allocate for work on another stream belong to that
stream: none lies in memory that the current stream has still to write."""
from __future__ import annotations

import pytest
import torch

from conftest import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


def helpers(fn):
    """name -> a call that allocates everything it returns."""
    g = torch.Generator().manual_seed(1)
    t = torch.bfloat16
    x, r, d = (torch.randn(3000, 1000, generator=g).to(t).cuda() for _ in range(3))
    w = torch.randn(1000, generator=g).to(t).cuda()
    out, rstd, h = fn.rms_norm(x, w, residual=r)
    codes, scales = fn.quantize_rows(x)
    b, b_scales = fn.quantize_rows(r[:700])
    images = torch.randint(0, 256, (8, 100, 120, 3), generator=g, dtype=torch.uint8).cuda()
    return {
        "rms_norm": lambda s: fn.rms_norm(x, w, residual=r, stream=s),
        "rms_norm_q8": lambda s: fn.rms_norm_q8(x, w, residual=r, stream=s),
        "quantize_rows": lambda s: fn.quantize_rows(x, stream=s),
        "rms_norm_backward": lambda s: fn.rms_norm_backward(d, h, w, rstd, stream=s),
        "matmul_q8": lambda s: (fn.matmul_q8(codes, scales, b, b_scales, stream=s),),
        "fused_normalize": lambda s: (fn.fused_normalize(images, (0.5,) * 3, (0.2,) * 3, 0.5, 0.5,
                                                         stream=s),),
        "sample_params": lambda s: (fn.sample_params(5000, 32, 32, 0.5, 0.5, stream=s),),
    }


NAMES = ["rms_norm", "rms_norm_q8", "quantize_rows", "rms_norm_backward", "matmul_q8",
         "fused_normalize", "sample_params"]


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_no_memory_that_the_current_stream_still_writes(fn, name, handle):
    call = helpers(fn)[name]
    want = [v.clone() for v in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the results' sizes (and the workspace's), freed with their last
    # use still to come on the current stream
    torch.cuda._sleep(20_000_000)
    stale = [torch.empty_like(v) for v in want] + [torch.empty(1 << 20, dtype=torch.uint8, device="cuda")]
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


def test_the_null_stream_from_another_one(fn):
    x = torch.randn(300, 500, device="cuda")
    want = [v.clone() for v in fn.quantize_rows(x)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = fn.quantize_rows(x, stream=0)
        assert torch.cuda.current_stream() == side
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_streams_and_two_threads_at_once(fn):
    """Every helper from two host threads, each on a stream of its own, over and
    over: the results of one stream alone."""
    import threading

    calls = helpers(fn)
    want = {k: [v.clone() for v in f(None)] for k, f in calls.items()}
    torch.cuda.synchronize()
    wrong = []

    def work(names):
        s = torch.cuda.Stream()
        for _ in range(20):
            kept = [(k, calls[k](s)) for k in names]
            s.synchronize()
            wrong.extend(k for k, got in kept for a, b in zip(got, want[k]) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(n,)) for n in (NAMES, NAMES[::-1])]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong
