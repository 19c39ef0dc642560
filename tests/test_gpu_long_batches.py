"""Batches of more images than one launch has threads for (HIP starts fewer
than 2^32): the whole batch equals its slices, bit for bit, and a test hook
refuses more than its one launch can hold."""
from __future__ import annotations

import pytest
import torch

from conftest import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


@pytest.mark.parametrize("N", [2**28 + 1003])
def test_decisions_of_a_long_batch(fn, N):
    args = (7, 9, 0.5, 0.7, 0.02, 0.33, 0.3, 3.3)
    out = torch.full((N, 8), -7, dtype=torch.int32, device="cuda")
    fn.fn_params(3, N, *args, out)
    step = 2**26 - 32
    part = torch.empty(step, 8, dtype=torch.int32, device="cuda")
    for at in range(0, N, step):
        n = min(step, N - at)
        fn.fn_params_ex(3, at, n, *args, part)
        assert torch.equal(out[at:at + n], part[:n]), at


@pytest.mark.parametrize("N,H,W,C,kind", [(2**27 + 1003, 1, 1, 1, "FP32"), (2**28 + 1003, 2, 2, 2, "FP16"),
                                          (2**28 + 77, 1, 8, 1, "FP16"), (2**28 + 77, 1, 3, 3, "FP16_PAD4")])
def test_images_of_a_long_batch(fn, N, H, W, C, kind):
    g = torch.Generator(device="cuda").manual_seed(N + H)
    images = torch.randint(0, 256, (N, H, W, C), generator=g, dtype=torch.uint8, device="cuda")
    code = getattr(fn, "FN_OUT_" + kind)
    t = torch.float32 if kind == "FP32" else torch.float16
    oc = 4 if kind == "FP16_PAD4" else C
    args = ((0.4,) * C, (0.25,) * C, 0.5, 0.5, 0.02, 0.33, 0.3, 3.3, 11)
    out = torch.full((N, H, W, oc), 7.0, dtype=t, device="cuda")
    fn.fn_fused_normalize(images, N, H, W, C, *args, code, out)
    step = 2**25
    part = torch.empty(step, H, W, oc, dtype=t, device="cuda")
    for at in range(0, N, step):
        n = min(step, N - at)
        fn.fn_fused_normalize_ex(images[at:], W * C, H * W * C, n, H, W, C, *args, at, code, part)
        assert torch.equal(out[at:at + n], part[:n]), at
    # one image read N times
    if H == W == 1:
        fn.fn_fused_normalize_ex(images, W * C, 0, N, H, W, C, *args, 0, code, out)
        fn.fn_fused_normalize_ex(images, W * C, 0, 1003, H, W, C, *args, 2**27, code, part)
        assert torch.equal(out[2**27:], part[:1003])


def test_narrow_strided_rows_of_a_long_batch(fn):
    """Tiles of 512 one-byte rows, three bytes apart: 2^23 of them and more."""
    N, H = 2**18 + 33, 16384
    image = torch.randint(0, 256, (H, 3), generator=torch.Generator().manual_seed(5),
                          dtype=torch.uint8).cuda()
    args = ((0.4,), (0.25,), 0.5, 0.9, 0.02, 0.33, 0.3, 3.3, 11)
    out = torch.full((N, H), 7.0, device="cuda")
    fn.fn_fused_normalize_ex(image, 3, 0, N, H, 1, 1, *args, 0, fn.FN_OUT_FP32, out)
    step = 2**15
    part = torch.empty(step, H, device="cuda")
    for at in range(0, N, step):
        n = min(step, N - at)
        fn.fn_fused_normalize_ex(image, 3, 0, n, H, 1, 1, *args, at, fn.FN_OUT_FP32, part)
        assert torch.equal(out[at:at + n], part[:n]), at


def test_hooks_refuse_more_than_one_launch(fn):
    for call in (lambda: fn.fn_test_erase_dims(None, None, 2**32, 8, 8, 0.02, 0.33, 0.3, 3.3, None, None, None),
                 lambda: fn.fn_test_cr_ops(0, None, None, 2**32, None),
                 lambda: fn.fn_test_stream(None, None, 2**35, 2),
                 lambda: fn.fn_test_stream(None, None, 2**36, 4)):
        with pytest.raises(fn.FnError) as e:
            call()
        assert e.value.code == -2
