"""The workspace of rms_norm_backward: bytes that lie together.  A view with
gaps is refused, for the bytes between would be written too."""
from __future__ import annotations

import pytest
import torch

from conftest import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


@pytest.mark.parametrize("rows,width", [(3000, 64), (3, 64), (5, 40001)])
def test_a_workspace_with_gaps_is_refused(fn, rows, width):
    h = torch.randn(rows, width, device="cuda")
    w, rstd = torch.ones(width, device="cuda"), torch.ones(rows, device="cuda")
    want = fn.rms_norm_backward(h, h, w, rstd)
    size = fn.rms_norm_backward_workspace(rows, width).numel()
    big = torch.full((max(size, 64), 4), 9, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        fn.rms_norm_backward(h, h, w, rstd, workspace=big[:, :2])
    assert (big == 9).all()
    got = fn.rms_norm_backward(h, h, w, rstd, workspace=big.view(-1)[: max(size, 64)])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (big.view(-1)[max(size, 64):] == 9).all()
