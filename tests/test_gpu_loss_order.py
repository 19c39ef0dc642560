"""What fixes the bits of the linear cross entropy: the sizes, the type, whether the
weight is read in place, and whether dx and dweight are both wanted.  Not the place
of x, not where a copied weight lies, not the call."""
from __future__ import annotations

import pytest
import torch

from test_gpu_cross_entropy import check_backward, check_forward, head

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


def placed(m, left, right):
    """m as columns of a wider buffer."""
    wide = torch.zeros(m.size(0), left + m.size(1) + right, dtype=m.dtype, device="cuda")
    wide[:, left:left + m.size(1)] = m
    return wide[:, left:left + m.size(1)]


# weights of more than a piece's 128 MiB, which a copy of them is made in parts of; and
# small ones
SIZES = [(100, 20000, 4096, torch.bfloat16), (300, 40000, 2048, torch.float16), (20, 70000, 512, torch.float32),
         (40, 500, 64, torch.bfloat16), (600, 3000, 328, torch.float32)]


@pytest.mark.parametrize("rows,classes,width,t", SIZES)
def test_only_the_place_of_the_weight_counts(fn, rows, classes, width, t):
    x, w, y, b = head(rows, rows, classes, width, t)
    d = torch.rand(rows, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") + 0.5
    e = 16 // t.itemsize

    def both(x, w):
        losses, lse = fn.linear_cross_entropy(x, w, y, bias=b, smoothing=0.1)
        return [losses, lse, *fn.linear_cross_entropy_backward(d, x, w, y, lse, bias=b, smoothing=0.1)]

    for w_, others in ((w, [placed(w, e, 2 * e)]), (placed(w, 1, 0), [placed(w, 3, 2), placed(w, e, 1)])):
        want = both(x, w_)
        for x2 in (x, placed(x, e, e), placed(x, 1, 0), placed(x, 3, 2)):
            for w2 in (w_, *others):
                assert all(torch.equal(p, q) for p, q in zip(both(x2, w2), want))
        _, lse = check_forward(fn, x, w_, y, b, 0.1)
        check_backward(fn, x, w_, y, b, 0.1, d, lse)


@pytest.mark.parametrize("rows,classes,width,t", SIZES)
def test_a_gradient_on_its_own_is_the_same_every_time(fn, rows, classes, width, t):
    x, w, y, b = head(rows, rows, classes, width, t)
    d = torch.full((rows,), 1 / rows, device="cuda")
    _, lse = fn.linear_cross_entropy(x, w, y, bias=b)
    for kw in (dict(want_dweight=False), dict(want_dx=False), dict()):
        want = check_backward(fn, x, w, y, b, 0.0, d, lse, **kw)
        for x2 in (x, placed(x, 1, 0)):
            got = fn.linear_cross_entropy_backward(d, x2, w, y, lse, bias=b, **kw)
            assert all(p is q or torch.equal(p, q) for p, q in zip(got, want))
