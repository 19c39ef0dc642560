"""Layer norm's gradients of many rows and of wide ones, whole: the rows' own and
the sums over the rows, with dropout and without, on both sides of the columns that
one launch of the sums takes (2^26)."""
from __future__ import annotations

import pytest
import torch

from test_gpu_layer_norm import EPS, SEED, U, backward_reference, check_close, depth, dropped, half, share, tiny

pytestmark = pytest.mark.gpu

T = torch.float16


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("rows,width", [(1_300_000, 12), (70_000, 40), (70_000, 770), (9_000, 5003), (3, 2**20 + 3), (130, 40001), (2, 2**26 + 5)])
def test_gradients_of_many_rows_and_of_wide_ones(fn, rows, width, p):
    g = torch.Generator(device="cuda").manual_seed(width)
    h, dout, dsum = (torch.randn(rows, width, generator=g, device="cuda").to(T) for _ in range(3))
    w = (torch.rand(width, generator=g, device="cuda") + 0.5).to(T)
    _, mean, rstd, _ = fn.layer_norm(h, w, None, EPS)
    dh, dx, dw, db = fn.layer_norm_backward(dout, h, w, mean, rstd, dsum=dsum, p=p, seed=SEED, first_row=3)
    # sums over the rows, a range of columns at a time: a term is off by 4 u, a chain of
    # additions is no longer than a slice of the rows and the partial rows
    for first in range(0, width, 2**24):
        part = slice(first, min(first + 2**24, width))
        d = dout[:, part].double()
        n = (h[:, part].double() - mean.double()[:, None]) * rstd.double()[:, None]
        chain = rows / 64 + 600
        check_close(dw[part], (d * n).sum(0), (chain + 4) * U * (d * n).abs().sum(0) + 1e-30, "dweight")
        check_close(db[part], d.sum(0), chain * U * d.abs().sum(0) + 1e-30, "dbias")
        del d, n
    at = sorted({0, 1, rows // 2, rows - 1})
    if rows > 1000:
        at = sorted({*at, 511, 512, rows // 3, rows - 2})
    D = depth(width)
    for k in at:
        row = slice(k, k + 1)
        ref, _, _, n, gg = backward_reference(dout[row], h[row], w, mean[row], rstd[row], dsum[row])
        gm, gnm, m = gg.abs().mean(), (gg * n).abs().mean(), (gg * n).mean().abs()
        off = rstd[k].double() * (4 * U * gg.abs() + (D + 4) * U * gm + (D + 6) * U * gnm * n.abs() + 5 * U * n.abs() * m)
        off = off + U * (ref.abs() + dsum[row].double().abs())
        check_close(dh[row], ref, off * (1 + half(T)) + ref.abs() * half(T) + tiny(T), "dh")
        if p > 0:
            scale = 65536 / (65536 - share(p))
            want = dropped(ref, p, 3 + k)
            check_close(dx[row], want, scale * off * (1 + half(T)) + want.abs() * (half(T) + 2 * U) + tiny(T), "dx")
        else:
            assert dx is dh
