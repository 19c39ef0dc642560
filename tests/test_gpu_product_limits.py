"""Products of more channels or tokens than one launch has threads for (HIP
starts fewer than 2^32): every route of few tokens or few channels, checked
bit for bit on the device with the documented fp32 steps."""
from __future__ import annotations

import pytest
import torch

from conftest import ROOT  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fn():
    from augmentation_amd import binding
    return binding


# tokens, channels, codes: work-groups of 512 threads for 16 channels, for 64
# channels, for tiles of 64x64 and, with many tokens, of 128x64
@pytest.mark.parametrize("m,n,k", [(1, 2**27 + 1021, 15), (2, 2**29 + 1021, 16), (17, 2**29 + 77, 1),
                                   (2**30 + 77, 3, 1)])
def test_more_than_one_launch(fn, m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m + n)
    a = torch.randint(-128, 128, (m, k), generator=g, dtype=torch.int8, device="cuda")
    b = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8, device="cuda")
    sa = torch.rand(m, generator=g, device="cuda")
    sb = torch.rand(n, generator=g, device="cuda")
    out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
    fn.matmul_q8(a, sa, b, sb, out=out)
    step = 1 << 22
    for m0 in range(0, m, step):
        for n0 in range(0, n, step):
            am, bn = a[m0:m0 + step].float(), b[n0:n0 + step].float()
            # sums of at most 16 products of codes: exact in fp32
            y = (am[:, None, :] * bn[None, :, :]).sum(2)
            y = y * sa[m0:m0 + step, None] * sb[None, n0:n0 + step]
            assert torch.equal(out[m0:m0 + step, n0:n0 + step], y.bfloat16()), (m0, n0)
