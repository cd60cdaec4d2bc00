"""Norms of queries and keys at the ends of their elements' range, on the GPU against the
definition in 64 bits (fp8_util.py)."""
import pytest
import torch

import gated_deltanet_paged_gb300 as gdn
from attention_util import within
from fp8_util import norm_rope_f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,rotary", [(64, 32), (128, 128), (136, 0), (200, 72), (248, 6), (256, 0), (256, 64), (256, 34), (256, 256)])
@pytest.mark.parametrize("size", [2.0**60, 2.0**-60])
def test_elements_of_every_size(dim, rotary, size):
    """Elements up to 2^60 keep their precision: 256 squares of 2^120 are 2^128, which is
    not an fp32 number.  (And small ones beside an eps that is smaller still.)"""
    gen = torch.Generator().manual_seed(dim + rotary)
    q = torch.randn(6, 5, dim, generator=gen).clamp(-1, 1)
    q[1:4] = q[1:4].sign()  # all of the largest size
    q[2, :, 1:] *= 2.0**-8  # ... or one
    q = (q.double() * size).bfloat16().cuda()
    k = q[:, 1:4].contiguous()
    w = (1 + 0.3 * torch.randn(2, dim, generator=gen)).bfloat16().cuda()
    pos = torch.randint(0, 1 << 20, (6,), generator=gen, dtype=torch.int32)
    f = gdn.gdn_rope_frequencies(rotary) if rotary else None
    for interleaved in (False, True):
        got = gdn.gdn_qk_norm_rope(q, k, w[0], w[1], f, pos.cuda(), eps=2.0**-126, interleaved=interleaved)
        for y, src, weight in zip(got, (q, k), w):
            ref, tol = norm_rope_f64(src, weight, pos, f, eps=2.0**-126, interleaved=interleaved)
            within(y, ref, tol + 2.0**-8 * ref.abs(), "norm and rotation")
