"""Attention at the ends of its options' ranges, on the GPU against the definition
in 64 bits: soft caps from far below the scores to far above them, and what
unread slots may change (nothing).  Tolerances as derived in attention_util.py."""
import pytest
import torch

import gated_deltanet_paged_gb300 as gdn
from attention_util import Batch, check_attention, within

pytestmark = pytest.mark.gpu

I16 = torch.int16


def _batch(decode, dim, q_scale, seed=41):
    new, prefix = ([1] * 4, [700, 0, 63, 2000]) if decode else ([140, 3, 0, 64], [700, 0, 63, 300])
    return Batch(new, prefix, 64, 8, 2, dim, seed=seed, q_scale=q_scale).fill()


# The capped score tends to the score itself as the cap grows: a form with an error
# that is a fixed part of the cap loses every score under a large one.
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("cap", [5e-5, 0.01, 1.0, 50.0, 60.0, 884.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e30, 3e38])
def test_caps_of_every_size(decode, cap):
    for dim, q_scale in ((128, 1.0), (64, 40.0)):
        check_attention(_batch(decode, dim, q_scale), decode=decode, softcap=cap)


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("cap", [2.0, 900.0, 1e6, 1e30])
def test_caps_with_a_bias(decode, cap):
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(8)], device="cuda")
    check_attention(_batch(decode, 128, 20.0), decode=decode, softcap=cap, slopes=slopes)


@pytest.mark.parametrize("decode", [False, True])
def test_slots_past_the_end_change_no_bit_under_a_cap(decode):
    """The last page's slots past the sequence's end are copied along with the
    tokens: their scores may be anything, and decide nothing."""
    first = None
    for junk in (0.0, float("nan"), 3.0, 1e30, float("inf")):
        b = _batch(decode, 128, 2.0)
        b.k_cache.fill_(junk)
        b.v_cache.fill_(junk)
        o, lse = check_attention(b.fill(), decode=decode, softcap=30.0)
        if first is None:
            first = o.clone(), lse.clone()
        assert torch.equal(o.view(I16), first[0].view(I16)) and torch.equal(lse, first[1]), "slots hold %r" % junk


# Scores at either end of the cap, and values near either end of bf16's range: the
# weights have to be taken relative to the row's largest score, as without a cap
# (weights of 2^80, or 2^-80, times such values leave fp32).
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("cap", [5.0, 30.0, 55.0, 70.0])
@pytest.mark.parametrize("size", [2.0**-100, 2.0**100])
@pytest.mark.parametrize("sign", [-1.0, 0.0, 1.0])
@pytest.mark.parametrize("window", [-1, 130])
def test_values_of_every_size_under_a_cap(decode, cap, size, sign, window):
    """sign: where all scores lie, far beyond the cap; 0: on both sides."""
    new, prefix = ([1] * 3, [700, 5, 2000]) if decode else ([300, 3, 64], [700, 0, 1300])
    b = Batch(new, prefix, 64, 8, 2, 64, seed=43, q_scale=100.0)
    if sign:
        b.q[:] = b.q.abs()
        b.k = [sign * k.abs() for k in b.k]
    b.v = [(v.float() * size).bfloat16() for v in b.v]
    check_attention(b.fill(), decode=decode, softcap=cap, window=window)


@pytest.mark.parametrize("slope", [0.25, 0.125, 0.3])
def test_bias_that_grows_with_the_distance(slope):
    """Negative slopes far from the token: the largest weights belong to the first
    keys, whose bias is 10^5 times the difference between neighbours.  What the 128
    keys of a block have in common is rounded once for all of them, and the rest at
    the size of slope * 128, so that the tolerance is that of small scores (zero keys
    make every score the bias alone; the values tell neighbours apart)."""
    p, n, ps, dim = 1500000, 3, 1024, 64
    pages = -(-(p + n) // ps)
    k = torch.zeros(pages, ps, 1, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    sign = torch.tensor([1.0 if j % 32 < 4 else -1.0 for j in range(ps)])
    v[0] = sign.bfloat16().cuda()[:, None, None]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    slopes = torch.tensor([-slope, -slope / 2], device="cuda")
    q = torch.randn(n, 2, dim, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    o, lse = gdn.gdn_attention_paged(q, k, v, i32(0, n), torch.arange(pages, dtype=torch.int32, device="cuda"),
                                     i32(0, pages), i32(p + n - (pages - 1) * ps), slopes=slopes, return_lse=True)
    j = torch.arange(ps, dtype=torch.float64)  # keys beyond have weights below e^-60
    for h in range(2):
        x = -slopes[h].double().cpu() * (torch.arange(p, p + n, dtype=torch.float64)[:, None] - j)
        want_lse = torch.logsumexp(x, -1)
        want = (torch.exp(x - want_lse[:, None]) @ sign.double())[:, None].expand(n, dim)
        within(lse[:, h], want_lse, 2.0**-19 * (16 + want_lse.abs()), "lse")
        within(o[:, h], want, 2.0**-8 * (want.abs() + 1) + 2.0**-14, "o")
