"""Capped attention over the 8-bit cache at the ends of its range, on the GPU against the
definition in 64 bits: scores far beyond either end of the cap, rows that see a single
key, values near either end of what the format holds, and what unread slots may change
(nothing).  Tolerances as derived in attention_util.py."""
import pytest
import torch

import gated_deltanet_paged_gb300 as gdn
from attention_util import Batch, check_attention, within
from fp8_util import E4M3, GROUP, U8, Batch8, check_attention8

pytestmark = pytest.mark.gpu

I16 = torch.int16
CAPS = [5.0, 30.0, 55.0, 70.0, 100.0, 1e3, 1e4]


def put(b, name, of, exponent=0):
    """Codes of one kind replaced by of(codes, sequence), their scales times 2^exponent."""
    for i, (c, e) in enumerate(b.codes[name]):
        c, e = of(c.float(), i).to(E4M3), e + exponent
        b.codes[name][i] = c, e
        getattr(b, name)[i] = c.double() * torch.exp2(e.double()).repeat_interleave(GROUP, 0)[: len(c), :, None]


def workspace_sizes(b):
    """(without room for a bf16 copy of what the batch sees, with it)"""
    sizes = (len(b.new), sum(b.new), b.hq, b.hkv, b.dim, b.indices.numel(), b.ps)
    return gdn.gdn_attention_workspace_bytes(*sizes), gdn.gdn_attention_fp8_workspace_bytes(*sizes)


def check_both_ways(b, **opts):
    """By way of a bf16 copy, as such a batch goes by itself, and converted in the kernel."""
    small, large = workspace_sizes(b)
    assert large > small
    check_attention8(b, **opts)
    check_attention8(b, workspace=torch.empty(max(small, 1), dtype=U8, device="cuda")[:small], **opts)


# Every score of a row may lie at the lower end: the weights have to be taken relative to
# the row's largest score, wherever that is (2^(x - 16) is zero for x below -142, and times
# values of 2^-100 long before).
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("sign", [-1.0, 0.0, 1.0])
@pytest.mark.parametrize("window", [-1, 0, 1, 130])
def test_values_of_every_size_under_a_cap(decode, cap, sign, window):
    """sign: where all scores lie, far beyond a small cap; 0: on both sides."""
    new, prefix, hq, hkv = ([1] * 4, [700, 0, 5, 2000], 8, 2) if decode else ([300, 3, 64], [700, 0, 1300], 32, 1)
    for exponent in (-100, 100):
        b = Batch8(new, prefix, 64, hq, hkv, 64, seed=43, q_scale=100.0)
        if sign:
            b.q[:] = b.q.abs()
            put(b, "k", lambda c, i: sign * c.abs())
        put(b, "v", lambda c, i: c, exponent)
        b.fill()
        if decode:
            check_attention8(b, decode=True, softcap=cap, window=window)
        else:
            check_both_ways(b, softcap=cap, window=window)


def swing(n, turns):
    """n numbers between -400, where they begin (turns < 0: at 400), and 400: |turns| times there or back."""
    return -400 * torch.cos(torch.linspace(0, torch.pi * turns, n) - (0 if turns > 0 else torch.pi))


@pytest.mark.parametrize("cap", [30.0, 100.0, 1e3])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("turns", [1, -1, 4, -9])
def test_scores_from_end_to_end_of_a_cap(cap, dim, decode, turns):
    """Scores that rise (or fall, or swing) along the keys from one end of the cap to the
    other: a row's largest one is met first, last, or again and again a little higher."""
    new, prefix, hq, hkv = ([1] * 4, [700, 0, 5, 2000], 8, 2) if decode else ([300, 3, 64], [700, 0, 1300], 32, 1)
    b = Batch8(new, prefix, 64, hq, hkv, dim, seed=44, q_scale=30.0, spread=1)
    b.q[:] = b.q.abs()
    put(b, "k", lambda c, i: swing(len(c), turns)[:, None, None].expand_as(c))
    b.fill()
    if decode:
        check_attention8(b, decode=True, softcap=cap)
    else:
        check_both_ways(b, softcap=cap)


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("cap", CAPS[4:])
@pytest.mark.parametrize("size", [2.0**-100, 2.0**100])
@pytest.mark.parametrize("sign", [-1.0, 0.0, 1.0])
@pytest.mark.parametrize("window", [-1, 0, 130])
def test_values_of_every_size_under_a_large_cap_16_bits(decode, cap, size, sign, window):
    """The same over the 16-bit cache, under caps that leave larger scores."""
    new, prefix = ([1] * 4, [700, 0, 5, 2000]) if decode else ([300, 3, 64], [700, 0, 1300])
    b = Batch(new, prefix, 64, 8, 2, 64, seed=43, q_scale=100.0)
    if sign:
        b.q[:] = b.q.abs()
        b.k = [sign * k.abs() for k in b.k]
    b.v = [(v.float() * size).bfloat16() for v in b.v]
    check_attention(b.fill(), decode=decode, softcap=cap, window=window)


# A block of keys holds slots that no row sees; their scores are computed along.  Some of
# the scores that are seen lie beyond the cap's polynomial, so that the others near them
# are evaluated again.
@pytest.mark.parametrize("cap", [30.0, 100.0])
@pytest.mark.parametrize("window", [1, 20, 130])
@pytest.mark.parametrize("dim", [64, 128])
def test_unread_slots_change_no_bit_under_a_cap(cap, window, dim):
    b = Batch8([300, 3, 64], [700, 0, 1300], 64, 32, 1, dim, seed=43, q_scale=cap).fill()
    want = check_attention8(b, softcap=cap, window=window)
    small, large = workspace_sizes(b)
    assert large > small

    def same(size, byte):
        ws = torch.full((max(size, 1),), byte, dtype=U8, device="cuda")[:size]
        got = gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table, softcap=cap, window=window, return_lse=True,
                                          workspace=ws)
        for x, y in zip(got, want):
            assert torch.equal(x.view(I16), y.view(I16)), (size, byte)

    for byte in (0x00, 0x45, 0xC6, 0xFF):  # as bf16 zeros, +-thousands, NaN
        same(large, byte)
        same(small, byte)
    # Tokens before every window, codes and scales.
    gen = torch.Generator().manual_seed(5)
    for seq, p in enumerate(b.prefix):
        page, slot = b.slots(seq, range(max(p - window, 0)))
        for cache in (b.k_cache, b.v_cache):
            cache[page, slot] = torch.randint(0, 256, (len(page), 1, dim), generator=gen).to(U8).cuda()
        for scales in (b.k_scales, b.v_scales):
            whole = len(page) // 16 * 16
            scales[page[:whole:16], slot[:whole:16] // 16] = 246
    same(large, 0xFF)
    same(small, 0xFF)


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("power", [0, 7, 14])
@pytest.mark.parametrize("dim,hq,hkv", [(64, 4, 2), (128, 1, 1), (128, 40, 4), (64, 34, 2)])
def test_scores_up_to_the_largest(decode, power, dim, hq, hkv):
    """Keys and queries of one element, so that scores (up to 0.9 * 2^23) are exact: the key with
    the largest one takes the whole softmax, and the output is its value, whatever the scales,
    within two roundings of 2^-8: the output's, and the weight's, which is 2 to the power of
    the score less the reference, and that is rounded to half a unit of a number of up to
    2^24 (2^-1), so that the weight lies between 2^-0.5 and 2^0.5 and is no power of two."""
    new, prefix = ([1] * 4, [700, 0, 5, 2000]) if decode else ([70, 3, 20], [700, 0, 1300])
    b = Batch8(new, prefix, 64, hq, hkv, dim, seed=45, spread=20)
    b.q[:] = 0
    b.q[:, :, 0] = 2.0**power
    largest = []

    def keys(c, i):  # codes of 0.4 to 56 and one of 448
        z = torch.zeros_like(c)
        z[:, :, 0] = torch.exp2(torch.randint(-2, 6, z.shape[:2], generator=torch.Generator().manual_seed(i)).float()) * 1.75
        largest.append(prefix[i] // 3)
        z[largest[-1], :, 0] = 448
        return z

    for i, (c, e) in enumerate(b.codes["k"]):
        b.codes["k"][i] = c, torch.zeros_like(e)
    put(b, "k", keys)
    b.fill()
    call = gdn.gdn_attention_decode_paged_fp8 if decode else gdn.gdn_attention_paged_fp8
    o = call(b.q, *b.cache, *([] if decode else [b.cu]), *b.table, scale=1.0)
    want = torch.cat([b.v[i][p].expand(n, hkv, dim).repeat_interleave(hq // hkv, 1) for i, (p, n) in enumerate(zip(largest, new))])
    within(o, want, 2.0**-7 * want.abs(), "o")


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("hq,hkv,dim", [(8, 2, 128), (3, 1, 64), (32, 2, 64)])
def test_zero_keys_beside_the_largest_one(decode, hq, hkv, dim):
    """A group's scale may be 2^119 for the sake of an element that the queries do not weigh:
    its other keys' scores are zero, however large the queries are."""
    new, prefix = ([1] * 3, [40, 200, 15]) if decode else ([20, 1], [40, 200])
    b = Batch8(new, prefix, 16, hq, hkv, dim, seed=3)
    b.q[:] = (b.q.sign() * 2.0**30).bfloat16()
    b.q[:, :, 0] = 0

    def keys(c, i):
        z = torch.zeros_like(c)
        z[::GROUP, :, 0] = 448
        return z

    for i, (c, e) in enumerate(b.codes["k"]):
        b.codes["k"][i] = c, torch.full_like(e, 119)
    put(b, "k", keys)
    check_attention8(b.fill(), decode=decode)
