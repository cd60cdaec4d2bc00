"""Paged attention over the 8-bit cache on the GPU against its definition in 64 bits."""
import pytest
import torch

import gated_deltanet_paged_gb300 as gdn
from fp8_util import Batch8, check_attention8

pytestmark = pytest.mark.gpu

I16 = torch.int16
SHAPES = [(8, 2, 128), (3, 1, 64), (1, 1, 128), (16, 1, 64), (5, 5, 128), (40, 2, 64), (34, 2, 128)]
CHUNKS = {"ragged": ([100, 37, 0, 1, 65], [0, 64, 7, 63, 1]), "one": ([1], [0]), "long": ([300, 2], [1000, 129]),
          "ends": ([127, 128, 129, 1], [1, 0, 127, 255]), "deep": ([3, 140], [5000, 2600])}


def options(name, hq, new, prefix):
    slopes = torch.tensor([2.0 ** (-4 * (h + 1) / hq) for h in range(hq)], device="cuda")
    full = torch.tensor([p + n // 2 for n, p in zip(new, prefix)], dtype=torch.int32, device="cuda")
    return {"plain": {}, "capped": {"softcap": 5.0}, "window": {"window": 50}, "slopes": {"slopes": slopes},
            "prefix": {"full_lens": full}, "both": {"softcap": 20.0, "slopes": slopes, "window": 130},
            "scale": {"scale": 0.3, "softcap": 30.0, "full_lens": full}}[name]


@pytest.mark.parametrize("lens", CHUNKS)
@pytest.mark.parametrize("page_size,layout", [(16, "nhd"), (48, "hnd"), (896, "fused")])
@pytest.mark.parametrize("hq,hkv,dim", SHAPES[:4])
def test_chunk(lens, page_size, layout, hq, hkv, dim):
    new, prefix = CHUNKS[lens]
    b = Batch8(new, prefix, page_size, hq, hkv, dim, layout=layout, seed=page_size + dim, q_pad=1, padded=layout == "hnd").fill()
    check_attention8(b)


@pytest.mark.parametrize("opts", ["capped", "window", "slopes", "prefix", "both", "scale"])
@pytest.mark.parametrize("lens", ["ragged", "long", "deep"])
@pytest.mark.parametrize("hq,hkv,dim", [SHAPES[0], SHAPES[5], SHAPES[1]])
def test_chunk_options(opts, lens, hq, hkv, dim):
    new, prefix = CHUNKS[lens]
    b = Batch8(new, prefix, 64, hq, hkv, dim, seed=len(opts), q_scale=2.0, layout="hnd").fill()
    check_attention8(b, **options(opts, hq, new, prefix))


ONES = {"short": [1, 2, 15, 16, 17, 101], "mixed": [1, 130, 4100, 700, 33], "long": [9000, 64]}


@pytest.mark.parametrize("lens", ONES)
@pytest.mark.parametrize("page_size,layout", [(16, "fused"), (48, "nhd"), (1024, "hnd")])
@pytest.mark.parametrize("hq,hkv,dim", SHAPES)
def test_decode(lens, page_size, layout, hq, hkv, dim):
    lengths = ONES[lens]
    b = Batch8([1] * len(lengths), [n - 1 for n in lengths], page_size, hq, hkv, dim, layout=layout, seed=page_size + hq,
               q_pad=1, padded=layout == "nhd").fill()
    check_attention8(b, decode=True)


@pytest.mark.parametrize("opts", ["capped", "window", "slopes", "prefix", "both", "scale"])
@pytest.mark.parametrize("lens", ["mixed", "long"])
@pytest.mark.parametrize("hq,hkv,dim", [SHAPES[0], SHAPES[5], SHAPES[6], SHAPES[1]])
def test_decode_options(opts, lens, hq, hkv, dim):
    lengths = ONES[lens]
    new, prefix = [1] * len(lengths), [n - 1 for n in lengths]
    b = Batch8(new, prefix, 64, hq, hkv, dim, seed=len(opts), q_scale=2.0).fill()
    check_attention8(b, decode=True, **options(opts, hq, new, prefix))


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("spread", [1, 40, 100])
def test_scales_far_apart(decode, spread):
    """Groups whose scales differ by up to 2^99: a group of large values takes the whole
    softmax or the whole sum, and the others' share is still right."""
    new, prefix = ([1] * 4, [40, 300, 15, 1500]) if decode else ([20, 200, 1], [40, 10, 700])
    b = Batch8(new, prefix, 32, 8, 2, 128, seed=spread, spread=spread)
    for name in "kv":  # keys small enough for scores that are finite numbers of any size
        for i, (c, e) in enumerate(b.codes[name]):
            e -= spread if name == "k" else spread // 2
            value = c.double() * torch.exp2(e.double()).repeat_interleave(16, 0)[: len(c), :, None]
            getattr(b, name)[i] = value
    b.fill()
    check_attention8(b, decode=decode)


def test_chunk_is_what_the_16_bit_cache_gives():
    """Read back into a 16-bit cache, the same attention gives the same outputs within the
    rounding of weights and outputs (2^-8 each of a weighted sum of values)."""
    new, prefix = [300, 1, 90], [100, 500, 0]
    b = Batch8(new, prefix, 64, 8, 2, 128, seed=11).fill()
    o8 = gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table)
    total = [n + p for n, p in zip(new, prefix)]
    cu = torch.tensor([0, 400, 901, 991], dtype=torch.int32, device="cuda")
    k, v = gdn.gdn_kv_read_paged_fp8(*b.cache, cu, sum(total), *b.table)
    kc = torch.zeros(*b.k_cache.shape, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    gdn.gdn_kv_append_paged(k, v, kc, vc, cu, *b.table)
    o16 = gdn.gdn_attention_paged(b.q, kc, vc, b.cu, *b.table)
    big = float(v.abs().max())
    assert (o8.float() - o16.float()).abs().max() <= 4 * 2.0**-8 * big


@pytest.mark.parametrize("decode", [False, True])
def test_reports_and_skips(decode):
    """A refused sequence's outputs stay as they were, a bad page reads as zeros; both are
    reported, and the others' outputs are what they are without."""
    new, prefix = [1] * 4 if decode else [5, 20, 3, 7], [30, 200, 16, 900]
    good = Batch8(new, prefix, 16, 4, 2, 64, seed=6).fill()
    call = (lambda b, **kw: gdn.gdn_attention_decode_paged_fp8(b.q, *b.cache, *b.table, **kw)) if decode else (
        lambda b, **kw: gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table, **kw))
    ref = call(good)
    rows = torch.ones(sum(new), dtype=torch.bool)
    rows[new[0] : new[0] + new[1]] = False
    for what in ("length", "page"):
        b = Batch8(new, prefix, 16, 4, 2, 64, seed=6).fill()
        if what == "length":
            b.last[1] = 0
        else:
            b.indices[b.indptr[1].item() + 3] = -5
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.full_like(ref, 7.0)
        call(b, o=o, err_word=err)
        assert int(err.item()) == ((2 if what == "length" else 1) << 24 | 1)
        assert torch.isfinite(o.float()).all()
        within = (o[rows].float() - ref[rows].float()).abs().max()
        assert within <= 2.0**-7 * ref.float().abs().max()
        assert (o[~rows] == 7.0).all() == (what == "length")


@pytest.mark.parametrize("opts", ["plain", "window", "slopes", "prefix", "both", "capped", "scale"])
@pytest.mark.parametrize("new,prefix,page_size,hq,hkv,dim,layout", [
    ([700, 0, 300, 1], [100, 40, 1500, 3], 64, 8, 2, 128, "nhd"), ([513, 600], [0, 17], 48, 6, 3, 64, "hnd"),
    ([400], [5000], 896, 16, 1, 128, "fused"), ([900, 0, 300, 1], [100, 40, 1500, 3], 64, 8, 2, 128, "nhd"),
    ([1800, 0, 300, 1], [100, 40, 1500, 3], 64, 8, 2, 128, "nhd"), ([1300, 800], [0, 17], 48, 6, 3, 64, "hnd")])
def test_a_copy_in_16_bits_gives_the_same_bits(new, prefix, page_size, hq, hkv, dim, layout, opts):
    """With the larger workspace what the batch sees is turned into bf16 first."""
    b = Batch8(new, prefix, page_size, hq, hkv, dim, seed=len(opts), layout=layout, padded=layout == "hnd").fill()
    sizes = (len(new), sum(new), hq, hkv, dim, b.indices.numel(), page_size)
    small, large = gdn.gdn_attention_workspace_bytes(*sizes), gdn.gdn_attention_fp8_workspace_bytes(*sizes)
    if sum(new) * hq // hkv >= 2048 * len(new):
        assert large >= small + 4 * b.indices.numel() * page_size * hkv * dim
    else:
        assert large == small
    opts = options(opts, hq, new, prefix)
    out = [check_attention8(b, **opts)]
    for size in (small, max(small, large - 1), large, large + 999):
        ws = torch.full((max(size, 1),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever nothing is written
        out.append(gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table, return_lse=True, workspace=ws[:size], **opts))
    for o, lse in out[1:]:
        assert torch.equal(o.view(I16), out[0][0].view(I16)) and torch.equal(lse, out[0][1])


def test_a_copy_reports_and_skips():
    """Refused sequences and bad pages, where the batch is copied."""
    new, prefix = [700, 600, 900], [30, 200, 900]
    good = Batch8(new, prefix, 16, 8, 2, 64, seed=6).fill()
    ref = gdn.gdn_attention_paged_fp8(good.q, *good.cache, good.cu, *good.table)
    rows = torch.ones(sum(new), dtype=torch.bool)
    rows[700:1300] = False
    for what in ("length", "page"):
        b = Batch8(new, prefix, 16, 8, 2, 64, seed=6).fill()
        if what == "length":
            b.last[1] = 0
        else:
            b.indices[b.indptr[1].item() + 3] = b.k_cache.shape[0]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.full_like(ref, 7.0)
        gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table, o=o, err_word=err)
        assert int(err.item()) == ((2 if what == "length" else 1) << 24 | 1)
        assert torch.isfinite(o.float()).all()
        assert (o[rows].float() - ref[rows].float()).abs().max() <= 2.0**-7 * ref.float().abs().max()
        assert (o[~rows] == 7.0).all() == (what == "length")


def test_a_copy_of_many_sequences():
    """More sequences than threads share a line, empty ones between."""
    new = [(i * 5) % 3 * 20 for i in range(400)]
    new[7] = 6000
    prefix = [(i * 11) % 60 for i in range(400)]
    b = Batch8(new, prefix, 16, 64, 1, 64, seed=2).fill()
    assert gdn.gdn_attention_fp8_workspace_bytes(400, sum(new), 64, 1, 64, b.indices.numel(), 16) > (
        gdn.gdn_attention_workspace_bytes(400, sum(new), 64, 1, 64, b.indices.numel(), 16))
    out = [gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table, window=w) for w in (-1, 50)]
    ws = torch.empty(gdn.gdn_attention_workspace_bytes(400, sum(new), 64, 1, 64, b.indices.numel(), 16), dtype=torch.uint8, device="cuda")
    for w, o in zip((-1, 50), out):
        want = gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table, window=w, workspace=ws)
        assert torch.equal(o.view(I16), want.view(I16))


@pytest.mark.parametrize("cap", [5e-5, 1e-3, 0.5, 5.0, 50.0, 1e4, 3e38])
@pytest.mark.parametrize("decode", [False, True])
def test_caps_of_any_size(cap, decode):
    """Scores from far below a cap to far beyond it."""
    new, prefix = ([1] * 3, [40, 700, 15]) if decode else ([100, 300, 1], [40, 10, 700])
    for q_scale in (0.25, 4.0, 30.0):
        b = Batch8(new, prefix, 32, 8, 2, 128, seed=17, q_scale=q_scale).fill()
        check_attention8(b, decode=decode, softcap=cap)


def test_without_room_for_a_copy():
    """Where the larger workspace cannot be had the call does with what it needs."""
    b = Batch8([700, 40], [0, 300], 16, 8, 1, 64, seed=3).fill()
    want = gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table)
    indices = torch.zeros(600_000, dtype=torch.int32, device="cuda")  # a table with room for 2.4 GB of bf16 pages
    indices[: b.indices.numel()] = b.indices
    sizes = (2, 740, 8, 1, 64, indices.numel(), 16)
    assert gdn.gdn_attention_fp8_workspace_bytes(*sizes) > 2 << 30
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 30)) / total)
    try:
        got = gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, indices, b.indptr, b.last)
        torch.cuda.synchronize()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert (got.float() - want.float()).abs().max() <= 2.0**-7 * want.float().abs().max()
    again = gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, indices, b.indptr, b.last)
    assert torch.equal(again.view(I16), got.view(I16))
