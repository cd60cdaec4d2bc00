"""Norms with the rotation, the quantising append and reading back, on the GPU against
their definitions in 64 bits (fp8_util.py)."""
import pytest
import torch

import gated_deltanet_paged_gb300 as gdn
from attention_util import within
from fp8_util import E4M3, E8M0, GROUP, U8, Batch8, check_codes, e4m3, norm_rope_f64

pytestmark = pytest.mark.gpu

I16 = torch.int16


def freqs(rotary, factor=1.0):
    return gdn.gdn_rope_frequencies(rotary, factor=factor, original_len=4096 if factor > 1 else 0) if rotary else None


def weights(dim, seed, offset):
    gen = torch.Generator().manual_seed(seed)
    return [(1 - offset + 0.3 * torch.randn(dim, generator=gen)).bfloat16().cuda() for _ in range(2)]


# ---------------------------------------------------------------- norm and rotation
@pytest.mark.parametrize("dim,rotary", [(128, 128), (128, 64), (64, 64), (64, 24), (128, 2), (72, 16), (256, 34), (256, 256),
                                        (8, 8), (40, 20), (80, 80), (248, 6), (128, 0), (96, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_norm_rope(dim, rotary, interleaved, offset):
    gen = torch.Generator().manual_seed(dim * 3 + rotary)
    T, hq, hkv = 23, 5, 2
    x = (torch.randn(T, hq + hkv + 1, dim, generator=gen) * torch.exp2(torch.randint(-9, 9, (T, hq + hkv + 1, 1), generator=gen))).bfloat16()
    x[1] = 0  # a head of zeros stays one
    x = x.cuda()
    q, k = x[:, :hq], x[:, hq : hq + hkv]
    if k.data_ptr() % 16:
        k = k.clone()
    pos = torch.randint(-5, 1 << 20, (T,), generator=gen, dtype=torch.int32)
    qw, kw = weights(dim, rotary, offset)
    f = freqs(rotary, 4.0)
    opts = dict(eps=1e-5, weight_offset=offset, interleaved=interleaved, amplitude=1.25)
    got = gdn.gdn_qk_norm_rope(q, k, qw, kw, f, pos.cuda() if rotary else None, **opts)
    opts["offset"] = opts.pop("weight_offset")
    for y, src, w in zip(got, (q, k), (qw, kw)):
        ref, tol = norm_rope_f64(src, w, pos, f, **opts)
        within(y, ref, tol + 2.0**-8 * ref.abs(), "norm and rotation")
    opts["weight_offset"] = opts.pop("offset")
    # In place, in the fused projection itself where its slices are aligned; and queries alone.
    z = x.clone()
    zq, zk = z[:, :hq], z[:, hq : hq + hkv]
    if zk.data_ptr() % 16 == 0:
        a, b = gdn.gdn_qk_norm_rope(zq, zk, qw, kw, f, pos.cuda() if rotary else None, q_out=zq, k_out=zk, **opts)
        assert a.data_ptr() == zq.data_ptr() and b.data_ptr() == zk.data_ptr()
        assert torch.equal(zq.contiguous().view(I16), got[0].view(I16)) and torch.equal(zk.contiguous().view(I16), got[1].view(I16))
        assert torch.equal(z[:, hq + hkv :].contiguous().view(I16), x[:, hq + hkv :].contiguous().view(I16))
    alone = gdn.gdn_qk_norm_rope(q, None, qw, None, f, pos.cuda() if rotary else None, **opts)
    assert alone[1] is None and torch.equal(alone[0].view(I16), got[0].view(I16))


@pytest.mark.parametrize("T,hq,hkv", [(0, 2, 1), (1, 1, 1), (1, 160, 8), (5000, 3, 1)])
def test_norm_rope_sizes(T, hq, hkv):
    gen = torch.Generator().manual_seed(T + hq)
    q, k = (torch.randn(T, h, 128, generator=gen).bfloat16().cuda() for h in (hq, hkv))
    pos = torch.randint(0, 300000, (T,), generator=gen, dtype=torch.int32)
    qw, kw = weights(128, T, 0.0)
    f = freqs(128)
    pick = torch.linspace(0, max(T - 1, 0), min(T, 40)).long()
    got = gdn.gdn_qk_norm_rope(q, k, qw, kw, f, pos.cuda())
    for y, src, w in zip(got, (q, k), (qw, kw)):
        assert y.shape == src.shape
        ref, tol = norm_rope_f64(src[pick.cuda()], w, pos[pick], f)
        within(y[pick.cuda()], ref, tol + 2.0**-8 * ref.abs(), "norm and rotation")


def test_norm_rope_of_non_finite_heads():
    """A head with an infinity or a NaN is its own affair."""
    q = torch.randn(4, 6, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    w = weights(64, 2, 0.0)[0]
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    clean = gdn.gdn_qk_norm_rope(q, None, w, None, freqs(64), pos)[0]
    q[1, 2, 7], q[2, 5, 0] = float("nan"), float("inf")
    got = gdn.gdn_qk_norm_rope(q, None, w, None, freqs(64), pos)[0]
    keep = torch.ones(4, 6, dtype=torch.bool, device="cuda")
    keep[1, 2] = keep[2, 5] = False
    assert torch.equal(got[keep].view(I16), clean[keep].view(I16))
    assert got[1, 2].isnan().all()


# ------------------------------------------------------------------------------ append
def check_append(b, k, v, q, *, rotary=0, interleaved=False, amplitude=1.0, offset=None, eps=1e-6, cu=True, fill=True, factor=1.0):
    """One append against the definition: every code, scale and query, and everything else
    as it was."""
    if fill:
        b.fill(upto_prefix=True)
    before = [x.clone() for x in (b.k_cache, b.v_cache, b.k_scales, b.v_scales)]
    f = freqs(rotary, factor)
    qw, kw = (None, None) if offset is None else weights(b.dim, 5, offset)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = gdn.gdn_kv_append_paged_fp8(k, v, *b.cache, b.cu if cu else None, *b.table, q=q, q_weight=qw, k_weight=kw, eps=eps,
                                        weight_offset=offset or 0.0, frequencies=f, interleaved=interleaved,
                                        amplitude=amplitude, err_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    pos = torch.cat([torch.arange(p, p + n) for n, p in zip(b.new, b.prefix)])
    opts = dict(eps=eps, offset=offset or 0.0, interleaved=interleaved, amplitude=amplitude)
    if q is not None:
        ref, tol = norm_rope_f64(q, qw, pos, f, **opts)
        within(q_out, ref, tol + 2.0**-8 * ref.abs(), "q")
    else:
        assert q_out is None
    ky, kt = norm_rope_f64(k, kw, pos, f, **opts)
    if offset is None and not rotary:
        kt = torch.zeros_like(kt)
    vy = v.double().cpu()
    touched = torch.zeros(b.k_cache.shape[:2], dtype=torch.bool, device="cuda")
    scaled = torch.zeros(b.k_scales.shape[:2], dtype=torch.bool, device="cuda")
    for name, y, tol, cache, scales, cache0, scales0 in (("k", ky, kt, b.k_cache, b.k_scales, before[0], before[2]),
                                                         ("v", vy, torch.zeros_like(vy), b.v_cache, b.v_scales, before[1], before[3])):
        t = 0
        for s, (n, p) in enumerate(zip(b.new, b.prefix)):
            for at in range(p // GROUP * GROUP, p + n if n else 0, GROUP):
                r0, r1 = max(p, at), min(p + n, at + GROUP)
                page, slot = b.slots(s, range(at, r1))
                group = (page[0], slot[0] // GROUP)
                scaled[group] = True
                touched[page, slot] = True
                codes = cache[page, slot].view(E4M3).cpu()
                bytes_, bytes0 = scales[group].cpu(), scales0[group].cpu()
                rows = slice(t + r0 - p, t + r1 - p)
                for h in range(b.hkv):
                    check_codes(name, int(bytes_[h]), codes[r0 - at :, h], y[rows, h], tol[rows, h], None, int(bytes0[h]), r0 - at)
                if r0 > at:  # earlier tokens' codes, rounded to the scale that may have grown
                    old = cache0[page, slot].view(E4M3).cpu()[: r0 - at].double()
                    want = e4m3(old * torch.exp2(bytes0.double() - bytes_.double())[:, None])
                    assert torch.equal(want.to(E4M3).view(U8), codes[: r0 - at].contiguous().view(U8)), "%s: earlier tokens" % name
            t += n
        assert torch.equal(cache[~touched], cache0[~touched]), "a slot outside the call's groups changed"
        assert torch.equal(scales[~scaled], scales0[~scaled]), "a scale outside the call's groups changed"
    return q_out


LENS = {"ragged": ([100, 37, 0, 1, 65], [0, 64, 7, 63, 1]), "one": ([1], [0]), "long": ([300, 2], [1000, 129]),
        "ends": ([15, 16, 17, 1, 1, 2, 31], [1, 16, 15, 15, 16, 31, 33])}


def inputs(b, seed, spread=4, q_heads=0):
    """New tokens' k, v (slices of a fused projection) and q, sizes spread over tokens."""
    gen = torch.Generator().manual_seed(seed)
    T = sum(b.new)
    size = torch.exp2(torch.randint(-spread, spread + 1, (T, 1, 1), generator=gen))
    fused = (torch.randn(T, 2 * b.hkv, b.dim, generator=gen) * size).bfloat16().cuda()
    return fused[:, : b.hkv], fused[:, b.hkv :], b.q if q_heads else None


@pytest.mark.parametrize("layout", ["nhd", "hnd", "fused"])
@pytest.mark.parametrize("page_size,lens,hq,hkv,dim,rotary,interleaved,offset",
                         [(64, "ragged", 8, 2, 128, 128, False, 0.0), (16, "long", 3, 3, 64, 32, True, 1.0),
                          (16, "one", 1, 1, 64, 24, False, None), (48, "ragged", 6, 1, 128, 64, True, None),
                          (896, "long", 0, 4, 128, 128, False, 0.0), (32, "ends", 5, 5, 64, 0, False, None),
                          (80, "ends", 33, 1, 128, 2, False, 1.0), (64, "ends", 4, 2, 128, 0, True, 0.0),
                          (16, "ragged", 2, 2, 128, 8, True, None), (1152, "ends", 16, 8, 64, 4, False, 0.0)])
def test_append(page_size, lens, hq, hkv, dim, rotary, interleaved, offset, layout):
    new, prefix = LENS[lens]
    b = Batch8(new, prefix, page_size, max(hq, 1), hkv, dim, layout=layout, seed=page_size, q_pad=2, padded=layout == "hnd")
    k, v, q = inputs(b, rotary, q_heads=hq)
    check_append(b, k, v, q, rotary=rotary, interleaved=interleaved, amplitude=1.5, offset=offset, eps=1e-5, factor=4.0)


def test_append_token_by_token_and_again():
    """Forty tokens one at a time, without cu_seqlens, their sizes growing and falling: scales
    never fall inside a group, and the same tokens appended twice leave the cache as it is."""
    tokens = 40
    b = Batch8([tokens, tokens], [0, 0], 32, 2, 2, 64, seed=3)
    gen = torch.Generator().manual_seed(4)
    last = None
    for i in range(tokens):
        step = Batch8([1, 1], [i, i], 32, 2, 2, 64, seed=3)
        for x in ("k_cache", "v_cache", "k_scales", "v_scales", "owned"):
            setattr(step, x, getattr(b, x))
        pages = i // 32 + 1
        step.indices = torch.tensor([p for own in b.owned for p in own[:pages]], dtype=torch.int32, device="cuda")
        k, v = ((torch.randn(2, 2, 64, generator=gen) * 2.0 ** (8 - abs(i % 16 - 8))).bfloat16().cuda() for _ in range(2))
        check_append(step, k, v, step.q, rotary=64, offset=0.0, cu=False, fill=False)
        again = [x.clone() for x in (b.k_cache, b.v_cache, b.k_scales, b.v_scales)]
        check_append(step, k, v, step.q, rotary=64, offset=0.0, cu=False, fill=False)
        for x, y in zip(again, (b.k_cache, b.v_cache, b.k_scales, b.v_scales)):
            assert torch.equal(x, y)
        scale = b.v_scales[b.owned[0][i // 32], i % 32 // GROUP].clone()
        if i % GROUP:
            assert (scale >= last).all()
        last = scale


def test_append_one_token_each_with_and_without_cu_seqlens():
    out = []
    for cu in (True, False):
        b = Batch8([1] * 70, [i * 13 for i in range(70)], 32, 4, 2, 64, seed=3)
        k, v, q = inputs(b, 1, q_heads=4)
        qo = check_append(b, k, v, q, rotary=64, offset=1.0, cu=cu)
        out.append([qo.view(I16), b.k_cache, b.v_cache, b.k_scales, b.v_scales])
    for x, y in zip(*out):
        assert torch.equal(x, y)


def test_append_many_sequences_finds_each_group():
    """More sequences than one step of the search covers, empty ones between."""
    new = [(i * 7) % 4 * (1 + 9 * (i % 50 == 0)) for i in range(1300)]
    b = Batch8(new, [(i * 5) % 37 for i in range(1300)], 16, 1, 1, 64, seed=9, spare=1)
    k, v, q = inputs(b, 2, q_heads=1)
    check_append(b, k, v, q)


@pytest.mark.parametrize("size", [2.0**-130, 2.0**-105, 2.0**-100, 2.0**100, 2.0**126, 0.0])
def test_append_ends_of_the_scales(size):
    """Sizes at and beyond both ends of the scales: 2^-112 at least, 2^119 at most."""
    b = Batch8([16, 3], [0, 20], 32, 1, 1, 64, seed=1)
    gen = torch.Generator().manual_seed(8)
    k, v = ((torch.randn(19, 1, 64, generator=gen).clamp(-1.9, 1.9) * size).bfloat16().cuda() for _ in range(2))
    check_append(b, k, v, None)
    page, slot = b.slots(0, [0])
    byte = int(b.v_scales[page[0], 0, 0])
    assert 15 <= byte <= 246


def test_append_of_infinities_and_nan():
    """An infinity is stored as the largest number and takes its group's scale along, NaN
    stays NaN and takes nothing along; other heads and groups are not touched."""
    b = Batch8([40], [0], 64, 1, 2, 64, seed=1)
    v = torch.randn(40, 2, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    clean = Batch8([40], [0], 64, 1, 2, 64, seed=1)
    gdn.gdn_kv_append_paged_fp8(v, v, *clean.cache, clean.cu, *clean.table)
    v[3, 0, 5], v[20, 1, 6] = float("-inf"), float("nan")
    gdn.gdn_kv_append_paged_fp8(v, v, *b.cache, b.cu, *b.table)
    page = b.owned[0][0]
    assert int(b.v_scales[page, 0, 0]) == 246 and int(b.v_cache[page, 3, 0, 5]) == 0xFE
    assert int(b.v_cache[page, 20, 1, 6]) & 0x7F == 0x7F
    same = torch.ones(40, 2, 64, dtype=torch.bool, device="cuda")
    same[:16, 0] = False
    same[20, 1, 6] = False
    assert torch.equal(b.v_cache[page, :40][same], clean.v_cache[page, :40][same])
    scales = b.v_scales[page].clone()
    scales[0, 0] = clean.v_scales[page, 0, 0]
    assert torch.equal(scales, clean.v_scales[page])


def test_append_reports_and_skips():
    """A refused sequence and a bad page leave the others' results; queries of a token on a
    bad page are rotated all the same."""
    new, prefix = [5, 20, 3, 7], [3, 0, 16, 40]
    good = Batch8(new, prefix, 16, 2, 1, 64, seed=6)
    k, v, q = inputs(good, 3, q_heads=2)
    good.fill(upto_prefix=True)
    ref = gdn.gdn_kv_append_paged_fp8(k, v, *good.cache, good.cu, *good.table, q=q, frequencies=freqs(64))
    for what in ("length", "page"):
        b = Batch8(new, prefix, 16, 2, 1, 64, seed=6)
        b.fill(upto_prefix=True)
        before = [x.clone() for x in (b.k_cache, b.k_scales)]
        if what == "length":
            b.last[1] = 17  # more than a page
            bad = b.owned[1]
        else:
            b.indices[b.indptr[1].item() + 1] = b.k_cache.shape[0]
            bad = b.owned[1][1:]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.full_like(q.contiguous(), 7.0)
        gdn.gdn_kv_append_paged_fp8(k, v, *b.cache, b.cu, *b.table, q=q, frequencies=freqs(64), q_out=q_out, err_word=err)
        assert int(err.item()) == ((2 if what == "length" else 1) << 24 | 1)
        keep = torch.ones(b.k_cache.shape[0], dtype=torch.bool)
        keep[bad] = False
        assert torch.equal(b.k_cache[keep], good.k_cache[keep]) and torch.equal(b.k_scales[keep], good.k_scales[keep])
        assert torch.equal(b.k_cache[~keep], before[0][~keep]) and torch.equal(b.k_scales[~keep], before[1][~keep])
        rows = torch.arange(sum(new)) if what == "page" else torch.cat([torch.arange(0, 5), torch.arange(25, 35)])
        assert torch.equal(q_out[rows].view(I16), ref[rows].view(I16))
        if what == "length":
            assert (q_out[5:25] == 7.0).all()


# -------------------------------------------------------------------------------- read
@pytest.mark.parametrize("layout", ["nhd", "hnd", "fused"])
@pytest.mark.parametrize("page_size,lens,hkv,dim", [(64, "ragged", 2, 128), (16, "long", 3, 64), (48, "ends", 1, 128),
                                                     (1152, "ends", 8, 64), (16, "one", 1, 64)])
def test_read(page_size, lens, hkv, dim, layout):
    new, prefix = LENS[lens]
    b = Batch8(new, prefix, page_size, 1, hkv, dim, layout=layout, seed=page_size, padded=layout != "nhd", spread=60).fill()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gdn.gdn_kv_read_paged_fp8(*b.cache, b.cu, sum(new), *b.table, err_word=err)
    assert int(err.item()) == 0
    for y, name in zip(got, "kv"):
        want = torch.cat([x[p:] for x, p in zip(getattr(b, name), prefix)])
        assert y.dtype == torch.bfloat16 and torch.equal(y.double().cpu(), want)
    # One token each, and into given rows of which the last sequence leaves some.
    if all(new):
        one = gdn.gdn_kv_read_paged_fp8(*b.cache, None, len(new), *b.table)
        assert torch.equal(one[0].double().cpu(), torch.stack([x[-1] for x in b.k]))
    T = sum(new) + 3
    outs = [torch.full((T, hkv, dim), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    a = gdn.gdn_kv_read_paged_fp8(*b.cache, b.cu, T, *b.table, k_out=outs[0], v_out=outs[1])
    assert a[0] is outs[0] and torch.equal(outs[1][:-3].view(I16), got[1].view(I16)) and (outs[0][-3:] == 9.0).all()


def test_read_back_what_was_appended():
    """The values read back are within half a step of what went in, every code and scale byte
    of an append reads as its value, and appending them again changes nothing."""
    b = Batch8([200, 33], [0, 0], 64, 1, 2, 128, seed=5)
    k, v, _ = inputs(b, 7, spread=12)
    gdn.gdn_kv_append_paged_fp8(k, v, *b.cache, b.cu, *b.table)
    kk, vv = gdn.gdn_kv_read_paged_fp8(*b.cache, b.cu, 233, *b.table)
    codes = [x.clone() for x in (b.k_cache, b.v_cache)]
    gdn.gdn_kv_append_paged_fp8(kk, vv, *b.cache, b.cu, *b.table)
    again = gdn.gdn_kv_read_paged_fp8(*b.cache, b.cu, 233, *b.table)
    assert torch.equal(again[0].view(I16), kk.view(I16)) and torch.equal(again[1].view(I16), vv.view(I16))
    # All 256 codes under all scales that an append writes.
    c = torch.arange(256, dtype=torch.int32).to(U8)
    kc = c.view(1, 1, 1, 256).expand(232, 16, 1, 256)[..., :128].contiguous().cuda()
    vc = c.view(1, 1, 1, 256).expand(232, 16, 1, 256)[..., 128:].contiguous().cuda()
    s = torch.arange(15, 247, dtype=torch.int32).to(U8).view(232, 1, 1).cuda()
    cache = kc.view(E4M3), vc.view(E4M3), s.view(E8M0), s.view(E8M0)
    table = [torch.arange(n, dtype=torch.int32, device="cuda") for n in (232, 233)] + [torch.full((232,), 1, dtype=torch.int32, device="cuda")]
    got = gdn.gdn_kv_read_paged_fp8(*cache, None, 232, *table)
    want = torch.exp2(s.double().cpu() - 127)[:, 0]
    for y, x in zip(got, (kc, vc)):
        ref = x[:, 0, 0].view(E4M3).double().cpu() * want
        assert torch.equal(y[:, 0].double().cpu().nan_to_num(1e300), ref.nan_to_num(1e300))


def test_read_of_a_bad_page_is_zeros():
    b = Batch8([20, 20], [0, 0], 16, 1, 1, 64, seed=2).fill()
    b.indices[1] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, _ = gdn.gdn_kv_read_paged_fp8(*b.cache, b.cu, 40, *b.table, err_word=err)
    assert int(err.item()) == 1 << 24
    assert (k[16:20] == 0).all() and torch.equal(k[20:].double().cpu(), b.k[1])


# --------------------------------------------------------------------------- refusals
def test_python_refusals():
    b = Batch8([4], [0], 32, 2, 1, 64, seed=2)
    k, v, q = inputs(b, 1, q_heads=2)
    w = weights(64, 1, 0.0)
    kc, vc, ks, vs = b.cache
    bad = [(ValueError, dict(q_weight=w[0])), (ValueError, dict(k_weight=w[0])), (TypeError, dict(q_weight=w[0].float(), k_weight=w[0])),
           (ValueError, dict(q_weight=w[0][:32], k_weight=w[0])), (ValueError, dict(q_out=q.clone()[:2], q=q))]
    for error, opts in bad:
        with pytest.raises(error):
            gdn.gdn_kv_append_paged_fp8(k, v, kc, vc, ks, vs, b.cu, *b.table, **opts)
    for cache, error in (((b.k_cache, vc, ks, vs), TypeError), ((kc, vc, b.k_scales, vs), TypeError), ((kc, vc[:, :16], ks, vs), ValueError),
                         ((kc, vc, ks[:, :1], vs), ValueError), ((kc, vc, ks, vs.expand(vs.shape[0], 2, 1)[:, :, :0]), ValueError),
                         ((kc[:, :24], vc[:, :24], ks, vs), ValueError), ((kc.cpu(), vc, ks, vs), ValueError)):
        with pytest.raises(error):
            gdn.gdn_kv_append_paged_fp8(k, v, *cache, b.cu, *b.table)
        with pytest.raises(error):
            gdn.gdn_attention_paged_fp8(q, *cache, b.cu, *b.table)
        with pytest.raises(error):
            gdn.gdn_kv_read_paged_fp8(*cache, b.cu, 4, *b.table)
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope(q, None, w[0], w[1])
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope(q, k, w[0], None)
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope(q, k, w[0], w[1], freqs(64))
    with pytest.raises(gdn.GdnError):
        gdn.gdn_qk_norm_rope(q, k, w[0], w[1], eps=0.0)
