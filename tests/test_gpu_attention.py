"""Rotary positions, the paged key / value append and paged attention on the
GPU against their definitions in 64 bits (tests/attention_util.py)."""
import itertools

import pytest
import torch

import gated_deltanet_paged_gb300 as gdn
from attention_util import Batch, attention_f64, check_attention, rope_f64, within

pytestmark = pytest.mark.gpu

I16 = torch.int16


def freqs(rotary, factor=1.0):
    return gdn.gdn_rope_frequencies(rotary, factor=factor, original_len=4096 if factor > 1 else 0)


# ------------------------------------------------------------------ rotation
@pytest.mark.parametrize("dim,rotary", [(128, 128), (128, 64), (64, 64), (64, 24), (128, 2), (72, 16), (256, 34),
                                        (8, 8), (40, 20)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(dim, rotary, interleaved, inverse):
    gen = torch.Generator().manual_seed(dim * rotary)
    T, H = 37, 5
    x = torch.randn(T, H + 3, dim, generator=gen).bfloat16().cuda()[:, 1 : 1 + H]
    if x.data_ptr() % 16:
        x = x.clone()
    pos = torch.randint(-5, 1 << 20, (T,), generator=gen, dtype=torch.int32)
    pos[:3] = torch.tensor([0, (1 << 31) - 1, -(1 << 31)])
    f = freqs(rotary, 4.0)
    y = gdn.gdn_rope(x, f, pos.cuda(), interleaved=interleaved, inverse=inverse, amplitude=1.25)
    ref, tol = rope_f64(x, pos, f.cpu(), interleaved, inverse, 1.25)
    within(y, ref, tol, "rope")
    assert torch.equal(y[..., rotary:].view(I16), x[..., rotary:].contiguous().view(I16))
    z = x.contiguous().clone()
    assert gdn.gdn_rope(z, f, pos.cuda(), interleaved=interleaved, inverse=inverse, amplitude=1.25, out=z) is z
    assert torch.equal(z.view(I16), y.view(I16)), "in place"


@pytest.mark.parametrize("T,H", [(0, 2), (1, 1), (1, 160), (5000, 3)])
def test_rope_sizes(T, H):
    gen = torch.Generator().manual_seed(T + H)
    x = torch.randn(T, H, 128, generator=gen).bfloat16().cuda()
    pos = torch.randint(0, 300000, (T,), generator=gen, dtype=torch.int32)
    f = freqs(128)
    pick = torch.linspace(0, max(T - 1, 0), min(T, 40)).long()
    y = gdn.gdn_rope(x, f, pos.cuda())
    ref, tol = rope_f64(x[pick.cuda()], pos[pick], f.cpu())
    within(y[pick.cuda()], ref, tol, "rope")


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """The rotation is linear: column e of its matrix is the difference
    R(x + e) - R(x), here at x = 0, and the gradient's rotation (inverse) has to
    be the transposed matrix, bit for bit (each entry is one rounding of the same
    product); against the formula through autograd in 64 bits as well."""
    D, rotary = 64, 48
    f = freqs(rotary)
    eye = torch.eye(D).bfloat16().cuda()[:, None]
    pos = torch.full((D,), 77, dtype=torch.int32, device="cuda")
    m = gdn.gdn_rope(eye, f, pos, interleaved=interleaved, amplitude=1.5)[:, 0]
    mt = gdn.gdn_rope(eye, f, pos, interleaved=interleaved, amplitude=1.5, inverse=True)[:, 0]
    assert torch.equal(m.float(), mt.float().T)
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(3, 2, D, generator=gen, dtype=torch.float64, requires_grad=True)
    w = torch.randn(3, 2, D, generator=gen).bfloat16()
    p = torch.tensor([3, 1000, 70000], dtype=torch.int32)
    half = rotary // 2
    ang = p.double()[:, None, None] * torch.tensor([10000.0 ** (-2 * i / rotary) for i in range(half)], dtype=torch.float64)
    a, b = (x[..., 0:rotary:2], x[..., 1:rotary:2]) if interleaved else (x[..., :half], x[..., half:rotary])
    ya, yb = a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()
    wa, wb = (w[..., 0:rotary:2], w[..., 1:rotary:2]) if interleaved else (w[..., :half], w[..., half:rotary])
    ((ya * wa).sum() + (yb * wb).sum() + (x[..., rotary:] * w[..., rotary:]).sum()).backward()
    got = gdn.gdn_rope(w.cuda(), f, p.cuda(), interleaved=interleaved, inverse=True)
    _, tol = rope_f64(w, p, f.cpu(), interleaved, True)
    within(got, x.grad, tol + 2.0**-40, "gradient")


# -------------------------------------------------------------------- append
LENS = {"ragged": ([100, 37, 0, 1, 65], [0, 64, 7, 63, 1]), "one": ([1], [0]), "long": ([300, 2], [1000, 129])}


@pytest.mark.parametrize("layout", ["nhd", "hnd", "fused"])
@pytest.mark.parametrize("page_size,lens,hq,hkv,dim,rotary,interleaved",
                         [(64, "ragged", 8, 2, 128, 128, False), (16, "long", 3, 3, 64, 32, True),
                          (1, "one", 1, 1, 64, 24, False), (7, "ragged", 6, 1, 128, 64, True),
                          (896, "long", 0, 4, 128, 128, False), (24, "ragged", 5, 5, 72, 0, False)])
def test_append(page_size, lens, hq, hkv, dim, rotary, interleaved, layout):
    new, prefix = LENS[lens]
    b = Batch(new, prefix, page_size, max(hq, 1), hkv, dim, layout=layout, seed=page_size, q_pad=2)
    b.fill(upto_prefix=True)
    k_before, v_before = b.k_cache.clone(), b.v_cache.clone()
    f = freqs(rotary) if rotary else None
    k = torch.cat([b.k[i][p:] for i, p in enumerate(prefix)])
    v = torch.cat([b.v[i][p:] for i, p in enumerate(prefix)])
    fused = torch.cat([k, v], 1).cuda()  # a fused projection: k and v are slices of it
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = b.q if hq else None
    q_out = gdn.gdn_kv_append_paged(fused[:, :hkv], fused[:, hkv:], b.k_cache, b.v_cache, b.cu, *b.table, q=q,
                                    frequencies=f, interleaved=interleaved, amplitude=1.5, err_word=err)
    assert int(err.item()) == 0
    pos = torch.cat([torch.arange(p, p + n) for n, p in zip(new, prefix)])
    none = torch.zeros(0, dtype=torch.int64)
    kr, kt = rope_f64(k, pos, f.cpu() if rotary else none, interleaved, False, 1.5)
    touched = torch.zeros(b.k_cache.shape[:2], dtype=torch.bool, device="cuda")
    t = 0
    for s, (n, p) in enumerate(zip(new, prefix)):
        page, slot = b.slots(s, range(p, p + n))
        touched[page, slot] = True
        within(b.k_cache[page, slot], kr[t : t + n], kt[t : t + n], "k cache")
        assert torch.equal(b.v_cache[page, slot].view(I16), v[t : t + n].cuda().view(I16)), "v cache"
        t += n
    for now, before in ((b.k_cache, k_before), (b.v_cache, v_before)):
        assert torch.equal(now[~touched].view(I16), before[~touched].view(I16)), "a slot outside the new tokens changed"
    if hq:
        qr, qt = rope_f64(b.q, pos, f.cpu() if rotary else none, interleaved, False, 1.5)
        within(q_out, qr, qt, "q")
    else:
        assert q_out is None


def test_append_one_token_each_without_cu_seqlens():
    b = Batch([1] * 70, [i * 13 for i in range(70)], 32, 4, 2, 64, seed=3)
    f = freqs(64)
    k = torch.stack([x[-1] for x in b.k]).cuda()
    v = torch.stack([x[-1] for x in b.v]).cuda()
    kc, vc = b.k_cache.clone(), b.v_cache.clone()
    q1 = gdn.gdn_kv_append_paged(k, v, b.k_cache, b.v_cache, b.cu, *b.table, q=b.q, frequencies=f)
    q2 = gdn.gdn_kv_append_paged(k, v, kc, vc, None, *b.table, q=b.q, frequencies=f)
    for x, y in ((q1, q2), (b.k_cache, kc), (b.v_cache, vc)):
        assert torch.equal(x.view(I16), y.view(I16))


def test_append_many_sequences_finds_each_token():
    """More sequences than one step of the search covers, empty ones between."""
    new = [(i * 7) % 4 for i in range(1500)]
    b = Batch(new, [1] * 1500, 8, 1, 1, 64, seed=9)
    k = torch.cat([x[1:] for x in b.k]).cuda()
    gdn.gdn_kv_append_paged(k, k, b.k_cache, b.v_cache, b.cu, *b.table)
    at = [b.slots(s, range(1, n + 1)) for s, n in enumerate(new)]
    page, slot = torch.cat([x[0] for x in at]), torch.cat([x[1] for x in at])
    assert torch.equal(b.k_cache[page, slot].view(I16), k.view(I16))
    assert int(torch.isnan(b.k_cache[:, :, 0, 0]).sum()) == b.k_cache.shape[0] * 8 - k.shape[0]


# ----------------------------------------------------------------- attention
SHAPES = {
    "ragged": ([100, 37, 0, 1, 65, 129], [0, 64, 7, 63, 1, 127]),
    "first": ([1, 2, 128], [0, 0, 0]),
    "long": ([300, 2, 17], [1000, 2303, 640]),
    "edge": ([128, 256, 127, 1], [128, 0, 1, 1151]),
}


@pytest.mark.parametrize("lens", list(SHAPES))
@pytest.mark.parametrize("page_size,hq,hkv,dim,layout", [(64, 4, 1, 128, "nhd"), (16, 6, 2, 64, "hnd"),
                                                         (1024, 16, 2, 128, "fused"), (24, 5, 5, 64, "nhd"),
                                                         (7, 14, 2, 128, "hnd"), (1152, 40, 1, 64, "nhd")])
def test_chunk_attention(lens, page_size, hq, hkv, dim, layout):
    b = Batch(*SHAPES[lens], page_size, hq, hkv, dim, layout=layout, seed=page_size + hq, q_pad=1).fill()
    check_attention(b)


def _options(name, hq, seqs):
    opts = {}
    if "cap" in name:
        opts["softcap"] = 100.0 if "highcap" in name else 12.0
    if "slope" in name:
        opts["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device="cuda")
    if "window" in name:
        opts["window"] = int(name.split("window")[1])
    if "prefix" in name:
        opts["full_lens"] = torch.tensor([(0, 50, 3, 10000, 64, 200)[i % 6] for i in range(seqs)], dtype=torch.int32,
                                         device="cuda")
    if "scale" in name:
        opts["scale"] = 0.3
    return opts


OPTIONS = ["cap", "slope", "window0", "window1", "window100", "window5000", "prefix", "cap slope window200", "scale",
           "cap slope prefix scale", "highcap", "highcap slope window64", "cap window100", "cap prefix", "cap window0"]


@pytest.mark.parametrize("name", OPTIONS)
@pytest.mark.parametrize("hq,hkv,dim,page_size", [(8, 2, 128, 64), (7, 1, 64, 16)])
def test_chunk_options(name, hq, hkv, dim, page_size):
    for lens in ("ragged", "long"):
        b = Batch(*SHAPES[lens], page_size, hq, hkv, dim, seed=3, q_scale=3.0).fill()
        check_attention(b, **_options(name, hq, len(b.new)))


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("window", [2**30 - 1, 2**30, 2**31 - 1])
def test_windows_beyond_any_sequence_hide_nothing(decode, window):
    new, prefix = ([1] * 3, [20, 1500, 0]) if decode else ([200, 3, 65], [20, 1500, 0])
    b = Batch(new, prefix, 64, 32, 8, 128, seed=22).fill()
    o, lse = check_attention(b, decode=decode, window=window)
    o2, lse2 = check_attention(b, decode=decode)
    assert torch.equal(o.view(I16), o2.view(I16)) and torch.equal(lse, lse2)


def test_single_row_groups_of_every_size():
    """Every number of query heads per key head up to the largest."""
    for g in (1, 2, 3, 5, 9, 16, 17, 31, 43, 64, 65, 100, 128):
        b = Batch([3, 1], [70, 300], 32, g, 1, 64, seed=g).fill()
        check_attention(b)
        d = Batch([1, 1, 1], [70, 300, 0], 32, g, 1, 64, seed=g).fill()
        check_attention(d, decode=True)


# How a batch is shared out: (new, prefix); with 32 query heads on 8 key heads a
# sequence has ceil(new / 64) * 8 items.
SHARED = {
    "few items, all short": ([64] * 8, [400, 0, 17, 300, 64, 960, 1, 128]),
    "many items, all short": ([500, 333, 64, 1, 400], [0, 100, 200, 1000, 3]),
    "few items, one cut into many": ([16], [4000]),
    "few items of unlike lengths": ([40, 64, 1], [5000, 90, 700]),
    "items longer than a share of the line": ([750], [4000]),
    "many items, some long": ([900, 1, 300], [300, 2500, 1100]),
    "a long one beside sequences without pages": ([0] * 60 + [40] + [0] * 9, [0] * 60 + [3000] + [0] * 9),
}


@pytest.mark.parametrize("window", [-1, 700])
@pytest.mark.parametrize("name", list(SHARED))
def test_every_way_of_sharing_out(name, window):
    b = Batch(*SHARED[name], 64, 32, 8, 128, seed=21).fill()
    check_attention(b, window=window)


@pytest.mark.parametrize("name", list(SHARED))
def test_every_way_of_sharing_out_under_a_cap(name):
    b = Batch(*SHARED[name], 64, 32, 8, 64, seed=23, q_scale=3.0).fill()
    check_attention(b, softcap=20.0, window=900)


@pytest.mark.parametrize("g", [1, 3, 16, 43, 100, 128])
def test_groups_under_a_cap(g):
    b = Batch([3, 150, 0, 1], [70, 300, 9, 0], 32, g, 1, 128, seed=g, q_scale=4.0).fill()
    check_attention(b, softcap=6.0)


# -------------------------------------------------------------------- decode
DECODE = {"one": [0], "short": [0, 1, 15, 16, 17, 63, 64, 65], "mixed": [5, 4000, 127, 128, 129, 1000, 0, 2222, 511],
          "long": [20000, 3]}


@pytest.mark.parametrize("lens", list(DECODE))
@pytest.mark.parametrize("page_size,hq,hkv,dim,layout", [(64, 4, 1, 128, "nhd"), (16, 6, 2, 64, "hnd"),
                                                         (1024, 16, 2, 128, "fused"), (24, 5, 5, 64, "nhd"),
                                                         (5, 14, 2, 128, "hnd"), (1152, 40, 2, 128, "nhd")])
def test_decode_attention(lens, page_size, hq, hkv, dim, layout):
    p = DECODE[lens]
    b = Batch([1] * len(p), p, page_size, hq, hkv, dim, layout=layout, seed=page_size + hq, q_pad=1).fill()
    check_attention(b, decode=True)


@pytest.mark.parametrize("name", OPTIONS)
@pytest.mark.parametrize("hq,hkv,dim,page_size", [(8, 2, 128, 64), (7, 1, 64, 16)])
def test_decode_options(name, hq, hkv, dim, page_size):
    p = DECODE["mixed"]
    b = Batch([1] * len(p), p, page_size, hq, hkv, dim, seed=3, q_scale=3.0).fill()
    check_attention(b, decode=True, **_options(name, hq, len(p)))


def test_decode_many_sequences():
    p = [(i * 37) % 400 for i in range(600)]
    check_attention(Batch([1] * 600, p, 16, 8, 2, 128, seed=4).fill(), decode=True)


def test_chunk_many_sequences():
    new, p = [(i * 7) % 6 for i in range(700)], [1 + (i * 37) % 90 for i in range(700)]
    check_attention(Batch(new, p, 16, 2, 1, 64, seed=4).fill())


# ------------------------------------------------ what lies in masked places
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3.38e38])
def test_keys_that_left_the_window_may_hold_anything(decode, bad):
    """Slots before every new token's window, and slots past the end, hold
    values that would spoil any sum they entered."""
    new = [1] * 4 if decode else [1, 40, 128, 7]
    prefix = [300, 517, 1000, 0]
    w = 90
    b = Batch(new, prefix, 48, 6, 2, 128, seed=8)
    b.k_cache.fill_(bad)
    b.v_cache.fill_(bad)
    b.fill(window_from=[max(0, p - w) for p in prefix])
    check_attention(b, decode=decode, window=w)


@pytest.mark.parametrize("decode", [False, True])
def test_large_scores_and_equal_scores(decode):
    """Scores whose exponentials overflow without the maximum, and all-equal
    scores (zero keys): finite outputs, the mean of the values."""
    new, prefix = ([1, 1], [200, 65]) if decode else ([50, 3], [200, 65])
    b = Batch(new, prefix, 64, 4, 2, 64, seed=2, q_scale=100.0).fill()
    check_attention(b, decode=decode)
    b = Batch(new, prefix, 64, 4, 2, 64, seed=2)
    for k in b.k:
        k.zero_()
    check_attention(b.fill(), decode=decode)


@pytest.mark.parametrize("decode", [False, True])
def test_rising_and_falling_maxima(decode):
    """Keys whose scores grow along the sequence (the running maximum moves at
    every block) and ones that shrink (it never does)."""
    for sign in (1.0, -1.0):
        new, prefix = ([1, 1], [1500, 400]) if decode else ([130, 1], [1500, 400])
        b = Batch(new, prefix, 128, 4, 1, 128, seed=2)
        b.q[:] = b.q.abs()
        for k in b.k:
            ramp = torch.linspace(0, 6, k.shape[0])[:, None, None]
            k[:] = (sign * ramp + 0.1 * k.float()).bfloat16()
        check_attention(b.fill(), decode=decode)


# --------------------------------------------------------------- bad batches
@pytest.mark.parametrize("decode", [False, True])
def test_refused_sequences_are_skipped_and_reported(decode):
    new, prefix = ([1] * 4, [100, 40, 7, 130]) if decode else ([60, 3, 70, 5], [100, 40, 7, 130])
    b = Batch(new, prefix, 16, 4, 2, 64, seed=6).fill()
    ref = attention_f64(b)
    start = [sum(new[:i]) for i in range(5)]
    for bad_len in (0, 17, -3):
        last = b.last.clone()
        last[2] = bad_len
        o = torch.full_like(b.q, 7.0)
        lse = torch.full(b.q.shape[:2], 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = dict(o=o, lse=lse, err_word=err)
        if decode:
            gdn.gdn_attention_decode_paged(b.q, b.k_cache, b.v_cache, b.indices, b.indptr, last, **args)
        else:
            gdn.gdn_attention_paged(b.q, b.k_cache, b.v_cache, b.cu, b.indices, b.indptr, last, **args)
        assert int(err.item()) == (2 << 24) | 2
        for s in range(4):
            rows = slice(start[s], start[s + 1])
            if s == 2:
                assert (o[rows] == 7.0).all() and (lse[rows] == 7.0).all()
            else:
                within(o[rows], ref[0][rows], ref[2][rows], "o")
                within(lse[rows], ref[1][rows], ref[3][rows], "lse")


@pytest.mark.parametrize("decode", [False, True])
def test_page_ids_outside_the_cache_are_not_followed(decode):
    new, prefix = ([1] * 3, [100, 40, 7]) if decode else ([60, 3, 70], [100, 40, 7])
    b = Batch(new, prefix, 16, 4, 2, 64, seed=6).fill()
    ref = attention_f64(b)
    start = [sum(new[:i]) for i in range(4)]
    for bad in (-1, b.k_cache.shape[0], 1 << 30):
        indices = b.indices.clone()
        indices[int(b.indptr[1])] = bad  # the first page of sequence 1
        o = torch.zeros_like(b.q)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        if decode:
            gdn.gdn_attention_decode_paged(b.q, b.k_cache, b.v_cache, indices, b.indptr, b.last, o=o, err_word=err)
        else:
            gdn.gdn_attention_paged(b.q, b.k_cache, b.v_cache, b.cu, indices, b.indptr, b.last, o=o, err_word=err)
        assert int(err.item()) == (1 << 24) | 1
        for s in (0, 2):
            rows = slice(start[s], start[s + 1])
            within(o[rows], ref[0][rows], ref[2][rows], "o")
        kc, vc = b.k_cache.clone(), b.v_cache.clone()
        err.zero_()
        k = torch.zeros(sum(new), 2, 64, dtype=torch.bfloat16, device="cuda")
        at = int(b.indptr[2]) - 1
        indices = b.indices.clone()
        indices[at] = bad  # the last page of sequence 1, which its new tokens go to
        gdn.gdn_kv_append_paged(k, k, kc, vc, b.cu, indices, b.indptr, b.last, err_word=err)
        assert int(err.item()) == (1 << 24) | 1


# --------------------------------------------------- streams, graphs, repeats
def _step(b, f, k, v, caches, decode):
    q = gdn.gdn_kv_append_paged(k, v, *caches, b.cu, *b.table, q=b.q, frequencies=f)
    if decode:
        return gdn.gdn_attention_decode_paged(q, *caches, *b.table, return_lse=True)
    return gdn.gdn_attention_paged(q, *caches, b.cu, *b.table, return_lse=True)


@pytest.mark.parametrize("decode", [False, True])
def test_graph_replay_other_stream_and_repeats_give_the_same_bits(decode):
    new, prefix = ([1] * 5, [100, 3000, 0, 64, 777]) if decode else ([60, 300, 128, 0, 1], [100, 1300, 0, 64, 777])
    b = Batch(new, prefix, 64, 16, 2, 128, seed=11).fill(upto_prefix=True)
    f = freqs(128)
    k = torch.cat([b.k[i][p:] for i, p in enumerate(prefix)]).cuda()
    v = torch.cat([b.v[i][p:] for i, p in enumerate(prefix)]).cuda()
    caches = (b.k_cache, b.v_cache)
    first = [x.clone() for x in _step(b, f, k, v, caches, decode)]
    for _ in range(3):
        for x, y in zip(first, _step(b, f, k, v, caches, decode)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), "repeat"
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _step(b, f, k, v, caches, decode)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(first, other):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), "side stream"
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _step(b, f, k, v, caches, decode)
    for _ in range(2):
        for x in captured:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(first, captured):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), "graph"


def test_chunk_equals_decode_and_split_chunks():
    """A chunk's rows do not depend on how its tokens reached the call: the last
    token as a decode, and the chunk in two calls."""
    b = Batch([90, 33], [500, 64], 64, 8, 2, 128, seed=21).fill()
    o, lse = check_attention(b)
    last = torch.tensor([89, 122], device="cuda")
    d, dl = gdn.gdn_attention_decode_paged(b.q[last].contiguous(), b.k_cache, b.v_cache, *b.table, return_lse=True)
    ref = attention_f64(b)
    within(d, ref[0][last.cpu()], ref[2][last.cpu()], "decode of the last token")
    within(dl, ref[1][last.cpu()], ref[3][last.cpu()], "lse of the last token")


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_outputs_on_any_16_byte_boundary(decode, dim):
    """o, q, the keys and the values start 16 bytes into their allocations."""
    new, prefix = ([1, 1], [100, 700]) if decode else ([70, 5], [100, 700])
    b = Batch(new, prefix, 64, 6, 2, dim, seed=13).fill()
    want, _ = check_attention(b, decode=decode)

    def shifted(t):
        raw = torch.empty(t.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:]
        assert raw.data_ptr() % 32 == 16
        return raw.view(t.shape).copy_(t)

    o, q, k, v = shifted(b.q), shifted(b.q), shifted(b.k_cache), shifted(b.v_cache)
    if decode:
        gdn.gdn_attention_decode_paged(q, k, v, *b.table, o=o)
    else:
        gdn.gdn_attention_paged(q, k, v, b.cu, *b.table, o=o)
    assert torch.equal(o.view(I16), want.view(I16))


def test_cache_beyond_32_bit_offsets():
    """A cache of more than 2^32 elements per array: tokens in its last pages."""
    pages, ps, hkv, dim = 4200, 1024, 8, 128
    assert pages * ps * hkv * dim > 2**32
    k = torch.empty(pages, ps, hkv, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    b = Batch([40, 1], [1500, 2100], ps, 16, hkv, dim, seed=5)
    far = torch.arange(pages - 5, pages)
    b.k_cache, b.v_cache = k, v
    b.owned = [far[:2].tolist(), far[2:].tolist()]
    b.indices = far.to(torch.int32).cuda()
    for c in (k, v):
        c[-5:] = float("nan")
    b.fill()
    check_attention(b)
    d = Batch([1, 1], [1539, 2100], ps, 16, hkv, dim, seed=5)
    d.k_cache, d.v_cache, d.owned, d.indices, d.k, d.v = k, v, b.owned, b.indices, b.k, b.v
    check_attention(d, decode=True)
    f = freqs(dim)
    new_k = torch.cat([b.k[0][1500:], b.k[1][2100:]]).cuda()
    gdn.gdn_kv_append_paged(new_k, new_k, k, v, b.cu, *b.table, frequencies=f)
    page, slot = b.slots(0, range(1500, 1540))
    ref, tol = rope_f64(new_k[:40], torch.arange(1500, 1540), f.cpu())
    within(k[page, slot], ref, tol, "k cache")
    assert torch.equal(v[page, slot].view(I16), new_k[:40].view(I16))


# ------------------------------------------------------------------- binding
def test_one_new_token_each_without_cu_seqlens():
    b = Batch([1] * 5, [3, 700, 64, 0, 129], 32, 8, 2, 128, seed=31).fill()
    o, lse = check_attention(b)
    o2, lse2 = gdn.gdn_attention_paged(b.q, b.k_cache, b.v_cache, None, *b.table, return_lse=True)
    assert torch.equal(o.view(I16), o2.view(I16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("decode", [False, True])
def test_outputs_and_workspace_of_the_caller(decode):
    new, prefix = ([1, 1], [3000, 20]) if decode else ([33, 2], [3000, 20])
    b = Batch(new, prefix, 64, 8, 2, 64, seed=32, spare=0).fill()
    want, want_lse = check_attention(b, decode=decode)
    T, Hq, D = b.q.shape
    S, entries = len(new), b.indices.numel()
    if decode:
        need = gdn.gdn_attention_decode_workspace_bytes(S, Hq, 2, D, entries, 64)
        call = lambda **kw: gdn.gdn_attention_decode_paged(b.q, b.k_cache, b.v_cache, *b.table, **kw)  # noqa: E731
    else:
        need = gdn.gdn_attention_workspace_bytes(S, T, Hq, 2, D, entries, 64)
        call = lambda **kw: gdn.gdn_attention_paged(b.q, b.k_cache, b.v_cache, b.cu, *b.table, **kw)  # noqa: E731
    assert need > 0
    guard = torch.full((need + 1024,), 0x5A, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, Hq, device="cuda")
    assert call(o=o, lse=lse, workspace=guard[:need]) is o
    assert torch.equal(o.view(I16), want.view(I16)) and torch.equal(lse, want_lse)
    assert (guard[need:] == 0x5A).all()
    with pytest.raises(ValueError):
        call(workspace=guard[: need - 1])


def test_binding_refuses_what_does_not_fit():
    b = Batch([3, 4], [10, 20], 16, 4, 2, 64, seed=33).fill()
    args = dict(q=b.q, k_cache=b.k_cache, v_cache=b.v_cache, cu_seqlens=b.cu, page_indices=b.indices,
                page_indptr=b.indptr, last_page_len=b.last)
    f = gdn.gdn_rope_frequencies(64)
    k = torch.zeros(7, 2, 64, dtype=torch.bfloat16, device="cuda")

    def attend(**kw):
        return gdn.gdn_attention_paged(**{**args, **kw})

    for kw, error in [(dict(q=b.q.float()), TypeError), (dict(q=b.q[:, 0]), ValueError), (dict(q=b.q.cpu()), ValueError),
                      (dict(q=b.q.transpose(0, 1)), ValueError), (dict(k_cache=b.k_cache[:-1]), ValueError),
                      (dict(k_cache=b.k_cache.half()), TypeError), (dict(cu_seqlens=b.cu[:-1]), ValueError),
                      (dict(cu_seqlens=None), ValueError), (dict(cu_seqlens=b.cu.long()), TypeError),
                      (dict(page_indptr=b.indptr[1:]), ValueError), (dict(last_page_len=b.last.cpu()), ValueError),
                      (dict(slopes=torch.zeros(3, device="cuda")), ValueError),
                      (dict(slopes=torch.zeros(4, device="cuda", dtype=torch.float64)), TypeError),
                      (dict(full_lens=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
                      (dict(o=torch.zeros(7, 4, 64, device="cuda")), TypeError),
                      (dict(o=torch.zeros(6, 4, 64, device="cuda", dtype=torch.bfloat16)), ValueError),
                      (dict(lse=torch.zeros(4, 7, device="cuda")), ValueError),
                      (dict(window="x"), TypeError), (dict(scale="x"), TypeError),
                      (dict(err_word=torch.zeros(1, device="cuda")), TypeError)]:
        with pytest.raises(error):
            attend(**kw)
    with pytest.raises(gdn.GdnError) as e:
        attend(window=3, full_lens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert e.value.status == -2
    with pytest.raises(gdn.GdnError) as e:
        attend(scale=float("nan"))
    assert e.value.status == -1
    with pytest.raises(gdn.GdnError):
        attend(softcap=1e-38, scale=1e6)  # the scale over the cap leaves fp32
    with pytest.raises(ValueError):
        gdn.gdn_rope(b.q, f, torch.zeros(6, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_rope(b.q, None, torch.zeros(7, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_rope(b.q, gdn.gdn_rope_frequencies(128), torch.zeros(7, dtype=torch.int32, device="cuda"))
    table = (b.cu, b.indices, b.indptr, b.last)
    with pytest.raises(ValueError):
        gdn.gdn_kv_append_paged(k[:6], k, b.k_cache, b.v_cache, *table)
    with pytest.raises(ValueError):
        gdn.gdn_kv_append_paged(k, k, b.k_cache, b.v_cache, *table, q_out=b.q)
    with pytest.raises(ValueError):
        gdn.gdn_kv_append_paged(k, k, b.k_cache, b.v_cache, *table, q=b.q[:5])
    before = b.k_cache.clone()
    with pytest.raises(gdn.GdnError):
        gdn.gdn_kv_append_paged(k, k, b.k_cache, b.v_cache, *table, amplitude=float("inf"), frequencies=f)
    assert torch.equal(before.view(I16), b.k_cache.view(I16))


def test_nothing_to_do():
    """No tokens, no sequences: empty outputs, nothing touched."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = gdn.gdn_attention_paged(q, c, c, i32(0, 0), i32(1), i32(0, 1), i32(5), return_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert gdn.gdn_attention_decode_paged(q, c, c, i32(), i32(0), i32()).shape == (0, 4, 64)
    assert gdn.gdn_kv_append_paged(k, k, c, c, i32(0, 0), i32(1), i32(0, 1), i32(5), q=q).shape == (0, 4, 64)
    assert not c.any()
