"""The 8-bit cache's operators as a serving loop runs them: prefill in chunks and decoding
over one table, captured and replayed, on another stream, on a cache that passes 32-bit
offsets, and with waits that run out."""
import pytest
import torch

import gated_deltanet_paged_gb300 as gdn
from attention_util import attention_f64, within
from fp8_util import E4M3, E8M0, GROUP, U8, Batch8, check_attention8

pytestmark = pytest.mark.gpu

I16 = torch.int16
TIMEOUT = 15


class Layer:
    """An attention layer with norms on an 8-bit cache; the inputs of every step are drawn."""

    def __init__(self, pages, page_size=32, hq=8, hkv=2, dim=128, seed=0):
        self.gen = torch.Generator().manual_seed(seed)
        self.ps, self.hq, self.hkv, self.dim = page_size, hq, hkv, dim
        codes = torch.full((2, pages, page_size, hkv, dim), 0x7F, dtype=U8, device="cuda")
        scales = torch.full((2, pages, page_size // GROUP, hkv), 0xFF, dtype=U8, device="cuda")
        self.cache = codes[0].view(E4M3), codes[1].view(E4M3), scales[0].view(E8M0), scales[1].view(E8M0)
        self.norm = dict(q_weight=torch.rand(dim, generator=self.gen).add(0.5).bfloat16().cuda(),
                         k_weight=torch.rand(dim, generator=self.gen).add(0.5).bfloat16().cuda())
        self.frequencies = gdn.gdn_rope_frequencies(64)

    def draw(self, tokens):
        return (torch.randn(tokens, self.hq + 2 * self.hkv, self.dim, generator=self.gen) * 2).bfloat16().cuda()

    def step(self, qkv, cu, table, err=None):
        hq, hkv = self.hq, self.hkv
        q = gdn.gdn_kv_append_paged_fp8(qkv[:, hq : hq + hkv], qkv[:, hq + hkv :], *self.cache, cu, *table, q=qkv[:, :hq],
                                        frequencies=self.frequencies, err_word=err, **self.norm)
        if cu is None:
            return q, gdn.gdn_attention_decode_paged_fp8(q, *self.cache, *table, err_word=err)
        return q, gdn.gdn_attention_paged_fp8(q, *self.cache, cu, *table, err_word=err)

    def table(self, lengths, owned):
        count = [-(-n // self.ps) for n in lengths]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return (i32([p for own, c in zip(owned, count) for p in own[:c]]), i32([sum(count[:i]) for i in range(len(count) + 1)]),
                i32([n - (c - 1) * self.ps for n, c in zip(lengths, count)]))

    def values(self, table, lengths):
        """Keys and values of every sequence, read back, in fp64."""
        cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
        k, v = gdn.gdn_kv_read_paged_fp8(*self.cache, cu, sum(lengths), *table)
        return [list(x.double().cpu().split(lengths)) for x in (k, v)]


class _Read:
    """What attention_f64 reads of a batch."""

    def __init__(self, layer, q, new, lengths, table):
        self.q, self.new, self.prefix = q, new, [n - m for n, m in zip(lengths, new)]
        self.hq, self.hkv, self.dim = layer.hq, layer.hkv, layer.dim
        self.k, self.v = layer.values(table, lengths)


@pytest.mark.parametrize("seed", [1, 2])
def test_chunked_prefill_and_decoding(seed):
    """Every step's outputs against the definition on what the cache holds then, and what it
    holds within half a step (2^-4, and once more for each growth of a group's scale) of
    what went in."""
    chunks = [[70, 1, 40], [33, 0, 100], [5, 20, 0]]
    room = [-(-(sum(x) + 20) // 32) for x in zip(*chunks)]
    layer = Layer(sum(room) + 2, seed=seed)
    order = torch.randperm(sum(room), generator=torch.Generator().manual_seed(seed)).tolist()
    owned = [order[sum(room[:i]) : sum(room[: i + 1])] for i in range(3)]
    lengths, values = [0, 0, 0], [[], [], []]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(len(chunks) + 18):
        new = chunks[step] if step < len(chunks) else [1, 1, 1]
        lengths = [n + m for n, m in zip(lengths, new)]
        table = layer.table(lengths, owned)
        cu = torch.tensor([sum(new[:i]) for i in range(4)], dtype=torch.int32, device="cuda") if step < len(chunks) else None
        qkv = layer.draw(sum(new))
        q, o = layer.step(qkv, cu, table, err)
        ref = _Read(layer, q, new, lengths, table)
        want = attention_f64(ref)
        within(o, want[0], want[2], "step %d" % step)
        t = 0
        for b, n in enumerate(new):
            values[b].append(qkv[t : t + n, layer.hq + layer.hkv :].double().cpu())
            t += n
    assert int(err.item()) == 0
    for b in range(3):
        went_in, held = torch.cat(values[b]), ref.v[b]
        groups = torch.arange(len(held)) // GROUP
        for g in range(int(groups.max()) + 1):
            x, y = went_in[groups == g], held[groups == g]
            most = x.abs().amax((0, 2), keepdim=True)
            # Sixteen roundings at most, each to a scale of at most most / 224.
            assert ((x - y).abs() <= 16 * torch.maximum(2.0**-4 * x.abs(), 2.0**-10 * most / 224)).all()


def test_captured_steps():
    """Two captured decode steps of their own lengths, replayed in turn, give the bits of the
    eager ones; each has its workspace, and both use one cache."""
    lengths = [[700, 40, 1300], [90, 16, 17]]
    layers, results = [], []
    for mode in ("eager", "captured"):
        layer = Layer(150, seed=5)
        owned = [[list(range(0, 45)), list(range(45, 50)), list(range(50, 100))], [list(range(100, 110)), [110, 111], [112, 113]]]
        steps = []
        for n, own in zip(lengths, owned):
            table = layer.table(n, own)
            cu = torch.tensor([0, n[0], n[0] + n[1], sum(n)], dtype=torch.int32, device="cuda")
            layer.step(layer.draw(sum(n)), cu, table)
            steps.append((layer.table([x + 1 for x in n], own), layer.draw(3)))
        torch.cuda.synchronize()
        out = []
        if mode == "eager":
            for table, qkv in steps:
                out.append([x.clone() for x in layer.step(qkv, None, table)])
        else:
            graphs = []
            for table, qkv in steps:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    captured = layer.step(qkv, None, table)
                graphs.append((graph, captured))
            for graph, _ in graphs + graphs[::-1]:
                graph.replay()
            torch.cuda.synchronize()
            out = [captured for _, captured in graphs]
        layers.append(layer)
        results.append(out)
    for a, b in zip(*results):
        for x, y in zip(a, b):
            assert torch.equal(x.view(I16), y.view(I16))
    for x, y in zip(layers[0].cache, layers[1].cache):
        assert torch.equal(x.view(U8), y.view(U8))


def test_captured_prefill():
    b = Batch8([90, 300, 0, 17], [40, 700, 3, 0], 64, 8, 2, 128, seed=9).fill()
    eager = gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table, softcap=20.0)
    kv = gdn.gdn_kv_read_paged_fp8(*b.cache, b.cu, 407, *b.table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table, softcap=20.0)
        kv2 = gdn.gdn_kv_read_paged_fp8(*b.cache, b.cu, 407, *b.table)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.view(I16), eager.view(I16))
    assert all(torch.equal(x.view(I16), y.view(I16)) for x, y in zip(kv, kv2))


@pytest.mark.parametrize("opts", [{}, {"softcap": 20.0}])
def test_captured_prefill_by_way_of_a_copy(opts):
    """Two captured calls that share one workspace and the copy in it, replayed in turn."""
    batches = [Batch8([1500, 700], [40, 700], 64, 8, 2, 128, seed=s).fill() for s in (9, 10)]
    n = batches[0].indices.numel()
    ws = torch.empty(gdn.gdn_attention_fp8_workspace_bytes(2, 2200, 8, 2, 128, n, 64), dtype=U8, device="cuda")
    assert ws.numel() > gdn.gdn_attention_workspace_bytes(2, 2200, 8, 2, 128, n, 64)
    call = lambda b: gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table, workspace=ws, **opts)  # noqa: E731
    eager = [call(b) for b in batches]
    graphs = []
    for b in batches:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = call(b)
        graphs.append((graph, o))
    for graph, o in graphs * 2:
        o.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for (_, o), want in zip(graphs, eager):
        assert torch.equal(o.view(I16), want.view(I16))


def test_on_another_stream():
    """Work of the caller's stream before and after the calls stays in order."""
    layer = Layer(60, seed=7)
    table = layer.table([500], [list(range(16))])
    cu = torch.tensor([0, 500], dtype=torch.int32, device="cuda")
    qkv = layer.draw(500)
    want = layer.step(qkv, cu, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        late = torch.zeros_like(qkv)
        torch.cuda._sleep(20_000_000)
        late.copy_(qkv)
        got = layer.step(late, cu, table)
        double = got[1].float() * 2
    side.synchronize()
    assert torch.equal(got[0].view(I16), want[0].view(I16)) and torch.equal(got[1].view(I16), want[1].view(I16))
    assert torch.equal(double, want[1].float() * 2)


@pytest.mark.parametrize("new,prefix", [([1, 1], [100, 700]), ([30, 200], [100, 700])])
def test_offsets_past_32_bits(new, prefix):
    """Pages that start more than 2^32 bytes into the cache, and scales as far into theirs."""
    ps, hkv, dim = 64, 2, 128
    b = Batch8(new, prefix, ps, 8, hkv, dim, seed=3).fill()
    pages = b.k_cache.shape[0]
    step = -(-(1 << 33) // pages // 4096) * 4096  # bytes between pages: the last start past 2^32
    codes = torch.zeros(2, pages, step, dtype=U8, device="cuda")
    scales = torch.zeros(2, pages, step // 2, dtype=U8, device="cuda")
    views = [codes[i, :, : ps * hkv * dim].view(pages, ps, hkv, dim) for i in (0, 1)]
    s_views = [scales[i, :, : ps // GROUP * hkv].view(pages, ps // GROUP, hkv) for i in (0, 1)]
    for x, y in zip(views + s_views, (b.k_cache, b.v_cache, b.k_scales, b.v_scales)):
        x.copy_(y)
    results = []
    for cache in ((b.k_cache, b.v_cache, b.k_scales, b.v_scales), tuple(views + s_views)):
        b.k_cache, b.v_cache, b.k_scales, b.v_scales = cache
        out = list(check_attention8(b, decode=new == [1, 1]))
        kv = gdn.gdn_kv_read_paged_fp8(*b.cache, b.cu, sum(new), *b.table)
        gdn.gdn_kv_append_paged_fp8(kv[0] * 3, kv[1] * 3, *b.cache, b.cu, *b.table)
        results.append(out + list(kv) + [x.clone() for x in cache])
    for x, y in zip(*results):
        assert torch.equal(x.contiguous().view(U8), y.contiguous().view(U8))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("opts", [{}, {"softcap": 20.0}, {"window": 333}])
def test_wait_that_runs_out_is_reported(decode, dim, opts):
    """As for the 16-bit cache: reported, nothing written, and the next call is right."""
    for new, prefix in (([1] * 3, [200, 5, 511]), ([1] * 2, [9000, 3])) if decode else (
            ([20], [0]), ([300, 0, 64], [0, 7, 900]), ([40], [9000]), ([2000, 700, 1], [0, 3000, 5000])):
        b = Batch8(new, prefix, 64, 8, 2, dim, seed=52).fill()
        o = torch.full_like(b.q, 7.0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_debug_set_wait_stall(True)
        try:
            if decode:
                gdn.gdn_attention_decode_paged_fp8(b.q, *b.cache, *b.table, o=o, err_word=err, **opts)
            else:
                gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table, o=o, err_word=err, **opts)
            torch.cuda.synchronize()
        finally:
            gdn.gdn_debug_set_wait_stall(False)
        assert int(err.item()) >> 24 == TIMEOUT
        assert (o == 7.0).all()
        check_attention8(b, decode=decode, **opts)


@pytest.mark.parametrize("decode", [False, True])
def test_all_codes(decode):
    """Subnormal codes, zeros of both signs and the largest, as keys and values."""
    new, prefix = ([1, 1], [255, 40]) if decode else ([70, 40], [200, 0])
    b = Batch8(new, prefix, 32, 4, 1, 128, seed=1)
    every = torch.arange(256, dtype=torch.int32).to(U8)
    every = torch.cat([every[:127], every[128:255]])  # no NaN
    for name in "kv":
        for i, (c, e) in enumerate(b.codes[name]):
            pick = torch.randint(0, len(every), c.shape, generator=torch.Generator().manual_seed(i + ord(name)))
            c = every[pick].view(E4M3)
            e -= 3
            b.codes[name][i] = (c, e)
            getattr(b, name)[i] = c.double() * torch.exp2(e.double()).repeat_interleave(GROUP, 0)[: len(c), :, None]
    check_attention8(b.fill(), decode=decode, scale=2.0**-9)


@pytest.mark.parametrize("decode", [False, True])
def test_a_nan_that_is_seen_shows(decode):
    """A NaN code makes NaN of the rows that see it, and of no other sequence's."""
    new, prefix = ([1, 1], [255, 40]) if decode else ([70, 40], [200, 0])
    for cache in ("k_cache", "v_cache"):
        b = Batch8(new, prefix, 32, 4, 1, 128, seed=1).fill()
        page, slot = b.slots(0, [100])
        getattr(b, cache)[page[0], slot[0], 0, 7] = 0x7F
        if decode:
            o = gdn.gdn_attention_decode_paged_fp8(b.q, *b.cache, *b.table)
        else:
            o = gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table)
        assert o[: new[0]].isnan().any(-1).all() and torch.isfinite(o[new[0] :].float()).all()


def test_queries_with_small_elements():
    """A large element beside small ones, of single tokens, whose queries go to fp16: small
    ones are kept to 2^-28 of the largest."""
    b = Batch8([1] * 3, [300, 17, 40], 32, 8, 2, 128, seed=13)
    b.q[:, :, 5] *= 2.0**12
    for i in range(3):  # keys without the large element's dimension
        c, e = b.codes["k"][i]
        c.view(U8)[..., 5] = 0
        b.k[i][..., 5] = 0
    check_attention8(b.fill(), decode=True)


def test_example_on_an_8_bit_cache():
    """The example with a recurrent and an attention layer runs on it, and its cache holds
    the values that were appended within half a step of e4m3 (2^-4, below 2^-6 of the
    scale 2^-10 of it; no group grows by more than its sixteen tokens)."""
    import importlib.util
    import os

    from conftest import ROOT

    spec = importlib.util.spec_from_file_location("hybrid_layers", os.path.join(ROOT, "examples", "hybrid_layers.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    layers, lengths, owned, history = ex.run((300, 64, 1, 129), steps=3, seed=4, eight_bit=True)
    table = ex.page_table(lengths, owned)
    cu = torch.tensor([sum(lengths[:i]) for i in range(5)], dtype=torch.int32, device="cuda")
    _, held = gdn.gdn_kv_read_paged_fp8(*layers._cache8(), cu, sum(lengths), *table)
    parts = [[] for _ in lengths]
    for new, attention, (o_r, o_a) in history:
        assert torch.isfinite(o_r).all() and torch.isfinite(o_a).all()
        for b, v in enumerate(attention["v"].split(new)):
            parts[b].append(v)
    for b, y in enumerate(held.double().split(lengths)):
        x = torch.cat(parts[b]).double()
        assert ((x - y).abs() <= 16 * (2.0**-4 * x.abs() + 2.0**-10 * x.abs().max() / 224)).all()
