"""Attention over the 8-bit cache, on the GPU: the bits that a 16-bit cache with the same
values gives, calls on two streams at once, and a captured call without room for a copy."""
import pytest
import torch

import gated_deltanet_paged_gb300 as gdn
from fp8_util import U8, Batch8

pytestmark = pytest.mark.gpu

I16 = torch.int16


def options(name, b):
    slopes = torch.tensor([2.0 ** (-4 * (h + 1) / b.hq) for h in range(b.hq)], device="cuda")
    full = torch.tensor([p + n // 2 for n, p in zip(b.new, b.prefix)], dtype=torch.int32, device="cuda")
    return {"plain": {}, "window": {"window": 50}, "slopes": {"slopes": slopes}, "prefix": {"full_lens": full},
            "all": {"softcap": 20.0, "slopes": slopes, "window": 130}}[name]


@pytest.mark.parametrize("opts", ["plain", "window", "slopes", "prefix", "all"])
@pytest.mark.parametrize("new,prefix,page_size,hq,hkv,dim", [
    ([300, 1, 0, 90], [100, 500, 7, 0], 64, 8, 2, 128), ([700, 0, 300, 1], [100, 40, 1500, 3], 48, 6, 3, 64),
    ([1800, 0, 300, 1], [100, 40, 1500, 3], 64, 8, 2, 128), ([1, 1, 1], [40, 5000, 700], 16, 40, 1, 128)])
def test_a_chunk_has_the_bits_of_the_16_bit_cache(new, prefix, page_size, hq, hkv, dim, opts):
    """But under a cap without slopes, which has a way of its own over the 8-bit cache."""
    b = Batch8(new, prefix, page_size, hq, hkv, dim, seed=len(opts)).fill()
    opts = options(opts, b)
    kc, vc = (torch.full(b.k_cache.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    for seq, n in enumerate(x + y for x, y in zip(new, prefix)):
        page, slot = b.slots(seq, range(n))
        kc[page, slot], vc[page, slot] = b.k[seq].bfloat16().cuda(), b.v[seq].bfloat16().cuda()
    want = gdn.gdn_attention_paged(b.q, kc, vc, b.cu, *b.table, return_lse=True, **opts)
    sizes = (len(new), sum(new), hq, hkv, dim, b.indices.numel(), page_size)
    small = gdn.gdn_attention_workspace_bytes(*sizes)
    for ws in (None, torch.full((max(small, 1),), 0xFF, dtype=U8, device="cuda")[:small]):
        got = gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, *b.table, return_lse=True, workspace=ws, **opts)
        for x, y in zip(got, want):
            assert torch.equal(x.view(I16), y.view(I16))


def test_two_streams_at_once():
    """Calls with copies of their own, one behind the other on each of two streams."""
    b = [Batch8([900, 300], [100, 1500], 64, 16, 2, 128, seed=s).fill() for s in (1, 2)]
    call = [lambda x=x: gdn.gdn_attention_paged_fp8(x.q, *x.cache, x.cu, *x.table, return_lse=True) for x in b]
    want = [f() for f in call]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in b]
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call[i]())
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o.view(I16), want[i][0].view(I16)) and torch.equal(lse, want[i][1])


def test_a_captured_call_without_room_for_a_copy():
    """Where the larger workspace cannot be had during a capture either, the call does with
    what it needs, and the graph is whole."""
    b = Batch8([700, 40], [0, 300], 16, 8, 1, 64, seed=3).fill()
    indices = torch.zeros(600_000, dtype=torch.int32, device="cuda")  # a table with room for 2.4 GB of bf16 pages
    indices[: b.indices.numel()] = b.indices
    call = lambda: gdn.gdn_attention_paged_fp8(b.q, *b.cache, b.cu, indices, b.indptr, b.last)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    graph = torch.cuda.CUDAGraph()
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 30)) / total)
    try:
        with torch.cuda.graph(graph):
            got = call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    for _ in range(2):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.view(I16), want.view(I16))
