"""The example that runs a recurrent and an attention layer over one page table:
its attention outputs against the definition in 64 bits, built from the keys and
values that the example drew, token by token."""
import importlib.util
import os

import pytest
import torch

from attention_util import Batch, attention_f64, rope_f64, within
from conftest import ROOT

pytestmark = pytest.mark.gpu


def _example():
    spec = importlib.util.spec_from_file_location("hybrid_layers", os.path.join(ROOT, "examples", "hybrid_layers.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_example_attention_against_its_definition():
    ex = _example()
    prompts = (300, 64, 1, 129)
    layers, lengths, owned, history = ex.run(prompts, steps=3, seed=4)
    torch.cuda.synchronize()
    freq = layers.frequencies.cpu()
    S = len(prompts)
    keys, values = [[] for _ in range(S)], [[] for _ in range(S)]
    done = [0] * S
    for new, attention, (_, o) in history:
        pos = torch.cat([torch.arange(d, d + n) for d, n in zip(done, new)])
        q, _ = rope_f64(attention["q"], pos, freq)
        k, k_tol = rope_f64(attention["k"], pos, freq)
        t = 0
        for s, n in enumerate(new):
            keys[s].append(k[t:t + n])
            values[s].append(attention["v"][t:t + n].double().cpu())
            t += n
        b = Batch([1], [0], 16, ex.HQ, ex.HKV, ex.D, device="cpu")
        b.new, b.prefix = new, done
        # the kernels attend over the rounded queries and keys
        b.q = q.bfloat16()
        b.k = [torch.cat(x).bfloat16() for x in keys]
        b.v = [torch.cat(x) for x in values]
        ref, _, tol, _ = attention_f64(b)
        # Rounding the 64-bit rotation here and the 32-bit one there can differ by one
        # bf16 step in single queries and keys: 2^-7 of a term, so at most 2^-7 S in a
        # score; S is below 2 for these heads, and a weight moves by its part of that.
        wide = max(x.abs().max() for x in b.v)
        within(o, ref, tol + 2.0**-6 * wide, "attention output")
        done = [d + n for d, n in zip(done, new)]
    assert done == lengths
    for s in range(S):
        page = torch.tensor([owned[s][i // ex.PAGE] for i in range(lengths[s])], device="cuda")
        slot = torch.tensor([i % ex.PAGE for i in range(lengths[s])], device="cuda")
        k = torch.cat(keys[s])
        within(layers.k_cache[page, slot], k, 2.0**-8 * k.abs() + 2.0**-18 * k.abs().max(), "key cache")
        assert torch.equal(layers.v_cache[page, slot].double().cpu(), torch.cat(values[s]))


def test_example_step_as_a_cuda_graph():
    """A captured decode step gives the bits of the eager one."""
    ex = _example()
    layers, lengths, owned, _ = ex.run((70, 5), steps=1, seed=9)
    lengths = [n + 1 for n in lengths]
    table = ex.page_table(lengths, owned)
    recurrent, attention = layers.draw(2)
    slots = ex.gdn.gdn_paged_decode_slots(table[1], table[0], table[2])
    state, cache = layers.state_pool.clone(), layers.k_cache.clone()
    eager = layers.decode(recurrent, attention, table, slots)
    after = layers.state_pool.clone(), layers.k_cache.clone()
    layers.state_pool.copy_(state)
    layers.k_cache.copy_(cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layers.decode(recurrent, attention, table, slots)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(eager + after, captured + (layers.state_pool, layers.k_cache)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
