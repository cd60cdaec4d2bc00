"""Chunks split into chunks and single tokens, and the example's layers, against the
definition in 64 bits at its own tolerances."""
import importlib.util
import os

import pytest
import torch

import gated_deltanet_paged_gb300 as gdn
from attention_util import Batch, attention_f64, rope_f64, within
from conftest import ROOT

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(b, lengths):
    """The page table of the batch's sequences cut off at `lengths` tokens."""
    count = [-(-n // b.ps) for n in lengths]
    return (_i32([p for owned, c in zip(b.owned, count) for p in owned[:c]]),
            _i32([sum(count[:i]) for i in range(len(count) + 1)]),
            _i32([n - (c - 1) * b.ps if c else 0 for n, c in zip(lengths, count)]))


OPTIONS = {"plain": {}, "cap": dict(softcap=12.0), "window": dict(window=100), "slopes": dict(slopes=True),
           "cap slopes window": dict(softcap=12.0, slopes=True, window=300)}


# Parts of each sequence's new tokens, with ends inside a page and inside a block of
# 128 keys, at the end of either, and parts of a single token and of none.
@pytest.mark.parametrize("parts", [[(50, 1), (40, 32)], [(1, 0), (88, 33), (1, 0)], [(20, 5), (0, 27), (69, 1), (1, 0)],
                                   [(12, 33), (78, 0)]])
@pytest.mark.parametrize("name", list(OPTIONS))
@pytest.mark.parametrize("page_size,dim", [(64, 128), (48, 64)])
def test_a_chunk_in_parts(parts, name, page_size, dim):
    prefix = [500, 64]
    new = [sum(p[s] for p in parts) for s in range(2)]
    b = Batch(new, prefix, page_size, 8, 2, dim, seed=21, q_scale=2.0).fill()
    opts = dict(OPTIONS[name])
    if "slopes" in opts:
        opts["slopes"] = torch.tensor([2.0 ** -(h + 1) for h in range(8)], device="cuda")
    ref, ref_lse, tol, lse_tol = attention_f64(b, **opts)
    first = [0, new[0]]
    done = [0, 0]
    for part in parts:
        rows = [first[s] + done[s] + i for s in range(2) for i in range(part[s])]
        lengths = [prefix[s] + done[s] + part[s] for s in range(2)]
        q = b.q[rows].contiguous()
        cu = _i32([0, part[0], part[0] + part[1]])
        o, lse = gdn.gdn_attention_paged(q, b.k_cache, b.v_cache, cu, *_table(b, lengths), return_lse=True, **opts)
        within(o, ref[rows], tol[rows], "o")
        within(lse, ref_lse[rows], lse_tol[rows], "lse")
        if part == (1, 1) or part == (1, 0):
            one = [s for s in range(2) if part[s]]
            t = _table(b, [lengths[s] if s in one else 0 for s in range(2)])
            keep = torch.tensor(one, device="cuda")
            indptr = torch.cat([t[1][:1], t[1][1:][keep]])
            d, dl = gdn.gdn_attention_decode_paged(q, b.k_cache, b.v_cache, t[0], indptr.contiguous(),
                                                   t[2][keep].contiguous(), return_lse=True, **opts)
            within(d, ref[rows], tol[rows], "single tokens")
            within(dl, ref_lse[rows], lse_tol[rows], "lse of single tokens")
        done = [done[s] + part[s] for s in range(2)]
    assert done == new


def test_example_attention_over_the_keys_that_its_cache_holds():
    """Queries and keys as the kernels saw them (rounded; each checked against its
    rotation), so that nothing is allowed for but the attention's own arithmetic."""
    spec = importlib.util.spec_from_file_location("hybrid_layers", os.path.join(ROOT, "examples", "hybrid_layers.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    prompts = (300, 64, 1, 129)
    S = len(prompts)
    layers, lengths, owned, history = ex.run(prompts, steps=3, seed=4)
    freq = layers.frequencies.cpu()
    keys, values = [], []
    for s in range(S):
        page = torch.tensor([owned[s][i // ex.PAGE] for i in range(lengths[s])], device="cuda")
        slot = torch.tensor([i % ex.PAGE for i in range(lengths[s])], device="cuda")
        keys.append(layers.k_cache[page, slot].cpu())
        values.append(layers.v_cache[page, slot].cpu())
    done = [0] * S
    for new, attention, (_, o) in history:
        pos = torch.cat([torch.arange(d, d + n) for d, n in zip(done, new)]).to(torch.int32)
        q = gdn.gdn_rope(attention["q"], layers.frequencies, pos.cuda())
        ref, tol = rope_f64(attention["q"], pos, freq)
        within(q, ref, tol, "queries")
        ref, tol = rope_f64(attention["k"], pos, freq)
        k = torch.cat([x[d:d + n] for x, d, n in zip(keys, done, new)])
        within(k, ref, tol, "keys")
        b = Batch([1], [0], 16, ex.HQ, ex.HKV, ex.D, device="cpu")
        b.new, b.prefix, b.q = new, done, q
        b.k = [x[:d + n] for x, d, n in zip(keys, done, new)]
        b.v = [x[:d + n] for x, d, n in zip(values, done, new)]
        ref, _, tol, _ = attention_f64(b)
        within(o, ref, tol, "attention output")
        done = [d + n for d, n in zip(done, new)]
    assert done == lengths
