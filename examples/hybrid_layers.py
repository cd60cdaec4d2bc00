"""One recurrent layer and one attention layer over the same page table.

A model that mixes Gated Delta-Rule layers with softmax-attention layers keeps two
kinds of pages under one CSR table: page j of a sequence holds the recurrent state
after its last token, and the keys and values of its tokens.  This program runs a
prefill of ragged prompts and then single-token steps through one layer of each
kind, as a serving loop would:

  - the page table, the slots and the rotation frequencies are made once per step
    (or once for all) and shared by every layer;
  - an attention layer rotates its queries and keys and appends keys and values in
    one launch, then attends over the cache;
  - a step reads only device data, so that it can be captured in a CUDA graph;
  - the attention layer's cache is in 16 bits, or in 8 (``eight_bit``): then its queries
    and keys take a norm per head as well, in the same launch as the rotation and the
    append.

    python examples/hybrid_layers.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_paged_gb300 as gdn  # noqa: E402

H, K, V = 16, 128, 128          # recurrent heads
HQ, HKV, D = 16, 4, 128         # attention heads
ROTARY = 64                     # rotated dimensions of an attention head
PAGE = 64                       # tokens per page


class Layers:
    """The state of one recurrent and one attention layer, and their projections'
    stand-ins: every call draws the inputs that a model would compute."""

    def __init__(self, num_pages, seed=0, device="cuda", eight_bit=False):
        self.gen = torch.Generator(device=device).manual_seed(seed)
        self.device = device
        self.state_pool = torch.zeros(num_pages, H, V, K, device=device)
        cache = torch.zeros(num_pages, 2, PAGE, HKV, D, dtype=torch.bfloat16, device=device)
        self.k_cache, self.v_cache = cache[:, 0], cache[:, 1]
        self.eight_bit = eight_bit
        if eight_bit:
            codes = torch.zeros(num_pages, 2, PAGE, HKV, D, dtype=torch.float8_e4m3fn, device=device)
            scales = torch.zeros(2, num_pages, PAGE // 16, HKV, dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu)
            self.k_cache, self.v_cache = codes[:, 0], codes[:, 1]
            self.k_scales, self.v_scales = scales[0], scales[1]
            self.q_weight, self.k_weight = torch.ones(2, D, dtype=torch.bfloat16, device=device)
        # positions up to 4 x 8,192: slow waves are slowed by 4, fast ones keep their speed
        self.frequencies = gdn.gdn_rope_frequencies(ROTARY, 10000.0, factor=4.0, original_len=8192, device=device)

    def _normal(self, *shape):
        return torch.randn(*shape, generator=self.gen, device=self.device)

    def draw(self, tokens):
        """Inputs of both layers for `tokens` new tokens."""
        unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).bfloat16()  # noqa: E731
        recurrent = dict(q=unit(self._normal(tokens, H, K)), k=unit(self._normal(tokens, H, K)),
                         v=self._normal(tokens, H, V).bfloat16(), g=-torch.rand(tokens, H, generator=self.gen, device=self.device),
                         beta=torch.rand(tokens, H, generator=self.gen, device=self.device))
        qkv = self._normal(tokens, HQ + 2 * HKV, D).bfloat16()  # one fused projection; no copies below
        return recurrent, dict(q=qkv[:, :HQ], k=qkv[:, HQ:HQ + HKV], v=qkv[:, HQ + HKV:])

    def prefill(self, recurrent, attention, cu_seqlens, table, slots):
        """(recurrent output, attention output) of ragged prompts."""
        indices, indptr, last = table
        r = recurrent
        o_r = gdn.gdn_chunk_gated_delta_rule_paged(r["q"], r["k"], r["v"], r["g"], r["beta"], cu_seqlens,
                                                   self.state_pool, indices, indptr, PAGE, last, slots=slots)
        if self.eight_bit:
            return o_r, gdn.gdn_attention_paged_fp8(self._append8(attention, cu_seqlens, table), *self._cache8(), cu_seqlens, *table)
        q = gdn.gdn_kv_append_paged(attention["k"], attention["v"], self.k_cache, self.v_cache, cu_seqlens, *table,
                                    q=attention["q"], frequencies=self.frequencies)
        return o_r, gdn.gdn_attention_paged(q, self.k_cache, self.v_cache, cu_seqlens, *table)

    def decode(self, recurrent, attention, table, slots):
        """The same for one token of every sequence."""
        indices, indptr, last = table
        r = recurrent
        o_r = gdn.gdn_gated_delta_rule_decode_paged(r["q"], r["k"], r["v"], r["g"], r["beta"], self.state_pool,
                                                    indices, indptr, last, slots=slots)
        if self.eight_bit:
            return o_r, gdn.gdn_attention_decode_paged_fp8(self._append8(attention, None, table), *self._cache8(), *table)
        q = gdn.gdn_kv_append_paged(attention["k"], attention["v"], self.k_cache, self.v_cache, None, *table,
                                    q=attention["q"], frequencies=self.frequencies)
        return o_r, gdn.gdn_attention_decode_paged(q, self.k_cache, self.v_cache, *table)

    def _cache8(self):
        return self.k_cache, self.v_cache, self.k_scales, self.v_scales

    def _append8(self, attention, cu_seqlens, table):
        """Norm, rotation and append to the 8-bit cache; the queries."""
        return gdn.gdn_kv_append_paged_fp8(attention["k"], attention["v"], *self._cache8(), cu_seqlens, *table,
                                           q=attention["q"], q_weight=self.q_weight, k_weight=self.k_weight,
                                           frequencies=self.frequencies)


def page_table(lengths, owned, device="cuda"):
    """(page_indices, page_indptr, last_page_len) of sequences of these lengths on
    the first pages that each of them owns."""
    count = [-(-n // PAGE) for n in lengths]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    return (i32([p for pages, c in zip(owned, count) for p in pages[:c]]),
            i32([sum(count[:i]) for i in range(len(count) + 1)]),
            i32([n - (c - 1) * PAGE for n, c in zip(lengths, count)]))


def run(prompts=(300, 64, 1, 129), steps=4, seed=0, device="cuda", eight_bit=False):
    """Prefill the prompts, then decode `steps` tokens of each sequence.  Returns the
    layers, the lengths and owned pages, and every call's inputs and outputs."""
    room = [-(-(n + steps) // PAGE) for n in prompts]
    order = torch.randperm(sum(room), generator=torch.Generator().manual_seed(seed)).tolist()
    owned = [order[sum(room[:i]):sum(room[:i + 1])] for i in range(len(room))]
    layers = Layers(sum(room), seed, device, eight_bit)
    history = []

    lengths = list(prompts)
    table = page_table(lengths, owned, device)
    cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device=device)
    recurrent, attention = layers.draw(sum(lengths))
    slots = gdn.gdn_paged_prefill_slots(cu, table[1], table[0], table[2], PAGE)
    history.append((list(lengths), attention, layers.prefill(recurrent, attention, cu, table, slots)))
    for _ in range(steps):
        lengths = [n + 1 for n in lengths]
        table = page_table(lengths, owned, device)
        recurrent, attention = layers.draw(len(lengths))
        slots = gdn.gdn_paged_decode_slots(table[1], table[0], table[2])
        history.append(([1] * len(lengths), attention, layers.decode(recurrent, attention, table, slots)))
    return layers, lengths, owned, history


def main():
    for eight_bit in (False, True):
        _, lengths, _, history = run(eight_bit=eight_bit)
        torch.cuda.synchronize()
        print("attention layer on a cache in %d bits" % (8 if eight_bit else 16))
        for new, _, (o_r, o_a) in history:
            print("%s new tokens: recurrent output %s, attention output %s, finite: %s"
                  % (new, tuple(o_r.shape), tuple(o_a.shape), bool(torch.isfinite(o_r).all() and torch.isfinite(o_a).all())))
        print("sequences now hold %s tokens" % lengths)


if __name__ == "__main__":
    main()
