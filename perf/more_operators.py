"""What is measured of the attention layer's 8-bit cache: norms of queries and keys with the rotation in the
same pass, the append that quantises keys and values as it writes them, reading them back, and attention of a
chunk of new tokens and of single tokens over such a cache.

The cache holds e4m3 values with a scale, a power of two, for every 16 tokens of a page and head.  Every case
below is one call that a serving step makes; `run` makes it either in plain torch operations in 32 bits or
through the package.  Sequence lengths come from a case's own `lens_seed`, tensors from `seed`.
"""
import math
import random

import torch

own = False

GROUP = 16  # tokens per scale
EPS = 1e-6


# ------------------------------------------------------------------------------------------------------
# Cases.
# ------------------------------------------------------------------------------------------------------
def _norm(name, tokens, hq, hkv, dim, rotary, interleaved, factor, offset, padded, max_pos):
    return {"name": name, "op": "norm", "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim, "rotary": rotary,
            "interleaved": interleaved, "factor": factor, "offset": offset, "padded": padded, "max_pos": max_pos}


def _paged(name, op, seqs, new, prefix, page_size, hq, hkv, dim, lens_seed, **more):
    """new, prefix: (smallest, largest, "log" or "flat")."""
    c = {"name": name, "op": op, "seqs": seqs, "new_min": new[0], "new_max": new[1], "new_spread": new[2],
         "prefix_min": prefix[0], "prefix_max": prefix[1], "prefix_spread": prefix[2], "page_size": page_size,
         "hq": hq, "hkv": hkv, "dim": dim, "lens_seed": lens_seed, "layout": "nhd"}
    if op == "append":
        c.update(rotary=dim, interleaved=False, factor=1.0, normed=True, offset=0.0)
    elif op in ("chunk", "decode"):
        c.update(softcap=0.0, window=-1, slopes=False, prefix_mask=False)
    c.update(more)
    return c


ONE = (1, 1, "flat")


def listed():
    return [
        # Queries and keys of a decode step of the long-context batch (4 sequences): latency.
        _norm("norm: 4 tokens", 4, 32, 8, 128, 128, False, 1.0, 0.0, False, 65536),
        # A long prompt where its queries and keys lie in the fused projection, half of each head rotated,
        # positions scaled by 8 for a long context, weights stored around zero.
        _norm("norm: 65,536 tokens of a fused projection", 65536, 32, 8, 128, 64, True, 8.0, 1.0, True, 262144),
        # One token for each of 256 sequences, somewhere in their groups of 16: the append of a decode step.
        _paged("append: 256 sequences by one token", "append", 256, ONE, (1, 600, "flat"), 64, 32, 8, 128, 31),
        # A prefill step of eight ragged prompts on 896-token pages, half of each head rotated, scaled.
        _paged("append: 8 ragged prompts", "append", 8, (300, 8192, "log"), (0, 2000, "flat"), 896, 32, 8, 128, 32,
               rotary=64, interleaved=True, factor=4.0, offset=1.0),
        # The last tokens of an odd batch on short pages, heads of 64, as a step that checks drafts reads them.
        _paged("read: 61 sequences, up to 100 tokens", "read", 61, (1, 100, "flat"), (0, 900, "flat"), 16, 4, 4, 64, 33),
        # Four whole sequences, on their way to a 16-bit cache.
        _paged("read: 4 sequences of 16,384", "read", 4, (16384, 16384, "flat"), (0, 0, "flat"), 1152, 8, 8, 128, 34,
               layout="hnd"),
        # The smallest chunk: two sequences of at most 101 new tokens on 64-token pages.
        _paged("chunk: 2 short prompts", "chunk", 2, (37, 100, "flat"), (0, 64, "flat"), 64, 2, 1, 128, 35),
        # A mixed serving step: 64 sequences, new tokens spread over three decades (some none), on a layer
        # with capped scores that sees 4,096 tokens.
        _paged("chunk: 64 mixed sequences, capped, windowed", "chunk", 64, (0, 8192, "log"), (0, 16384, "flat"), 896,
               16, 4, 128, 36, softcap=30.0, window=4095),
        # A prefill step of four long prompts.
        _paged("chunk: 4 prompts of 8,192", "chunk", 4, (8192, 8192, "flat"), (0, 0, "flat"), 1152, 32, 8, 128, 37),
        # The smallest decode step: two short sequences.
        _paged("decode: 2 short sequences", "decode", 2, ONE, (64, 101, "flat"), 64, 2, 1, 128, 38),
        # An odd batch on short pages, heads of 64 in groups of five, with a distance bias in a window.
        _paged("decode: 61 sequences, distance bias", "decode", 61, ONE, (1, 9000, "log"), 16, 20, 4, 64, 39,
               slopes=True, window=8191),
        # A full serving batch.
        _paged("decode: 256 sequences", "decode", 256, ONE, (1, 32767, "flat"), 1024, 32, 4, 128, 40, layout="fused"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(lo * math.exp(rng.random() * math.log((hi + 1) / lo))))


def draw(rng):
    op = rng.choice(["norm", "append", "append", "read", "chunk", "chunk", "decode", "decode"])
    dim = rng.choice([64, 128, 128])
    factor = rng.choice([1.0, 4.0, 8.0])
    offset = rng.choice([0.0, 1.0])
    seed = rng.randrange(1 << 30)
    if op == "norm":
        dim = rng.choice([64, 80, 128, 128, 256])
        rotary = rng.choice([dim, dim // 2, dim // 4, 24, 0])
        c = _norm("", _log_int(rng, 1, 65536), rng.randint(1, 32), rng.randint(1, 8), dim, rotary, rng.random() < 0.5, factor,
                  offset, rng.random() < 0.5, 262144)
        while c["tokens"] * (c["hq"] + c["hkv"]) * dim > 65536 * 40 * 128:
            c["tokens"] //= 2
        del c["name"]
        return c
    page = rng.choice([16, 48, 64, 128, 896, 1024, 1152])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if hkv * group > 40:
        group = 4
    layout = rng.choice(["nhd", "hnd", "fused"])
    if op in ("append", "read"):
        if rng.random() < 0.5:
            c = _paged("", op, _log_int(rng, 1, 256), ONE, (0, 600, "flat"), min(page, 64), hkv * group, hkv, dim, seed)
        else:
            c = _paged("", op, rng.randint(1, 8), (1, _log_int(rng, 16, 8192), "log"), (0, 2000, "flat"), page,
                       hkv * group, hkv, dim, seed)
        c.update(layout=layout)
        if op == "append":
            c.update(rotary=rng.choice([dim, dim // 2, dim // 4, 24, 0]), interleaved=rng.random() < 0.5, factor=factor,
                     normed=rng.random() < 0.7, offset=offset)
        del c["name"]
        return c
    opts = {"softcap": rng.choice([0.0, 0.0, 30.0]), "window": rng.choice([-1, -1, _log_int(rng, 32, 8191)]),
            "slopes": rng.random() < 0.25, "layout": layout}
    if opts["window"] < 0 and rng.random() < 0.25:
        opts["prefix_mask"] = True
    if op == "decode":
        c = _paged("", op, _log_int(rng, 1, 256), ONE, (0, _log_int(rng, 64, 32767), rng.choice(["flat", "log"])), page,
                   hkv * group, hkv, dim, seed, **opts)
        return _shrunk(c, "bytes", 4.5e9, "prefix_max")
    c = _paged("", op, _log_int(rng, 1, 64), (0, _log_int(rng, 8, 8192), "log"), (0, _log_int(rng, 16, 16384), "flat"),
               page, hkv * group, hkv, dim, seed, **opts)
    return _shrunk(c, "flops", 2e12, "new_max")


def _shrunk(c, what, most, field):
    """The case with `field` halved until its unmasked work is no more than `most`."""
    whole = dict(c, window=-1)
    while work(whole)[what] > most:
        whole[field] = c[field] = max(1, c[field] // 2)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------------
# Lengths and work.
# ------------------------------------------------------------------------------------------------------
def _lens(case):
    """(new, prefix) token counts per sequence; every sequence holds at least one token, and one of them a new one."""
    rng = random.Random(case["lens_seed"])

    def one(lo, hi, spread):
        if spread == "log":
            return min(hi, max(lo, int(math.exp(math.log(lo + 1) + rng.random() * math.log((hi + 1) / (lo + 1)))) - (lo == 0)))
        return rng.randint(lo, hi)

    new, prefix = [], []
    for _ in range(case["seqs"]):
        new.append(one(case["new_min"], case["new_max"], case["new_spread"]))
        p = one(case["prefix_min"], case["prefix_max"], case["prefix_spread"])
        prefix.append(max(p, 1 - new[-1]))
    if sum(new) == 0:
        new[0] = 1
    return new, prefix


def _full(case):
    """Keys per sequence that every token sees under the prefix mask."""
    new, prefix = _lens(case)
    return [p + n // 2 for n, p in zip(new, prefix)]


def work(case):
    if case["op"] == "norm":
        n = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": 4 * n * case["dim"] + 4 * case["tokens"] + 4 * case["rotary"] + 4 * case["dim"],
                "flops": n * (4 * case["dim"] + 3 * case["rotary"])}
    new, prefix = _lens(case)
    tokens, d, hq, hkv = sum(new), case["dim"], case["hq"], case["hkv"]
    table = 4 * (2 * case["seqs"] + sum(-(-(n + p) // case["page_size"]) for n, p in zip(new, prefix)))
    groups = lambda n, p: -(-(n + p) // GROUP) - p // GROUP  # noqa: E731
    if case["op"] in ("append", "read"):
        scales = 2 * hkv * sum(groups(n, p) for n, p in zip(new, prefix) if n)
        moved = 6 * tokens * d * hkv + scales + table
        if case["op"] == "read":
            return {"bytes": moved, "flops": 2 * tokens * d * hkv}
        return {"bytes": moved + 4 * tokens * d * hq,
                "flops": tokens * ((hq + hkv) * (4 * d * case["normed"] + 3 * case["rotary"]) + 4 * hkv * d)}
    pairs = keys = 0
    for n, p, f in zip(new, prefix, _full(case)):
        if n == 0:
            continue
        w = case["window"]
        f = f if case["prefix_mask"] else 0
        hi = torch.arange(p, p + n, dtype=torch.int64) + 1
        lo = (hi - 1 - w).clamp(min=0) if w >= 0 else torch.zeros_like(hi)
        pairs += int((hi.clamp(min=f) - lo).sum())
        keys += max(p + n, f) - int(lo[0])
    return {"bytes": 4 * tokens * d * hq + 4 * tokens * hq + 2 * keys * hkv * d + 2 * keys * hkv // GROUP + table,
            "flops": 4 * pairs * d * hq}


# ------------------------------------------------------------------------------------------------------
# Inputs.
# ------------------------------------------------------------------------------------------------------
def _thetas(rotary, factor):
    """Radians per position of each rotated pair.  factor > 1 stretches a context of 8,192 positions: waves
    that turn less than once in it are slowed by the factor, waves that turn 32 times keep their speed."""
    out = []
    for i in range(rotary // 2):
        t = 10000.0 ** (-2.0 * i / rotary)
        keep = min(1.0, max(0.0, (8192 * t / (2 * math.pi) - 1.0) / 31.0))
        out.append(t * keep + t / factor * (1.0 - keep))
    return out


def _frequencies(rotary, factor):
    """The same as whole multiples of 2^-64 turns (the form that a program keeps)."""
    if not rotary:
        return None
    inc = [int(math.ldexp(t / (2 * math.pi), 64)) for t in _thetas(rotary, factor)]
    return torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in inc], dtype=torch.int64, device="cuda")


def _amplitude(factor):
    return 0.1 * math.log(factor) + 1.0


def _cache(case, pages, gen):
    """e4m3 keys and values with spread sizes, and scales that differ from group to group by up to 4."""
    ps, h, d = case["page_size"], case["hkv"], case["dim"]
    shape = {"nhd": (2, pages, ps, h, d), "hnd": (2, pages, h, ps, d), "fused": (pages, 2, ps, h, d)}[case["layout"]]
    x = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i : i + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda", dtype=torch.bfloat16).mul_(100).clamp_(-448, 448))
    k, v = (x[:, 0], x[:, 1]) if case["layout"] == "fused" else (x[0], x[1])
    if case["layout"] == "hnd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    scales = torch.randint(119, 122, (2, pages, ps // GROUP, h), generator=gen, device="cuda", dtype=torch.uint8)
    return k, v, scales[0].view(torch.float8_e8m0fnu), scales[1].view(torch.float8_e8m0fnu)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": case}
    weight = lambda: (1.0 - case["offset"] + 0.2 * torch.randn(case["dim"], generator=gen, device="cuda")).bfloat16()  # noqa: E731
    if case["op"] == "norm":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        x = normal(t, hq + hkv * (2 if case["padded"] else 1), case["dim"]) * 3
        s["q"], s["k"] = x[:, :hq], x[:, hq : hq + hkv]
        s["q_weight"], s["k_weight"] = weight(), weight()
        s["positions"] = torch.randint(0, case["max_pos"], (t,), generator=gen, device="cuda", dtype=torch.int32)
        s["frequencies"] = _frequencies(case["rotary"], case["factor"])
        return s
    new, prefix = _lens(case)
    ps = case["page_size"]
    count = [-(-(n + p) // ps) for n, p in zip(new, prefix)]
    s["new"], s["prefix"], s["most_pages"], s["total"] = new, prefix, max(count), sum(new)
    s["page_indices"] = torch.randperm(sum(count), generator=gen, device="cuda").to(torch.int32)
    cum = lambda x: i32([sum(x[:i]) for i in range(len(x) + 1)])  # noqa: E731
    s["page_indptr"], s["cu_seqlens"] = cum(count), cum(new)
    s["last_page_len"] = i32([n + p - (c - 1) * ps for n, p, c in zip(new, prefix, count)])
    s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"] = _cache(case, sum(count), gen)
    if case["op"] == "read":
        return s
    s["q"] = normal(sum(new), case["hq"], case["dim"])
    if case["op"] == "append":
        s["k"], s["v"] = normal(sum(new), case["hkv"], case["dim"]), normal(sum(new), case["hkv"], case["dim"])
        s["frequencies"] = _frequencies(case["rotary"], case["factor"])
        s["q_weight"] = s["k_weight"] = None
        if case["normed"]:
            s["q_weight"], s["k_weight"] = weight(), weight()
        return s
    if case["softcap"]:
        s["q"] *= 4  # scores that the cap bends
    s["slopes"] = s["full_lens"] = None
    if case["slopes"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / case["hq"]) for h in range(case["hq"])], device="cuda")
    if case["prefix_mask"]:
        s["full_lens"] = i32(_full(case))
    return s


# ------------------------------------------------------------------------------------------------------
# One pass.
# ------------------------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import gated_deltanet_paged_gb300 as gdn

        if op == "norm":
            q, k = gdn.gdn_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["frequencies"], s["positions"],
                                        eps=EPS, weight_offset=case["offset"], interleaved=case["interleaved"],
                                        amplitude=_amplitude(case["factor"]))
            return {"q": q, "k": k}
        cache = (s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])
        table = (s["page_indices"], s["page_indptr"], s["last_page_len"])
        if op == "append":
            q = gdn.gdn_kv_append_paged_fp8(s["k"], s["v"], *cache, s["cu_seqlens"], *table, q=s["q"],
                                            q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                            weight_offset=case["offset"], frequencies=s["frequencies"],
                                            interleaved=case["interleaved"], amplitude=_amplitude(case["factor"]))
            return {"q": q, "k_cache": cache[0], "v_cache": cache[1], "k_scales": cache[2], "v_scales": cache[3]}
        if op == "read":
            k, v = gdn.gdn_kv_read_paged_fp8(*cache, s["cu_seqlens"], s["total"], *table)
            return {"k": k, "v": v}
        opts = {"softcap": case["softcap"], "window": case["window"], "slopes": s["slopes"], "full_lens": s["full_lens"],
                "return_lse": True}
        if op == "chunk":
            o, lse = gdn.gdn_attention_paged_fp8(s["q"], *cache, s["cu_seqlens"], *table, **opts)
        else:
            o, lse = gdn.gdn_attention_decode_paged_fp8(s["q"], *cache, *table, **opts)
        return {"o": o, "lse": lse}
    if op == "norm":
        return {n: _plain_norm_rope(s[n], s[n + "_weight"], s["positions"], s["frequencies"], case).to(s[n].dtype) for n in "qk"}
    if op == "append":
        return _plain_append(s, case)
    if op == "read":
        return _plain_read(s, case)
    return _plain_chunk(s, case) if op == "chunk" else _plain_decode(s, case)


def _plain_norm_rope(x, weight, positions, frequencies, case):
    """Each head over its root mean square, times offset + weight; then pair (a, b) of its rotated dimensions
    becomes (a cos - b sin, a sin + b cos).  In 32 bits."""
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * (weight.float() + case["offset"])
    r = case["rotary"]
    if not r:
        return y
    turns = (positions.long()[:, None] * frequencies) >> 32  # the top 32 bits of the angle, in 2^-32 turns
    angle = turns.float() * (2 * math.pi / 2**32)
    amplitude = _amplitude(case["factor"])
    cos, sin = (angle.cos() * amplitude)[:, None], (angle.sin() * amplitude)[:, None]
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if case["interleaved"] else (y[..., : r // 2], y[..., r // 2 : r])
    turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1 if case["interleaved"] else -2).flatten(-2)
    return torch.cat((turned, y[..., r:]), -1)


def _token_positions(s):
    """Each new token's sequence and its position there."""
    new = torch.diff(s["cu_seqlens"].long())
    pages = torch.diff(s["page_indptr"].long())
    total = (pages - 1) * s["case"]["page_size"] + s["last_page_len"]
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device="cuda"), new, output_size=s["total"])
    token = torch.arange(s["total"], device="cuda")
    return seq, token - s["cu_seqlens"].long()[seq] + (total - new)[seq], total - new, total


def _values(codes, scales):
    """What e4m3 codes [.., tokens, heads, d] stand for with the scales [.., tokens / 16, heads], in 32 bits."""
    return codes.float() * scales.float().repeat_interleave(GROUP, -2)[..., None]


def _of_pages(s, name, pages):
    """The values on these pages: [len(pages) * page_size, heads, d]."""
    codes = s[name + "_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn)
    scales = s[name + "_scales"].view(torch.uint8)[pages].view(torch.float8_e8m0fnu)
    return _values(codes, scales)


def _plain_append(s, case):
    """The scale of a group of 16 tokens is the least power of two that brings its values to 448 at most.  Where
    earlier tokens of the sequence are in the group already, it is not less than it was, and where it grows,
    their codes are rounded to it."""
    ps = case["page_size"]
    seq, pos, first, total = _token_positions(s)
    page = s["page_indices"].long()[s["page_indptr"].long()[seq] + pos // ps]
    slot = pos % ps
    p32 = pos.to(torch.int32)
    # The group in which each sequence's new tokens begin, and its slots of earlier tokens.
    start = torch.minimum(first, total - 1) // GROUP * GROUP
    e_page = s["page_indices"].long()[s["page_indptr"].long()[:-1] + start // ps][:, None]
    e_slot = start[:, None] % ps + torch.arange(GROUP, device="cuda")
    earlier = (start[:, None] + torch.arange(GROUP, device="cuda") < first[:, None]) & (torch.diff(s["cu_seqlens"]) > 0)[:, None]
    grown = (pos // GROUP * GROUP < first[seq])[:, None]
    k = _plain_norm_rope(s["k"], s["k_weight"], p32, s["frequencies"], case)
    q = _plain_norm_rope(s["q"], s["q_weight"], p32, s["frequencies"], case).to(s["q"].dtype)
    for x, name in ((k, "k"), (s["v"].float(), "v")):
        codes, scales = s[name + "_cache"].view(torch.uint8), s[name + "_scales"].view(torch.uint8)
        group = page * (ps // GROUP) + slot // GROUP
        most = torch.zeros(scales.shape[0] * scales.shape[1], x.shape[1], device="cuda")
        most.scatter_reduce_(0, group[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        m, e = torch.frexp(most)
        e = torch.where(most > 0, e - 9 + (m > 0.875), -112).clamp(-112, 119)[group]
        old = scales[page, slot // GROUP].int() - 127
        e = torch.where(grown, torch.maximum(e, old), e)
        of_group = lambda: scales[e_page[:, 0], e_slot[:, 0] // GROUP].view(torch.float8_e8m0fnu).float()  # noqa: E731
        before = of_group()
        scales[page, slot // GROUP] = (e + 127).to(torch.uint8)
        there = codes[e_page, e_slot]
        less = (before / of_group())[:, None, :, None]
        moved = (there.view(torch.float8_e4m3fn).float() * less).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[e_page, e_slot] = torch.where(earlier[..., None, None], moved, there)
        y = torch.ldexp(x, -e[..., None]).clamp(-448, 448)
        codes[page, slot] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _plain_read(s, case):
    ps = case["page_size"]
    seq, pos, _, _ = _token_positions(s)
    page = s["page_indices"].long()[s["page_indptr"].long()[seq] + pos // ps]
    slot = pos % ps
    out = {}
    for n in "kv":
        codes = s[n + "_cache"].view(torch.uint8)[page, slot].view(torch.float8_e4m3fn)
        scales = s[n + "_scales"].view(torch.uint8)[page, slot // GROUP].view(torch.float8_e8m0fnu)
        out[n] = (codes.float() * scales.float()[..., None]).bfloat16()
    return out


def _plain_scores(x, pos_q, lens, full, s, case):
    """The masked scores of products x [.., hq, n, keys]; pos_q [.., n] and lens, full [..] of its sequences."""
    x *= case["dim"] ** -0.5
    if case["softcap"]:
        x = torch.tanh_(x.div_(case["softcap"])).mul_(case["softcap"])
    key = torch.arange(x.shape[-1], device="cuda")
    back = pos_q[..., None] - key
    if s["slopes"] is not None:
        x -= s["slopes"][:, None, None] * back.abs().unsqueeze(-3)
    seen = back >= 0
    if case["window"] >= 0:
        seen &= back <= case["window"]
    if case["prefix_mask"]:
        seen |= key < full[..., None, None]
    seen &= key < lens[..., None, None]
    return x.masked_fill_(~seen.unsqueeze(-3), -math.inf)


def _plain_softmax(x):
    """exp(x) over its sum, in place, and the logarithm of that sum."""
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    return x.div_(l), (m + l.log()).squeeze(-1)


def _plain_chunk(s, case):
    """One sequence after the other: padding 64 ragged sequences to one batch would cost many times the work."""
    ps, hq, hkv, d = case["page_size"], case["hq"], case["hkv"], case["dim"]
    o, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[0], hq, device="cuda")
    t = page = 0
    for b, (n, p) in enumerate(zip(s["new"], s["prefix"])):
        length, count = n + p, -(-(n + p) // ps)
        if n:
            pages = s["page_indices"][page : page + count].long()
            k = _of_pages(s, "k", pages).reshape(-1, hkv, d)[:length].permute(1, 2, 0)
            v = _of_pages(s, "v", pages).reshape(-1, hkv, d)[:length].transpose(0, 1)
            q = s["q"][t : t + n].float().reshape(n, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
            x = (q @ k).view(hq, n, length)
            full = s["full_lens"][b] if case["prefix_mask"] else None
            x = _plain_scores(x, torch.arange(p, length, device="cuda"), torch.tensor(length, device="cuda"), full, s, case)
            x, e = _plain_softmax(x)
            y = (x.view(hkv, -1, length) @ v).view(hq, n, d)
            o[t : t + n], lse[t : t + n] = y.transpose(0, 1).to(o.dtype), e.transpose(0, 1)
        t, page = t + n, page + count
    return {"o": o, "lse": lse}


def _plain_decode(s, case):
    ps, hq, hkv, d = case["page_size"], case["hq"], case["hkv"], case["dim"]
    first, most = s["page_indptr"][:-1].long(), s["most_pages"]
    count = torch.diff(s["page_indptr"].long())
    entry = first[:, None] + torch.minimum(torch.arange(most, device="cuda"), count[:, None] - 1)
    pages = s["page_indices"].long()[entry]
    lens = (count - 1) * ps + s["last_page_len"]
    k = _of_pages(s, "k", pages).reshape(len(lens), -1, hkv, d).permute(0, 2, 3, 1)
    q = s["q"].float().view(len(lens), hkv, hq // hkv, d)
    x = (q @ k).view(len(lens), hq, 1, -1)
    del k
    x, lse = _plain_softmax(_plain_scores(x, (lens - 1)[:, None], lens, s["full_lens"], s, case))
    v = _of_pages(s, "v", pages).reshape(len(lens), -1, hkv, d).transpose(1, 2)
    o = x.view(len(lens), hkv, hq // hkv, -1) @ v
    return {"o": o.view(len(lens), hq, d).to(s["q"].dtype), "lse": lse.view(len(lens), hq)}


# ------------------------------------------------------------------------------------------------------
# The definitions in 64 bits.
# ------------------------------------------------------------------------------------------------------
def _exact_head(x, weight, pos, case):
    """The norm, then each pair as a complex number times amplitude * exp(i pos theta)."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(torch.sum(y**2, -1, keepdim=True) / case["dim"] + EPS) * (case["offset"] + weight.double())
    r = case["rotary"]
    if not r:
        return y
    theta = torch.tensor(_thetas(r, case["factor"]), dtype=torch.float64, device="cuda")
    angle = pos.double()[:, None, None] * theta
    turn = torch.polar(torch.full_like(angle, _amplitude(case["factor"])), angle)
    even = torch.arange(0, r, 2, device="cuda") if case["interleaved"] else torch.arange(r // 2, device="cuda")
    odd = even + 1 if case["interleaved"] else even + r // 2
    z = torch.complex(y[..., even], y[..., odd]) * turn
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """The nearest e4m3 value, ties to even: three bits behind the leading one, steps of 2^-9 at the least."""
    x = x.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0**-6))) - 3)
    return torch.round(x / step) * step


def _exact_append(s, case):
    ps, h, d = case["page_size"], case["hkv"], case["dim"]
    pages, starts = s["page_indices"].tolist(), s["page_indptr"].tolist()
    pos = torch.cat([torch.arange(p, p + n) for n, p in zip(s["new"], s["prefix"])]).cuda()
    out = {"q": _exact_head(s["q"], s["q_weight"], pos, case)}
    for name, rows in (("k", _exact_head(s["k"], s["k_weight"], pos, case)), ("v", s["v"].double())):
        codes = s[name + "_cache"].double().reshape(-1, h, d)
        scales = s[name + "_scales"].double().reshape(-1, h).clone()
        t = 0
        for b, (n, p) in enumerate(zip(s["new"], s["prefix"])):
            if n == 0:
                continue
            a = p // GROUP * GROUP  # from the start of the group in which the new tokens begin
            ids = torch.tensor([pages[starts[b] + i // ps] * ps + i % ps for i in range(a, p + n)], device="cuda")
            x = torch.zeros(-(-(p + n - a) // GROUP) * GROUP, h, d, dtype=torch.float64, device="cuda")
            x[p - a : p - a + n] = rows[t : t + n]
            most = x.view(-1, GROUP, h, d).abs().amax((1, 3))
            scale = torch.exp2(torch.ceil(torch.log2(most / 448)).clamp(-112, 119))
            at = ids[::GROUP] // GROUP
            if p > a:
                scale[0] = torch.maximum(scale[0], scales[at[0]])
                x[: p - a] = codes[ids[: p - a]] * scales[at[0]][:, None]
            scales[at] = scale
            codes[ids] = _exact_e4m3(x / scale.repeat_interleave(GROUP, 0)[..., None])[: len(ids)]
            t += n
        out[name + "_cache"] = codes.view(-1, ps, h, d)
        out[name + "_scales"] = scales.view(-1, ps // GROUP, h)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return {n: _exact_head(s[n], s[n + "_weight"], s["positions"], case) for n in "qk"}
    if case["op"] == "append":
        return _exact_append(s, case)
    ps, hq, hkv, d = case["page_size"], case["hq"], case["hkv"], case["dim"]
    pages = s["page_indices"].tolist()
    starts = s["page_indptr"].tolist()

    def tokens(name, b, length):
        """Keys or values of a sequence, [length, hkv, d]."""
        ids = torch.tensor(pages[starts[b] : starts[b + 1]], device="cuda")
        codes = s[name + "_cache"].view(torch.uint8).index_select(0, ids).flatten(0, 1)[:length]
        scales = s[name + "_scales"].view(torch.uint8).index_select(0, ids).flatten(0, 1)
        scales = scales.double().sub(127).exp2()[torch.arange(length, device="cuda") // GROUP]
        return codes.view(torch.float8_e4m3fn).double() * scales[..., None]

    if case["op"] == "read":
        parts = {n: [tokens(n, b, m + p)[p:] for b, (m, p) in enumerate(zip(s["new"], s["prefix"]))] for n in "kv"}
        return {n: torch.cat(x) for n, x in parts.items()}
    heads = torch.arange(hq, device="cuda") // (hq // hkv)
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, p) in enumerate(zip(s["new"], s["prefix"])):
        if n == 0:
            continue
        k, v = tokens("k", b, n + p), tokens("v", b, n + p)
        key = torch.arange(n + p, device="cuda")
        for i in range(0, n, 1024):  # queries i .. j
            j = min(n, i + 1024)
            at = torch.arange(p + i, p + j, device="cuda")
            see = key[None] <= at[:, None]
            if case["window"] >= 0:
                see = see & (key[None] >= at[:, None] - case["window"])
            if case["prefix_mask"]:
                see = see | (key[None] < int(s["full_lens"][b]))
            for h in range(hq):
                x = s["q"][t + i : t + j, h].double() @ k[:, heads[h]].T / math.sqrt(d)
                if case["softcap"]:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"][h].double() * (at[:, None] - key[None]).abs()
                x = torch.where(see, x, -math.inf)
                e = torch.logsumexp(x, -1)
                lse[t + i : t + j, h] = e
                o[t + i : t + j, h] = torch.exp(x - e[:, None]) @ v[:, heads[h]]
        t += n
    return {"o": o, "lse": lse}
