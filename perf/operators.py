"""What is measured of the attention layer's operators: rotary positions, the append of keys and
values to a paged cache, attention of a chunk of new tokens over that cache, and its single-token form.

A model that mixes Gated Delta-Rule layers with attention layers runs both over one CSR page table.  Every
case below is one call that such a model makes in a step; `run` makes it either in plain torch operations
in 32 bits or through the package.  Sequence lengths come from a case's own `lens_seed`, tensors from `seed`.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------------------------------------------
# Cases.
# ------------------------------------------------------------------------------------------------------
def _rope(name, tokens, heads, dim, rotary, interleaved, inverse, factor, padded, max_pos):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "dim": dim, "rotary": rotary,
            "interleaved": interleaved, "inverse": inverse, "factor": factor, "padded": padded, "max_pos": max_pos}


def _paged(name, op, seqs, new, prefix, page_size, hq, hkv, dim, lens_seed, **more):
    """new, prefix: (smallest, largest, "log" or "flat")."""
    c = {"name": name, "op": op, "seqs": seqs, "new_min": new[0], "new_max": new[1], "new_spread": new[2],
         "prefix_min": prefix[0], "prefix_max": prefix[1], "prefix_spread": prefix[2], "page_size": page_size,
         "hq": hq, "hkv": hkv, "dim": dim, "lens_seed": lens_seed, "layout": "nhd"}
    if op == "append":
        c.update(rotary=dim, interleaved=False, factor=1.0)
    else:
        c.update(softcap=0.0, window=-1, slopes=False, prefix_mask=False)
    c.update(more)
    return c


ONE = (1, 1, "flat")


def listed():
    return [
        # The queries of a decode step of the long-context batch (4 sequences, 32 heads): latency.
        _rope("rope: 4 queries", 4, 32, 128, 128, False, False, 1.0, False, 65536),
        # Queries and keys of a long prompt where they lie in the fused projection (32 + 8 of its 48 heads),
        # half of each head rotated, positions scaled by 8 for a long context.
        _rope("rope: 65,536 tokens of a fused projection", 65536, 40, 128, 64, True, False, 8.0, True, 262144),
        # One token for each of 256 sequences: the append of a decode step, queries rotated on the way.
        _paged("append: 256 sequences by one token", "append", 256, ONE, (1, 600, "flat"), 64, 32, 8, 128, 11),
        # A prefill step of eight ragged prompts on 896-token pages, half of each head rotated, scaled.
        _paged("append: 8 ragged prompts", "append", 8, (300, 8192, "log"), (0, 2000, "flat"), 896, 32, 8, 128, 12,
               rotary=64, interleaved=True, factor=4.0),
        # The smallest chunk: two sequences of at most 101 new tokens on 64-token pages.
        _paged("chunk: 2 short prompts", "chunk", 2, (37, 100, "flat"), (0, 64, "flat"), 64, 2, 1, 128, 13),
        # The paged example: 452 new tokens after 2,048 cached ones on 1,024-token pages, with a prefix
        # (such as an image's tokens) that all of its tokens see.
        _paged("chunk: 452 tokens after 2,048, prefix mask", "chunk", 1, (452, 452, "flat"), (2048, 2048, "flat"),
               1024, 16, 2, 128, 14, prefix_mask=True),
        # A mixed serving step: 64 sequences, new tokens spread over three decades (some none), on a layer
        # with capped scores that sees 4,096 tokens.
        _paged("chunk: 64 mixed sequences, capped, windowed", "chunk", 64, (0, 8192, "log"), (0, 16384, "flat"), 896,
               16, 4, 128, 15, softcap=30.0, window=4095),
        # A prefill step of four long prompts.
        _paged("chunk: 4 prompts of 8,192", "chunk", 4, (8192, 8192, "flat"), (0, 0, "flat"), 1152, 32, 8, 128, 16),
        # The smallest decode step: two short sequences.
        _paged("decode: 2 short sequences", "decode", 2, ONE, (64, 101, "flat"), 64, 2, 1, 128, 17),
        # A decode step of a few long sequences: fewer (sequence, head) pairs than SMs.
        _paged("decode: 4 long sequences", "decode", 4, ONE, (65536, 65600, "flat"), 1152, 32, 8, 128, 18, layout="hnd"),
        # An odd batch on short pages, heads of 64 in groups of five, with a distance bias in a window.
        _paged("decode: 61 sequences, distance bias", "decode", 61, ONE, (1, 9000, "log"), 16, 20, 4, 64, 19,
               slopes=True, window=8191),
        # A full serving batch.
        _paged("decode: 256 sequences", "decode", 256, ONE, (1, 32767, "flat"), 1024, 32, 4, 128, 20, layout="fused"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(lo * math.exp(rng.random() * math.log((hi + 1) / lo))))


def draw(rng):
    op = rng.choice(["rope", "append", "chunk", "chunk", "decode", "decode"])
    dim = rng.choice([64, 128, 128])
    rotary = rng.choice([dim, dim // 2, dim // 4, 24])
    factor = rng.choice([1.0, 4.0, 8.0])
    seed = rng.randrange(1 << 30)
    if op == "rope":
        c = _rope("", _log_int(rng, 1, 65536), rng.randint(1, 40), dim, rotary, rng.random() < 0.5, rng.random() < 0.3,
                  factor, rng.random() < 0.5, 262144)
        del c["name"]
        return c
    page = rng.choice([16, 40, 64, 128, 896, 1024, 1152])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if hkv * group > 40:
        group = 4
    layout = rng.choice(["nhd", "hnd", "fused"])
    if op == "append":
        if rng.random() < 0.5:
            c = _paged("", op, _log_int(rng, 1, 256), ONE, (0, 600, "flat"), min(page, 64), hkv * group, hkv, dim, seed)
        else:
            c = _paged("", op, rng.randint(1, 8), (1, _log_int(rng, 16, 8192), "log"), (0, 2000, "flat"), page,
                       hkv * group, hkv, dim, seed)
        c.update(rotary=rotary, interleaved=rng.random() < 0.5, factor=factor, layout=layout)
        del c["name"]
        return c
    opts = {"softcap": rng.choice([0.0, 0.0, 30.0]), "window": rng.choice([-1, -1, _log_int(rng, 32, 8191)]),
            "slopes": rng.random() < 0.25, "layout": layout}
    if opts["window"] < 0 and rng.random() < 0.25:
        opts["prefix_mask"] = True
    if op == "decode":
        c = _paged("", op, _log_int(rng, 1, 256), ONE, (0, _log_int(rng, 64, 32767), rng.choice(["flat", "log"])), page,
                   hkv * group, hkv, dim, seed, **opts)
        return _shrunk(c, "bytes", 9e9, "prefix_max")
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
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * case["dim"] + 4 * case["tokens"] + 4 * case["rotary"], "flops": 3 * n * case["rotary"]}
    new, prefix = _lens(case)
    tokens, d, hq, hkv = sum(new), case["dim"], case["hq"], case["hkv"]
    table = 4 * (2 * case["seqs"] + sum(-(-(n + p) // case["page_size"]) for n, p in zip(new, prefix)))
    if case["op"] == "append":
        return {"bytes": 4 * tokens * d * (hq + 2 * hkv) + table, "flops": 3 * tokens * (hq + hkv) * case["rotary"]}
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
    return {"bytes": 4 * tokens * d * hq + 4 * tokens * hq + 4 * keys * hkv * d + table, "flops": 4 * pairs * d * hq}


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
    """The same as whole multiples of 2^-64 turns (the form that a program keeps): position times
    frequency modulo 2^64 is then the angle, however large the position."""
    inc = [int(math.ldexp(t / (2 * math.pi), 64)) for t in _thetas(rotary, factor)]
    return torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in inc], dtype=torch.int64, device="cuda")


def _amplitude(factor):
    return 0.1 * math.log(factor) + 1.0


def _cache(case, pages, gen, empty):
    ps, h, d = case["page_size"], case["hkv"], case["dim"]
    shape = {"nhd": (2, pages, ps, h, d), "hnd": (2, pages, h, ps, d), "fused": (pages, 2, ps, h, d)}[case["layout"]]
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    x = x.zero_() if empty else x.normal_(generator=gen)
    k, v = (x[:, 0], x[:, 1]) if case["layout"] == "fused" else (x[0], x[1])
    return (k.transpose(1, 2), v.transpose(1, 2)) if case["layout"] == "hnd" else (k, v)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "rope":
        t, h = case["tokens"], case["heads"]
        s["x"] = normal(t, h + (8 if case["padded"] else 0), case["dim"])[:, :h]
        s["positions"] = torch.randint(0, case["max_pos"], (t,), generator=gen, device="cuda", dtype=torch.int32)
        s["frequencies"] = _frequencies(case["rotary"], case["factor"])
        return s
    new, prefix = _lens(case)
    ps = case["page_size"]
    count = [-(-(n + p) // ps) for n, p in zip(new, prefix)]
    s["new"], s["prefix"], s["most_pages"] = new, prefix, max(count)
    s["page_indices"] = torch.randperm(sum(count), generator=gen, device="cuda").to(torch.int32)
    cum = lambda x: i32([sum(x[:i]) for i in range(len(x) + 1)])  # noqa: E731
    s["page_indptr"], s["cu_seqlens"] = cum(count), cum(new)
    s["last_page_len"] = i32([n + p - (c - 1) * ps for n, p, c in zip(new, prefix, count)])
    s["k_cache"], s["v_cache"] = _cache(case, sum(count), gen, case["op"] == "append")
    s["q"] = normal(sum(new), case["hq"], case["dim"])
    if case["op"] == "append":
        s["k"], s["v"] = normal(sum(new), case["hkv"], case["dim"]), normal(sum(new), case["hkv"], case["dim"])
        s["frequencies"] = _frequencies(case["rotary"], case["factor"])
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

        if op == "rope":
            return gdn.gdn_rope(s["x"], s["frequencies"], s["positions"], interleaved=case["interleaved"],
                                inverse=case["inverse"], amplitude=_amplitude(case["factor"]))
        table = (s["page_indices"], s["page_indptr"], s["last_page_len"])
        if op == "append":
            q = gdn.gdn_kv_append_paged(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu_seqlens"], *table, q=s["q"],
                                        frequencies=s["frequencies"], interleaved=case["interleaved"],
                                        amplitude=_amplitude(case["factor"]))
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        opts = {"softcap": case["softcap"], "window": case["window"], "slopes": s["slopes"], "full_lens": s["full_lens"],
                "return_lse": True}
        if op == "chunk":
            o, lse = gdn.gdn_attention_paged(s["q"], s["k_cache"], s["v_cache"], s["cu_seqlens"], *table, **opts)
        else:
            o, lse = gdn.gdn_attention_decode_paged(s["q"], s["k_cache"], s["v_cache"], *table, **opts)
        return {"o": o, "lse": lse}
    if op == "rope":
        return _plain_rope(s["x"], s["positions"], s["frequencies"], case)
    if op == "append":
        return _plain_append(s, case)
    return _plain_chunk(s, case) if op == "chunk" else _plain_decode(s, case)


def _plain_rope(x, positions, frequencies, case):
    """Pair (a, b) of each rotated pair of dimensions becomes (a cos - b sin, a sin + b cos)."""
    r = case["rotary"]
    turns = (positions.long()[:, None] * frequencies) >> 32  # the top 32 bits of the angle, in 2^-32 turns
    angle = turns.float() * (2 * math.pi / 2**32)
    amplitude = _amplitude(case["factor"])
    cos, sin = (angle.cos() * amplitude)[:, None], (angle.sin() * amplitude)[:, None]
    if case.get("inverse"):
        sin = -sin
    y = x.float()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if case["interleaved"] else (y[..., : r // 2], y[..., r // 2 : r])
    turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1 if case["interleaved"] else -2).flatten(-2)
    return torch.cat((turned, y[..., r:]), -1).to(x.dtype)


def _token_positions(s):
    """Each new token's sequence and its position there."""
    new = torch.diff(s["cu_seqlens"].long())
    pages = torch.diff(s["page_indptr"].long())
    total = (pages - 1) * s["case"]["page_size"] + s["last_page_len"]
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device="cuda"), new, output_size=s["q"].shape[0])
    token = torch.arange(s["q"].shape[0], device="cuda")
    return seq, token - s["cu_seqlens"].long()[seq] + (total - new)[seq]


def _plain_append(s, case):
    seq, pos = _token_positions(s)
    page = s["page_indices"].long()[s["page_indptr"].long()[seq] + pos // case["page_size"]]
    slot = pos % case["page_size"]
    p32 = pos.to(torch.int32)
    s["k_cache"][page, slot] = _plain_rope(s["k"], p32, s["frequencies"], case)
    s["v_cache"][page, slot] = s["v"]
    return {"q": _plain_rope(s["q"], p32, s["frequencies"], case), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


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
            k = s["k_cache"][pages].reshape(-1, hkv, d)[:length].float().permute(1, 2, 0)
            v = s["v_cache"][pages].reshape(-1, hkv, d)[:length].float().transpose(0, 1)
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
    k = s["k_cache"][pages].reshape(len(lens), -1, hkv, d).permute(0, 2, 3, 1).float()
    q = s["q"].float().view(len(lens), hkv, hq // hkv, d)
    x = (q @ k).view(len(lens), hq, 1, -1)
    del k
    x, lse = _plain_softmax(_plain_scores(x, (lens - 1)[:, None], lens, s["full_lens"], s, case))
    v = s["v_cache"][pages].reshape(len(lens), -1, hkv, d).transpose(1, 2).float()
    o = x.view(len(lens), hkv, hq // hkv, -1) @ v
    return {"o": o.view(len(lens), hq, d).to(s["q"].dtype), "lse": lse.view(len(lens), hq)}


# ------------------------------------------------------------------------------------------------------
# The definitions in 64 bits.
# ------------------------------------------------------------------------------------------------------
def _exact_rotation(x, pos, case):
    """Each pair as a complex number times amplitude * exp(i pos theta)."""
    theta = torch.tensor(_thetas(case["rotary"], case["factor"]), dtype=torch.float64, device="cuda")
    angle = pos.double()[:, None, None] * theta * (-1.0 if case.get("inverse") else 1.0)
    turn = torch.polar(torch.full_like(angle, _amplitude(case["factor"])), angle)
    y = x.double()
    r = case["rotary"]
    even = torch.arange(0, r, 2, device="cuda") if case["interleaved"] else torch.arange(r // 2, device="cuda")
    odd = even + 1 if case["interleaved"] else even + r // 2
    z = torch.complex(y[..., even], y[..., odd]) * turn
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotation(s["x"], s["positions"], case)
    ps, hq, hkv, d = case["page_size"], case["hq"], case["hkv"], case["dim"]
    heads = torch.arange(hq, device="cuda") // (hq // hkv)
    pages = s["page_indices"].tolist()
    starts = s["page_indptr"].tolist()
    if case["op"] == "append":
        pos = torch.cat([torch.arange(p, p + n) for n, p in zip(s["new"], s["prefix"])]).cuda()
        ids = [pages[starts[b] + i // ps] * ps + i % ps
               for b, (n, p) in enumerate(zip(s["new"], s["prefix"])) for i in range(p, p + n)]
        out = {"q": _exact_rotation(s["q"], pos, case)}
        for name, rows in (("k_cache", _exact_rotation(s["k"], pos, case)), ("v_cache", s["v"].double())):
            flat = torch.zeros(len(pages) * ps, hkv, d, dtype=torch.float64, device="cuda")
            flat[torch.tensor(ids, device="cuda")] = rows
            out[name] = flat.view(len(pages), ps, hkv, d)
        return out
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    t = 0
    for b, (n, p) in enumerate(zip(s["new"], s["prefix"])):
        own_pages = torch.tensor(pages[starts[b] : starts[b + 1]], device="cuda")
        k = s["k_cache"].index_select(0, own_pages).flatten(0, 1)[: n + p]
        v = s["v_cache"].index_select(0, own_pages).flatten(0, 1)[: n + p]
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
                x = s["q"][t + i : t + j, h].double() @ k[:, heads[h]].double().T / math.sqrt(d)
                if case["softcap"]:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"][h].double() * (at[:, None] - key[None]).abs()
                x = torch.where(see, x, -math.inf)
                e = torch.logsumexp(x, -1)
                lse[t + i : t + j, h] = e
                o[t + i : t + j, h] = torch.exp(x - e[:, None]) @ v[:, heads[h]].double()
        t += n
    return {"o": o, "lse": lse}
