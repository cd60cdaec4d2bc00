"""Definitions in 64 bits of the attention layer's operators, on the CPU, with
the inputs of their tests.

Acceptance, derived from the arithmetic and used by every test.  A bf16 value has
8 significant bits: rounding to nearest is off by at most 2^-8 relative (1 + 2^-8
lies halfway between 1 and its neighbour 1 + 2^-7); fp32 by 2^-24.
  - rotation: one bf16 rounding of the result, 2^-8 |y|, and fp32 sines, angles
    and products, together below 2^-19 (|a| + |b|) amplitude;
  - attention: the weights may be rounded to bf16 before they meet the values
    (2^-8 sum p |v|), the output once (2^-8 |o|); scores are exact products
    summed in fp32, so that a score is off by less than 2^-19 S with S the
    largest scale * sum |q_d k_d| of the row, and the weights and the output
    relative to sum p |v| by twice that; 2^-14 covers exp2, its argument and
    the tanh;
  - lse: 2^-19 S, and 2^-19 (16 + |lse|) for the sum, the logarithm and the
    options;
  - written cache slots: as the rotation (keys), bit for bit (values); every
    other slot bit for bit.
"""
import math

import torch

import gated_deltanet_paged_gb300 as gdn


def rope_f64(x, pos, freq, interleaved=False, inverse=False, amplitude=1.0):
    """(rotated x in fp64, its tolerance).  freq: int64, 2^-64 turns."""
    y = x.double().cpu().clone()
    tol = torch.zeros_like(y)
    half = freq.numel()
    f = [int(v) % (1 << 64) for v in freq.tolist()]
    ang = torch.tensor([[((int(p) * v) % (1 << 64)) / 2.0**64 * 2 * math.pi for v in f] for p in pos.tolist()],
                       dtype=torch.float64).reshape(len(pos), 1, half)
    c, s = amplitude * ang.cos(), amplitude * ang.sin() * (-1 if inverse else 1)
    i = torch.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = y[..., ia].clone(), y[..., ib].clone()
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    t = 2.0**-19 * (a.abs() + b.abs()) * abs(amplitude)
    tol[..., ia], tol[..., ib] = 2.0**-8 * y[..., ia].abs() + t, 2.0**-8 * y[..., ib].abs() + t
    return y, tol


class Batch:
    """A paged batch with NaN in every cache slot that no token owns."""

    def __init__(self, new, prefix, page_size, hq, hkv, dim, *, layout="nhd", seed=0, spare=2, q_pad=0, device="cuda",
                 q_scale=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.new, self.prefix, self.ps, self.hq, self.hkv, self.dim = new, prefix, page_size, hq, hkv, dim
        count = [-(-(n + p) // page_size) for n, p in zip(new, prefix)]
        pages = sum(count) + spare
        ids = torch.randperm(pages, generator=gen)[: sum(count)]
        self.owned, at = [], 0
        for c in count:
            self.owned.append(ids[at : at + c].tolist())
            at += c
        T = sum(new)
        normal = lambda *s: torch.randn(*s, generator=gen).bfloat16()  # noqa: E731
        cum = lambda x: torch.tensor([sum(x[:i]) for i in range(len(x) + 1)], dtype=torch.int32)  # noqa: E731
        self.cu, self.indptr, self.indices = cum(new), cum(count), ids.to(torch.int32)
        self.last = torch.tensor([n + p - (c - 1) * page_size if c else 0 for n, p, c in zip(new, prefix, count)],
                                 dtype=torch.int32)
        shape = {"nhd": (2, pages, page_size, hkv, dim), "hnd": (2, pages, hkv, page_size, dim),
                 "fused": (pages, 2, page_size, hkv, dim)}[layout]
        raw = torch.full(shape, float("nan")).bfloat16()
        raw = raw.to(device)
        k, v = (raw[:, 0], raw[:, 1]) if layout == "fused" else (raw[0], raw[1])
        self.k_cache, self.v_cache = (k.transpose(1, 2), v.transpose(1, 2)) if layout == "hnd" else (k, v)
        self.k = [normal(n + p, hkv, dim) for n, p in zip(new, prefix)]
        self.v = [normal(n + p, hkv, dim) for n, p in zip(new, prefix)]
        self.q = (normal(T, hq + q_pad, dim) * q_scale).bfloat16()[:, :hq].to(device) if T else normal(0, hq, dim).to(device)
        for name in ("cu", "indptr", "indices", "last"):
            setattr(self, name, getattr(self, name).to(device))

    def slots(self, b, positions):
        p = torch.as_tensor(positions, dtype=torch.long)
        pages = torch.tensor(self.owned[b], dtype=torch.long)
        return pages[p // self.ps].to(self.k_cache.device), (p % self.ps).to(self.k_cache.device)

    def fill(self, upto_prefix=False, window_from=None):
        """Write the cached tokens (all, or the prefix only) into the cache."""
        for b, (n, p) in enumerate(zip(self.new, self.prefix)):
            end = p if upto_prefix else n + p
            first = window_from[b] if window_from else 0
            page, slot = self.slots(b, range(first, end))
            self.k_cache[page, slot] = self.k[b][first:end].to(self.k_cache.device)
            self.v_cache[page, slot] = self.v[b][first:end].to(self.k_cache.device)
        return self

    @property
    def table(self):
        return self.indices, self.indptr, self.last


def attention_f64(batch, *, scale=0.0, softcap=0.0, window=-1, slopes=None, full_lens=None):
    """Per sequence the outputs, lse and their tolerances: o, lse, o_tol, lse_tol."""
    outs = [[], [], [], []]
    t = 0
    g = batch.hq // batch.hkv
    scale = scale if scale > 0 else batch.dim**-0.5
    for b, (n, p) in enumerate(zip(batch.new, batch.prefix)):
        if n == 0:
            continue
        q = batch.q[t : t + n].double().cpu().transpose(0, 1)
        k = batch.k[b].double().transpose(0, 1).repeat_interleave(g, 0)
        v = batch.v[b].double().transpose(0, 1).repeat_interleave(g, 0)
        x = q @ k.transpose(1, 2) * scale
        size = (q.abs() @ k.abs().transpose(1, 2) * scale)
        if softcap > 0:
            x = softcap * torch.tanh(x / softcap)
        i, j = torch.arange(p, p + n)[:, None], torch.arange(n + p)[None]
        if slopes is not None:
            x = x - slopes.double().cpu()[:, None, None] * (i - j).abs()
        see = j <= i
        if window >= 0:
            see = see & (j >= i - window)
        if full_lens is not None:
            see = see | (j < int(full_lens[b]))
        x = x.masked_fill(~see, -math.inf)
        lse = torch.logsumexp(x, -1)
        w = torch.exp(x - lse[..., None])
        o = w @ v
        S = size.masked_fill(~see, 0).amax(-1, keepdim=True)
        wide = w @ v.abs()
        outs[0].append(o.transpose(0, 1))
        outs[1].append(lse.transpose(0, 1))
        outs[2].append((2.0**-8 * (o.abs() + wide) + (2.0**-18 * S + 2.0**-14) * wide).transpose(0, 1))
        outs[3].append((2.0**-19 * (S[..., 0] + 16 + lse.abs())).transpose(0, 1))
        t += n
    return [torch.cat(x) for x in outs]


def within(got, ref, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), "%s: non-finite" % what
    over = (got - ref).abs() - tol
    assert over.numel() == 0 or over.max() <= 0, "%s: off by %.3g over its tolerance (largest error %.3g)" % (
        what, over.max(), (got - ref).abs().max())


def check_attention(batch, decode=False, poison=None, **opts):
    """Both outputs of one call against the definition."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if decode:
        o, lse = gdn.gdn_attention_decode_paged(batch.q, batch.k_cache, batch.v_cache, *batch.table, return_lse=True,
                                                err_word=err, **opts)
    else:
        o, lse = gdn.gdn_attention_paged(batch.q, batch.k_cache, batch.v_cache, batch.cu, *batch.table,
                                         return_lse=True, err_word=err, **opts)
    torch.cuda.synchronize()
    assert int(err.item()) == 0, "device error word %#x" % int(err.item())
    ref = attention_f64(batch, **opts)
    within(lse, ref[1], ref[3], "lse")
    within(o, ref[0], ref[2], "o")
    return o, lse
