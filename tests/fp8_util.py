"""The 8-bit cache's operators in 64 bits on the CPU, with the inputs of their tests.

Acceptance, derived from the arithmetic.
  - norm and rotation: one bf16 rounding, 2^-8 |y|; before it fp32: the sum of at most
    256 squares (all positive, at most 20 roundings one after the other, 2^-19 of it),
    the reciprocal root (2 units, 2^-22), four products, sines and angles (2^-19, as
    for the rotation alone): together below 2^-17 (|a| + |b|) amplitude;
  - codes: e4m3 keeps 4 significant bits, so that rounding is off by half a step, 2^-4
    of the value, and below 2^-6 of the scale by 2^-10 of it; plus the fp32 error above
    (none for values, which are not computed);
  - scales: exactly the definition's, unless the fp32 error of the group's largest
    value reaches across the border between two;
  - earlier tokens' codes, whatever is read back, slots and scales that a call does not
    own: bit for bit;
  - attention: as over a 16-bit cache (attention_util.py), on the codes' values.
"""
import math

import torch

import gated_deltanet_paged_gb300 as gdn
from attention_util import Batch, attention_f64, rope_f64, within

GROUP = 16
E4M3, E8M0, U8 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.uint8
NO_ROTATION = torch.zeros(0, dtype=torch.int64)


def norm_rope_f64(x, weight, pos, freq, *, eps=1e-6, offset=0.0, interleaved=False, amplitude=1.0):
    """(norm and rotation in fp64, tolerance before the last rounding)."""
    y = x.double().cpu()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * (offset + weight.double().cpu())
    freq = NO_ROTATION if freq is None else freq.cpu()
    z, _ = rope_f64(y, pos, freq, interleaved, False, amplitude)
    tol = y.abs()
    half = freq.numel()
    i = torch.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    both = (tol[..., ia] + tol[..., ib]) * abs(amplitude)
    tol[..., ia] = both
    tol[..., ib] = both
    return z, 2.0**-17 * tol


def least_exponent(most):
    """e of the least power of two with most <= 448 * 2^e, between -112 and 119 (fp64 tensor)."""
    m, e = torch.frexp(most)
    return torch.where(most > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -112)).clamp(-112, 119)


def e4m3(x):
    """fp64 -> the nearest e4m3 value, ties to even, beyond 448 to 448; keeps NaN and the sign of zero."""
    y = x.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)
    return torch.copysign(torch.round(y / step) * step, x)


class Batch8(Batch):
    """A paged batch on an 8-bit cache: codes of spread sizes under scales that differ from
    group to group, NaN codes in every slot that no token owns and NaN scales (0xFF) in
    every group that holds none.  `padded`: scales with strides of their own."""

    def __init__(self, new, prefix, page_size, hq, hkv, dim, *, layout="nhd", seed=0, spare=2, q_pad=0, device="cuda",
                 q_scale=1.0, padded=False, spread=3):
        super().__init__(new, prefix, page_size, hq, hkv, dim, layout=layout, seed=seed, spare=spare, q_pad=q_pad,
                         device=device, q_scale=q_scale)
        gen = torch.Generator().manual_seed(seed + 1)
        pages = self.k_cache.shape[0]
        shape = {"nhd": (2, pages, page_size, hkv, dim), "hnd": (2, pages, hkv, page_size, dim),
                 "fused": (pages, 2, page_size, hkv, dim)}[layout]
        raw = torch.full(shape, 0x7F, dtype=U8, device=device)
        k, v = (raw[:, 0], raw[:, 1]) if layout == "fused" else (raw[0], raw[1])
        self.k_cache, self.v_cache = (k.transpose(1, 2), v.transpose(1, 2)) if layout == "hnd" else (k, v)
        groups = page_size // GROUP
        wide = torch.full((2, hkv + 3, groups + 1, pages) if padded else (2, pages, groups, hkv), 0xFF, dtype=U8, device=device)
        s = wide[:, :hkv, :groups].permute(0, 3, 2, 1) if padded else wide
        self.k_scales, self.v_scales = s[0], s[1]
        self.codes = {}
        for name in "kv":
            values, codes = [], []
            for n, p in zip(new, prefix):
                c = (torch.randn(n + p, hkv, dim, generator=gen) * 100).clamp(-448, 448).to(E4M3)
                e = torch.randint(-8, -8 + spread, (-(-(n + p) // GROUP), hkv), generator=gen)
                codes.append((c, e))
                values.append((c.double() * torch.exp2(e.double()).repeat_interleave(GROUP, 0)[: n + p, :, None]))
            self.codes[name] = codes
            setattr(self, name, values)

    def fill(self, upto_prefix=False):
        for name, cache, scales in (("k", self.k_cache, self.k_scales), ("v", self.v_cache, self.v_scales)):
            for b, (n, p) in enumerate(zip(self.new, self.prefix)):
                end = p if upto_prefix else n + p
                if not end:
                    continue
                c, e = self.codes[name][b]
                page, slot = self.slots(b, range(end))
                cache[page, slot] = c[:end].view(U8).to(cache.device)
                scales[page[::GROUP], slot[::GROUP] // GROUP] = (e[: -(-end // GROUP)] + 127).to(U8).to(cache.device)
        return self

    @property
    def cache(self):
        return self.k_cache.view(E4M3), self.v_cache.view(E4M3), self.k_scales.view(E8M0), self.v_scales.view(E8M0)


def check_attention8(batch, decode=False, **opts):
    """Both outputs of one call against the definition on the codes' values."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if decode:
        o, lse = gdn.gdn_attention_decode_paged_fp8(batch.q, *batch.cache, *batch.table, return_lse=True, err_word=err, **opts)
    else:
        o, lse = gdn.gdn_attention_paged_fp8(batch.q, *batch.cache, batch.cu, *batch.table, return_lse=True, err_word=err,
                                             **opts)
    torch.cuda.synchronize()
    assert int(err.item()) == 0, "device error word %#x" % int(err.item())
    ref = attention_f64(batch, **{k: v for k, v in opts.items() if k not in ("o", "lse", "workspace")})
    within(lse, ref[1], ref[3], "lse")
    within(o, ref[0], ref[2], "o")
    return o, lse


def check_codes(name, scales, codes, y, tol, new_scale_of, before_scale, rows0):
    """One head's group after an append: y [rows, D] in fp64 with its tolerance, the group's
    scale byte and codes, and the byte before where the group has earlier tokens."""
    lo = int(least_exponent((y.abs() - tol).clamp(min=0).amax())) + 127
    hi = int(least_exponent((y.abs() + tol).amax())) + 127
    allowed = {max(x, before_scale) if rows0 else x for x in (lo, hi)}
    assert scales in allowed, "%s scale %d, expected %s" % (name, scales, allowed)
    s = 2.0 ** (scales - 127)
    value = codes.double() * s
    half = torch.maximum(2.0**-4 * y.abs(), torch.full_like(y, 2.0**-10 * s))
    off = (value - y.clamp(-448 * s, 448 * s)).abs() - half - tol
    assert off.max() <= 0, "%s off by %.3g over half a step" % (name, off.max())
    return math.log2(s)
