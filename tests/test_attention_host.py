"""Host side of the attention layer's calls: refused arguments (nothing is
queued) and the rotation frequencies, which are computed on the host."""
import ctypes
import math

import pytest
import torch

import gated_deltanet_paged_gb300 as gdn

P, I32, I64, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class KVCache(ctypes.Structure):  # gdn_kv_cache
    _fields_ = [("k", P), ("v", P), ("num_pages", I32), ("page_size", I32), ("num_heads", I32), ("head_dim", I32),
                ("page_stride", I64), ("token_stride", I64), ("head_stride", I64)]


class PageTable(ctypes.Structure):  # gdn_page_table
    _fields_ = [("page_indices", P), ("num_entries", I32), ("page_indptr", P), ("last_page_len", P), ("num_seqs", I32)]


class AttentionOptions(ctypes.Structure):  # gdn_attention_options
    _fields_ = [("softcap", F32), ("slopes", P), ("window", I32), ("full_lens", P)]


FAKE = 0x10000  # aligned, never dereferenced: every call below ends in a host check


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, num_pages=4, page_size=16, num_heads=2, head_dim=128, page_stride=16 * 256,
             token_stride=256, head_stride=128)
    a.update(kw)
    return ctypes.byref(KVCache(*a.values()))


def table(**kw):
    a = dict(page_indices=FAKE, num_entries=400, page_indptr=FAKE, last_page_len=FAKE, num_seqs=2)
    a.update(kw)
    return ctypes.byref(PageTable(*a.values()))


def options(**kw):
    a = dict(softcap=0.0, slopes=None, window=-1, full_lens=None)
    a.update(kw)
    return ctypes.byref(AttentionOptions(*a.values()))


def rope(**kw):
    a = dict(x=FAKE, xs=256, y=FAKE + 4096, ys=256, pos=FAKE, freq=FAKE, T=3, H=2, D=128, rotary=64, inter=0, inv=0,
             amp=1.0)
    a.update(kw)
    return gdn.library().gdn_rope(*a.values(), None)


def append(**kw):
    a = dict(q=FAKE, qs=512, q_out=FAKE + 4096, k=FAKE, ks=256, v=FAKE, vs=256, cu=FAKE, T=5, Hq=4, cache=cache(),
             table=table(), freq=FAKE, rotary=128, inter=0, amp=1.0, err=None)
    a.update(kw)
    return gdn.library().gdn_kv_append_paged(*a.values(), None)


def attend(**kw):
    a = dict(q=FAKE, qs=512, o=FAKE, lse=None, cu=FAKE, T=5, Hq=4, cache=cache(), table=table(), scale=0.0,
             options=None, ws=FAKE, wsb=1 << 40, err=None)
    a.update(kw)
    return gdn.library().gdn_attention_paged(*a.values(), None)


def decode(**kw):
    a = dict(q=FAKE, qs=512, o=FAKE, lse=None, Hq=4, cache=cache(), table=table(), scale=0.0, options=None, ws=FAKE,
             wsb=1 << 40, err=None)
    a.update(kw)
    return gdn.library().gdn_attention_decode_paged(*a.values(), None)


def test_empty_calls_queue_nothing():
    assert rope(T=0) == 0
    assert append(T=0) == 0 and attend(T=0) == 0
    assert append(T=0, cu=None, table=table(num_seqs=0)) == 0
    empty = table(num_seqs=0, num_entries=0, page_indices=None, last_page_len=None)
    assert append(T=0, cu=None, table=empty) == 0 and append(T=0, cu=None, table=empty, q=None, q_out=None) == 0
    assert attend(T=0, cu=None, table=empty, q=None, o=None) == 0
    assert decode(table=empty, q=None, o=None) == 0
    assert attend(T=0, table=table(num_seqs=0)) == 0 and decode(table=table(num_seqs=0)) == 0


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(D=12), dict(D=0), dict(rotary=0), dict(rotary=63), dict(rotary=130), dict(freq=None),
    dict(pos=None), dict(x=None), dict(y=None), dict(x=FAKE + 8), dict(xs=248), dict(ys=260), dict(freq=FAKE + 4),
    dict(amp=math.inf), dict(y=FAKE, ys=512)])
def test_rope_refuses(kw):
    assert rope(**kw) == -1


PAGED = [dict(cache=None), dict(table=None), dict(cache=cache(k=None)), dict(cache=cache(v=FAKE + 8)),
         dict(cache=cache(num_pages=0)), dict(cache=cache(page_size=0)), dict(cache=cache(num_heads=0)),
         dict(cache=cache(token_stride=252)), dict(cache=cache(head_stride=64)), dict(cache=cache(page_stride=-8)),
         dict(table=table(page_indices=None)), dict(table=table(page_indptr=None)), dict(table=table(num_seqs=-1)),
         dict(table=table(last_page_len=None)), dict(table=table(num_entries=-1))]


@pytest.mark.parametrize("kw", PAGED + [
    dict(cu=None), dict(T=-1), dict(k=None), dict(v=FAKE + 2), dict(ks=248), dict(vs=257), dict(q=None),
    dict(q_out=None), dict(Hq=0), dict(Hq=-1), dict(qs=504), dict(freq=None), dict(rotary=0), dict(rotary=256),
    dict(q=FAKE, q_out=FAKE, qs=520), dict(amp=math.nan), dict(cache=cache(head_dim=100))])
def test_append_refuses(kw):
    assert append(**kw) == -1


@pytest.mark.parametrize("kw", PAGED + [
    dict(cu=None), dict(T=-1), dict(q=None), dict(q=FAKE + 8), dict(qs=504), dict(o=None), dict(o=FAKE + 2),
    dict(Hq=0), dict(Hq=5), dict(ws=None), dict(ws=FAKE + 8), dict(wsb=0), dict(options=options(softcap=math.nan)),
    dict(lse=FAKE + 2)])
def test_attention_refuses(kw):
    assert attend(**kw) == -1


@pytest.mark.parametrize("kw", PAGED + [
    dict(q=None), dict(qs=508), dict(o=None), dict(Hq=3), dict(ws=None), dict(wsb=0), dict(lse=FAKE + 2),
    dict(options=options(softcap=math.inf))])
def test_decode_refuses(kw):
    assert decode(**kw) == -1


def test_unsupported_forms():
    for call in (attend, decode):
        assert call(cache=cache(head_dim=96, head_stride=96, token_stride=192, page_stride=16 * 192)) == -2
        assert call(options=options(window=5, full_lens=FAKE)) == -2
        assert call(Hq=258, qs=258 * 128, cache=cache(num_heads=2)) == -2  # 129 query heads per key head


def test_workspace_sizes():
    lib = gdn.library()
    assert lib.gdn_attention_workspace_bytes(2, 100, 4, 2, 128, 1000, 16) > 0
    assert lib.gdn_attention_decode_workspace_bytes(2, 4, 2, 64, 1000, 16) > 0
    # a table that holds no long sequence: nothing is cut
    assert lib.gdn_attention_workspace_bytes(2, 100, 4, 2, 128, 4, 16) == 0
    assert lib.gdn_attention_decode_workspace_bytes(2, 4, 2, 64, 4, 16) == 0
    for bad in ((-1, 100, 4, 2, 128, 1000, 16), (2, -1, 4, 2, 128, 1000, 16), (2, 100, 5, 2, 128, 1000, 16),
                (2, 100, 0, 2, 128, 1000, 16), (2, 100, 4, 0, 128, 1000, 16), (2, 100, 4, 2, 96, 1000, 16),
                (2, 100, 4, 2, 128, -1, 16), (2, 100, 4, 2, 128, 1000, 0)):
        assert lib.gdn_attention_workspace_bytes(*bad) == 0
    for bad in ((-1, 4, 2, 128, 1000, 16), (2, 5, 2, 128, 1000, 16), (2, 4, 0, 128, 1000, 16), (2, 4, 2, 80, 1000, 16),
                (2, 4, 2, 128, -1, 16), (2, 4, 2, 128, 1000, 0)):
        assert lib.gdn_attention_decode_workspace_bytes(*bad) == 0


def turns(freq):
    return [(int(v) % (1 << 64)) / 2.0**64 for v in freq.tolist()]


def test_frequencies_plain_and_interpolated():
    f = turns(gdn.gdn_rope_frequencies(64, 500000.0, device="cpu"))
    g = turns(gdn.gdn_rope_frequencies(64, 500000.0, factor=4.0, device="cpu"))
    for i in range(32):
        want = 500000.0 ** (-2 * i / 64) / (2 * math.pi)
        assert abs(f[i] - want) <= 1e-14 * want + 2.0**-64
        assert abs(g[i] - want / 4) <= 1e-14 * want + 2.0**-64


def test_frequencies_blended():
    lo, hi, length, factor = 1.0, 32.0, 8192, 8.0
    f = turns(gdn.gdn_rope_frequencies(128, 10000.0, factor=factor, original_len=length, low_turns=lo, high_turns=hi,
                                       device="cpu"))
    seen = set()
    for i in range(64):
        base = 10000.0 ** (-2 * i / 128) / (2 * math.pi)
        r = length * base
        c = min(1.0, max(0.0, (r - lo) / (hi - lo)))
        seen.add(0 if c == 0 else 1 if c == 1 else 2)
        assert abs(f[i] - base * (c + (1 - c) / factor)) <= 1e-14 * base + 2.0**-64
    assert seen == {0, 1, 2}


@pytest.mark.parametrize("args", [(0, 1e4, 1, 0, 1, 32), (63, 1e4, 1, 0, 1, 32), (64, 0.5, 1, 0, 1, 32),
                                  (64, 1e4, 0.5, 0, 1, 32), (64, 1e4, 2, 100, 3, 3), (64, math.nan, 1, 0, 1, 32),
                                  (64, 1e4, math.inf, 0, 1, 32)])
def test_frequencies_refuse(args):
    out = (ctypes.c_int64 * 64)()
    assert gdn.library().gdn_rope_frequencies(*[args[0], *map(float, args[1:])], out) == -1


def test_binding_checks_tensors():
    """The binding refuses host tensors and wrong types before any call."""
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    f = torch.zeros(64, dtype=torch.int64)
    p = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_rope(x, f, p)
    with pytest.raises(TypeError):
        gdn.gdn_rope(x.float(), f, p)
    c = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gdn.gdn_attention_paged(x, c, c, p, p, p, p)
    with pytest.raises(ValueError):
        gdn.gdn_kv_append_paged(x, x, c, c, p, p, p, p)
    with pytest.raises(TypeError):
        gdn.gdn_rope([1], f, p)
    with pytest.raises(ValueError):
        gdn.gdn_attention_decode_paged(None, c, c, p, p, p)
