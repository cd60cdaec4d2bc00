"""Host side of the 8-bit cache's calls: refused arguments, with nothing queued."""
import ctypes

import pytest

import gated_deltanet_paged_gb300 as gdn
from test_attention_host import FAKE, I32, I64, F32, P, options, table


class KVCache8(ctypes.Structure):  # gdn_kv_cache_fp8
    _fields_ = [("k", P), ("v", P), ("k_scales", P), ("v_scales", P), ("num_pages", I32), ("page_size", I32),
                ("num_heads", I32), ("head_dim", I32), ("page_stride", I64), ("token_stride", I64), ("head_stride", I64),
                ("scale_page_stride", I64), ("scale_group_stride", I64), ("scale_head_stride", I64)]


class Norm(ctypes.Structure):  # gdn_qk_norm
    _fields_ = [("q_weight", P), ("k_weight", P), ("eps", F32), ("weight_offset", F32)]


def cache8(**kw):
    a = dict(k=FAKE, v=FAKE, k_scales=FAKE + 1, v_scales=FAKE + 3, num_pages=4, page_size=32, num_heads=2, head_dim=128,
             page_stride=32 * 256, token_stride=256, head_stride=128, scale_page_stride=4, scale_group_stride=2,
             scale_head_stride=1)
    a.update(kw)
    return ctypes.byref(KVCache8(*a.values()))


def norm(**kw):
    a = dict(q_weight=FAKE, k_weight=FAKE, eps=1e-6, weight_offset=0.0)
    a.update(kw)
    return ctypes.byref(Norm(*a.values()))


def norm_rope(**kw):
    a = dict(q=FAKE, qs=256, q_out=FAKE + 4096, qos=256, k=FAKE, ks=256, k_out=FAKE + 4096, kos=256, norm=norm(), pos=FAKE,
             freq=FAKE, T=3, Hq=2, Hkv=2, D=128, rotary=64, inter=0, amp=1.0)
    a.update(kw)
    return gdn.library().gdn_qk_norm_rope(*a.values(), None)


def append(**kw):
    a = dict(q=FAKE, qs=512, q_out=FAKE + 4096, k=FAKE, ks=256, v=FAKE, vs=256, cu=FAKE, T=5, Hq=4, cache=cache8(),
             table=table(), norm=norm(), freq=FAKE, rotary=128, inter=0, amp=1.0, err=None)
    a.update(kw)
    return gdn.library().gdn_kv_append_paged_fp8(*a.values(), None)


def read(**kw):
    a = dict(cache=cache8(), table=table(), cu=FAKE, T=5, k_out=FAKE, v_out=FAKE, err=None)
    a.update(kw)
    return gdn.library().gdn_kv_read_paged_fp8(*a.values(), None)


def attend(**kw):
    a = dict(q=FAKE, qs=512, o=FAKE, lse=None, cu=FAKE, T=5, Hq=4, cache=cache8(), table=table(), scale=0.0,
             options=None, ws=FAKE, wsb=1 << 40, err=None)
    a.update(kw)
    return gdn.library().gdn_attention_paged_fp8(*a.values(), None)


def decode(**kw):
    a = dict(q=FAKE, qs=512, o=FAKE, lse=None, Hq=4, cache=cache8(), table=table(), scale=0.0, options=None, ws=FAKE,
             wsb=1 << 40, err=None)
    a.update(kw)
    return gdn.library().gdn_attention_decode_paged_fp8(*a.values(), None)


NONE = table(num_seqs=0)
CALLS = {"append": append, "read": read, "attend": attend, "decode": decode}


def test_empty_calls_queue_nothing():
    assert norm_rope(T=0) == 0
    assert append(T=0) == 0 and read(T=0) == 0 and attend(T=0) == 0
    for f in (append, read, attend):
        assert f(T=0, cu=None, table=NONE) == 0
    assert decode(table=NONE) == 0


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad,status", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k_scales=None), -1), (dict(v_scales=None), -1), (dict(k=FAKE + 8), -1),
    (dict(num_pages=0), -1), (dict(page_size=0), -1), (dict(page_size=40), -2), (dict(page_size=8), -2),
    (dict(num_heads=0), -1), (dict(head_dim=72), -2), (dict(head_dim=256, token_stride=512, head_stride=256, page_stride=1 << 14), -2),
    (dict(head_dim=96), -2), (dict(page_stride=32 * 256 + 8), -1), (dict(token_stride=264), -1), (dict(head_stride=136), -1),
    (dict(token_stride=64), -1), (dict(scale_page_stride=0), -1), (dict(scale_group_stride=0), -1),
    (dict(scale_head_stride=-1), -1), (dict(num_heads=70000, head_stride=128, token_stride=128 * 70000), -2)])
def test_bad_caches(call, bad, status):
    assert CALLS[call](cache=cache8(**bad)) == status


@pytest.mark.parametrize("call", CALLS)
def test_bad_tables(call):
    f = CALLS[call]
    assert f(cache=None) == -1 and f(table=None) == -1
    for bad in (dict(page_indices=None), dict(page_indptr=None), dict(last_page_len=None), dict(num_seqs=-1), dict(num_entries=-1)):
        assert f(table=table(**bad)) == -1
    if call != "decode":
        assert f(cu=None) == -1 and f(T=-1) == -1  # five tokens, two sequences


def test_bad_norms():
    for f in (norm_rope, append):
        for bad in (dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                    dict(weight_offset=float("nan")), dict(q_weight=None), dict(q_weight=FAKE + 2), dict(k_weight=FAKE + 8)):
            assert f(norm=norm(**bad)) == -1, bad
    assert append(norm=norm(k_weight=None)) == -1
    assert norm_rope(norm=None) == -1


def test_bad_norm_rope():
    assert norm_rope(D=264, qs=528, qos=528, ks=528, kos=528, rotary=64) == -2
    for bad in (dict(q=None), dict(q_out=None), dict(q=FAKE + 8), dict(qs=255), dict(qs=100), dict(kos=128), dict(k=None),
                dict(k_out=None), dict(Hkv=0, k=FAKE, k_out=FAKE, T=3, Hq=0), dict(Hq=0), dict(Hkv=-1), dict(T=-1), dict(D=100),
                dict(rotary=63), dict(rotary=130), dict(rotary=0), dict(freq=None), dict(freq=FAKE + 4), dict(pos=None),
                dict(amp=float("inf")), dict(q_out=FAKE, qos=512), dict(k_out=FAKE, kos=512)):
        assert norm_rope(**bad) == -1, bad


def test_bad_appends():
    for bad in (dict(q=None), dict(q_out=None), dict(Hq=0), dict(Hq=-1), dict(k=None), dict(v=FAKE + 2), dict(ks=128),
                dict(vs=260), dict(rotary=130), dict(freq=None), dict(q_out=FAKE, qs=1024), dict(amp=float("nan"))):
        assert append(**bad) == -1, bad


def test_bad_reads():
    for bad in (dict(k_out=None), dict(v_out=None), dict(k_out=FAKE + 8)):
        assert read(**bad) == -1, bad


@pytest.mark.parametrize("f", [attend, decode])
def test_bad_attention(f):
    for bad in (dict(Hq=3), dict(Hq=0), dict(q=None), dict(o=None), dict(qs=500), dict(lse=FAKE + 2),
                dict(options=options(softcap=float("nan"))), dict(scale=float("nan"))):
        assert f(**bad) == -1, bad
    assert f(Hq=2 * 129, qs=2 * 129 * 128) == -2
    assert f(options=options(window=3, full_lens=FAKE)) == -2
    big = table(num_entries=100000)
    assert f(table=big, ws=None) == -1 and f(table=big, wsb=16) == -1 and f(table=big, ws=FAKE + 8) == -1


def test_workspace_sizes():
    f, least = gdn.gdn_attention_fp8_workspace_bytes, gdn.gdn_attention_workspace_bytes
    few = (4, 8191 // 4, 8, 2, 128, 100, 64)       # 2,047 x 4 rows, 4 sequences
    assert f(*few) == least(*few)
    many = (4, 2048, 8, 2, 128, 100, 64)           # 2,048 rows each
    assert f(*many) >= least(*many) + 100 * 64 * 2 * 128 * 2 * 2 + 4 * 100
    short = (1, 2048, 1, 1, 64, 16, 64)            # nothing is cut: the copy alone
    assert least(*short) == 0 and f(*short) >= 16 * 64 * 64 * 2 * 2
    huge = (1, 1 << 20, 8, 8, 128, 1 << 20, 64)    # no copy of more than 4 GiB
    assert f(*huge) == least(*huge)
    for bad in ((-1, 2048, 8, 2, 128, 100, 64), (4, 2048, 3, 2, 128, 100, 64), (4, 2048, 8, 2, 96, 100, 64), (4, 2048, 8, 2, 128, 100, 0)):
        assert f(*bad) == 0
