"""A wait of an attention kernel that runs out is reported, whichever warp gives up,
and the next call on the same context is right.  The test hook has the consumers of
keys and values wait for a barrier that nothing completes, for a millisecond; the
copies that are on their way by then complete, and are waited for."""
import pytest
import torch

import gated_deltanet_paged_gb300 as gdn
from attention_util import Batch, check_attention

pytestmark = pytest.mark.gpu

TIMEOUT = 15

# An item of one block; items of a few blocks that are not cut; items that are cut.
LENGTHS = {"one block": [20], "whole items": [200, 5, 511], "cut items": [9000, 3]}


def _stalled(call):
    gdn.gdn_debug_set_wait_stall(True)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        gdn.gdn_debug_set_wait_stall(False)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_decode_wait_that_runs_out_is_reported(name, dim):
    prefix = LENGTHS[name]
    b = Batch([1] * len(prefix), prefix, 64, 8, 2, dim, seed=51).fill()
    o = torch.full_like(b.q, 7.0)
    lse = torch.full(b.q.shape[:2], 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _stalled(lambda: gdn.gdn_attention_decode_paged(b.q, b.k_cache, b.v_cache, *b.table, o=o, lse=lse, err_word=err))
    assert int(err.item()) >> 24 == TIMEOUT
    assert (o == 7.0).all() and (lse == 7.0).all()
    check_attention(b, decode=True)


# A CTA per item; items cut evenly among CTAs; equal pieces of the batch; tokens for
# one of the two tiles only, and a window that has a first block of values cleared.
CHUNKS = {"one block": ([20], [0]), "whole items": ([300, 0, 64], [0, 7, 900]), "cut items": ([40], [9000]),
          "pieces of the batch": ([2000, 700, 1], [0, 3000, 5000])}


@pytest.mark.parametrize("opts", [{}, {"softcap": 20.0}, {"window": 333}])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("name", list(CHUNKS))
def test_chunk_wait_that_runs_out_is_reported(name, dim, opts):
    b = Batch(*CHUNKS[name], 64, 8, 2, dim, seed=52).fill()
    o = torch.full_like(b.q, 7.0)
    lse = torch.full(b.q.shape[:2], 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _stalled(lambda: gdn.gdn_attention_paged(b.q, b.k_cache, b.v_cache, b.cu, *b.table, o=o, lse=lse, err_word=err,
                                             **opts))
    assert int(err.item()) >> 24 == TIMEOUT
    assert (o == 7.0).all() and (lse == 7.0).all()
    check_attention(b, **opts)
