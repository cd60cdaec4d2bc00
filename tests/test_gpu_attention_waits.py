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
