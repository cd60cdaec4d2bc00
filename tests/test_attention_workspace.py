"""When a chunk call may do without a workspace: where no sequence can be long, also
beside sequences that own no page."""
import pytest

import gated_deltanet_paged_gb300 as gdn


def need(seqs, entries, page_size):
    return gdn.gdn_attention_workspace_bytes(seqs, 16, 32, 8, 128, entries, page_size)


@pytest.mark.parametrize("seqs,entries,page_size", [
    (129, 128, 1024),   # one sequence of 131,072 tokens beside 128 without pages
    (129, 129, 1024),   # and with a page more: as many entries as sequences
    (61, 47, 64),       # one of 3,000 beside 60
    (500, 300, 16)])
def test_long_sequences_beside_ones_without_pages_can_be_cut(seqs, entries, page_size):
    assert need(seqs, entries, page_size) > 0


@pytest.mark.parametrize("seqs,entries,page_size", [(1, 1, 1024), (16, 16, 128), (4, 4, 1024), (2, 6, 64),
                                                    (0, 0, 64)])
def test_short_batches_need_no_workspace(seqs, entries, page_size):
    assert need(seqs, entries, page_size) == 0
