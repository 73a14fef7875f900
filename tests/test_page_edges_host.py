"""Host-only checks of page maps at their edges."""
import pytest

import block_sparse_long_quest_gb300 as kt
from test_pages_host import BIG, FAKE, by, fake_map


def test_moves_of_a_pool_of_one_page():
    """Nothing can move, so the array has no entries (an empty tensor has no address)."""
    torch = pytest.importorskip("torch")
    moves, count = torch.zeros(0, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    kt.kt_copy_pages(kt.page_pools([torch.zeros(1, 8)]), moves, count, ws, stream=1)
    for bad in ((None, count), (moves, None), (moves.long(), count), (moves, count.float())):
        with pytest.raises(kt.KtError) as e:
            kt.kt_copy_pages(kt.page_pools([torch.zeros(1, 8)]), *bad, ws, stream=1)
        assert e.value.status == kt.KT_ERR_INVALID_ARG
    small = kt.kt_page_workspace_bytes(fake_map(num_pages=1)) - 1  # (refused behind the pointers)
    for pages, want in ((1, kt.KT_ERR_WORKSPACE_TOO_SMALL), (2, kt.KT_ERR_INVALID_ARG)):
        assert kt.lib.kt_compact_pages(by(fake_map(num_pages=pages)), None, None, None, FAKE, FAKE,
                                       small, None) == want
    assert kt.lib.kt_compact_pages(by(fake_map(num_pages=1)), None, None, None, None, FAKE, BIG,
                                   None) == kt.KT_ERR_INVALID_ARG
