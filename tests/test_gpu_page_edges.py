"""Page maps at their edges on the GPU, against the plain reference."""
import pytest

import pages_ref
from test_gpu_pages import State, dev, pools_of

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_long_quest_gb300 as kt
    return kt


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("held", [False, True])
def test_a_pool_of_one_page(kt, held, in_place):
    """moves has num_pages / 2 = 0 entries."""
    st = State(kt, [[0]], [100 * held], [1 * held], [1 * held])
    moves = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    count = dev([-1])
    new_table, new_refs = dev([[-9]]), dev([-9])
    kw = {} if in_place else dict(new_table=new_table, new_refs=new_refs)
    kt.kt_compact_pages(st.map, moves, count, st.ws, **kw)
    assert count.item() == 0
    if not in_place:
        assert new_table.tolist() == [[0 if held else -9]] and new_refs.tolist() == [int(held)]
    pools = pools_of(1, [64, 12])
    want = [p.clone() for p in pools]
    kt.kt_copy_pages(kt.page_pools(pools), moves, count, st.ws)
    for p, w in zip(pools, want):
        assert torch.equal(p, w)
    st.check()
    assert pages_ref.Map([[0]], [0], [0], [int(held)]).compact()[0] == []


class CheckedMap(pages_ref.Map):
    """The reference, with lengths beyond the pages that a sequence holds recorded too."""

    def reserve(self, more=None):
        more = [1] * len(self.lens) if more is None else list(more)
        for b, (n, have) in enumerate(zip(self.lens, self.blocks)):
            if more[b] != 0 and not self.check(n <= 128 * have):
                more[b] = 0
        super().reserve(more)


def test_reserve_for_a_length_beyond_its_pages(kt):
    """Tokens that no page of the sequence holds (appended without a page) do not get one later."""
    table = [[0, 9, 9, 9], [1, 2, 9, 9], [9, 9, 9, 9], [3, 9, 9, 9], [9, 9, 9, 9]]
    st = State(kt, table, [129, 256, 1, 128, 0], [1, 2, 0, 1, 0], [1, 1, 1, 1] + [0] * 8)
    st.ref.__class__ = CheckedMap
    st.reserve()
    assert st.blocks.tolist() == [1, 3, 0, 2, 1]
    st.reserve([0, 1, 0, 300, 0])  # who asks for none is not looked at
    st.reserve([-1, 0, 5, 0, 0])
