"""Table entries that name a page which nobody is said to hold: compaction records them, wherever
the page lies, and takes them over as they are."""
import pytest

import pages_ref
from test_gpu_pages import State, dev, random_state

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_long_quest_gb300 as kt
    return kt


class CountedMap(pages_ref.Map):
    """The reference, with the count of every held entry's page looked at before pages move."""

    def compact(self):
        for row, n in zip(self.table, self.blocks):
            for p in row[:min(max(n, 0), len(row))]:
                self.check(0 <= p < len(self.refs) and self.refs[p] > 0)
        return super().compact()


def counted(st):
    st.ref.__class__ = CountedMap
    return st


@pytest.mark.parametrize("in_place", [False, True])
def test_an_entry_that_names_a_hole(kt, in_place):
    """Page 3 moves to page 1, which sequence 0 still names."""
    st = counted(State(kt, [[0, 1], [3, 0]], [256, 100], [2, 1], [1, 0, 0, 1]))
    moves, count = st.compact(in_place)  # (looks at the status too)
    assert count.item() == 1 and moves[0].tolist() == [3, 1]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [0, 1, 4, 5, 6, 7, 8, 9])
def test_every_place_of_such_a_page(kt, page, in_place):
    """Pages 2, 3 and 6 are held once, page 9 twice: holes 0 and 1, behind them 4, 5, 7, 8."""
    refs = [0, 0, 1, 1, 0, 0, 1, 0, 0, 2]
    table = [[2, 3, 6], [9, 5, 5], [9, page, 5]]
    st = counted(State(kt, table, [384, 100, 256], [3, 1, 2], refs))
    st.compact(in_place)
    st = counted(State(kt, table, [384, 100, 128], [3, 1, 1], refs))  # the entry is not held
    st.compact(in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,width,pages", [(4, 7, 40), (70, 20, 1500), (3, 1100, 9000)])
def test_random_maps_with_wrong_counts(kt, batch, width, pages, in_place):
    for seed in range(6):
        st, rng = random_state(kt, seed, batch, width, pages)
        counted(st)
        if seed % 3:  # a held page is counted as free (a few, or one)
            held = sorted({p for row, n in zip(st.ref.table, st.ref.blocks) for p in row[:n]})
            for p in rng.sample(held, min(len(held), seed)):
                st.ref.refs[p] = rng.choice([0, -1])
            st.refs.copy_(dev(st.ref.refs))
        if in_place:  # negative counts stay where they are, others of free pages become 0
            st.ref.refs = [max(r, 0) for r in st.ref.refs]
            st.refs.copy_(dev(st.ref.refs))
        st.compact(in_place)


def test_the_workspace_of_an_earlier_compaction(kt):
    """What an earlier call left in the workspace (other holes) does not count."""
    st, rng = random_state(kt, 7, 9, 33, 333)
    counted(st)
    for _ in range(4):
        st.compact(True)
        live = [b for b in range(9) if st.ref.blocks[b]]
        if live:
            st.free([rng.choice(live)])
        st.reserve([rng.choice([0, 130]) for _ in range(9)])
    st.compact(False)
