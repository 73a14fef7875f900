"""Sequences that share pages on the GPU: freeing, forking, reserving, compacting and copying,
against the plain reference (pages_ref), number for number."""
import random

import pytest

import pages_ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_long_quest_gb300 as kt
    return kt


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class State:
    """A page map on the device beside its reference."""

    def __init__(self, kt, table, lens, blocks, refs):
        self.kt, self.ref = kt, pages_ref.Map(table, lens, blocks, refs)
        self.table, self.lens, self.blocks, self.refs = dev(table), dev(lens), dev(blocks), dev(refs)
        self.map = kt.page_map(self.table, self.lens, self.blocks, self.refs)
        self.ws = kt.page_workspace(self.map)

    def check(self):
        assert self.lens.tolist() == self.ref.lens
        assert self.blocks.tolist() == self.ref.blocks
        assert self.refs.tolist() == self.ref.refs
        assert self.table.tolist() == self.ref.table
        want = self.kt.KT_ERR_DEVICE_CHECK if self.ref.bad else self.kt.KT_OK
        assert self.kt.kt_read_device_status(self.ws) == want
        self.ref.bad = False

    def fork(self, src, dst):
        moves = torch.full((len(src), 2), -7, dtype=torch.int32, device="cuda")
        count = dev([-1])
        self.kt.kt_fork_seqs(self.map, dev(src), dev(dst), moves, count, self.ws)
        want = self.ref.fork(src, dst)
        self.check()
        assert count.item() == len(want)
        assert moves.tolist() == [list(m) for m in want] + [[-7, -7]] * (len(src) - len(want))
        return moves, count

    def free(self, seqs):
        self.kt.kt_free_seqs(self.map, dev(seqs), self.ws)
        self.ref.free(seqs)
        self.check()

    def reserve(self, more=None):
        self.kt.kt_reserve_pages(self.map, self.ws, None if more is None else dev(more))
        self.ref.reserve(more)
        self.check()

    def compact(self, in_place):
        n = len(self.ref.refs)
        moves = torch.full((max(1, n // 2), 2), -7, dtype=torch.int32, device="cuda")
        count = dev([-1])
        new_table = torch.full_like(self.table, -9)
        new_refs = torch.full_like(self.refs, -9)
        kw = {} if in_place else dict(new_table=new_table, new_refs=new_refs)
        self.kt.kt_compact_pages(self.map, moves, count, self.ws, **kw)
        want, table, refs = self.ref.compact()
        assert count.item() == len(want)
        assert moves.tolist() == [list(m) for m in want] + \
            [[-7, -7]] * (moves.shape[0] - len(want))
        if in_place:
            self.ref.table = [[o if w is None else w for w, o in zip(row, old)]
                              for row, old in zip(table, self.ref.table)]
            self.ref.refs = refs
        else:
            assert new_table.tolist() == [[-9 if w is None else w for w in row] for row in table]
            assert new_refs.tolist() == refs
        self.check()
        return moves, count


def random_state(kt, seed, batch, width, pages, fill=0.6):
    """Sequences with random lengths over random pages, some of them shared, some reserved."""
    rng = random.Random(seed)
    order = list(range(pages))
    rng.shuffle(order)
    table = [[rng.randrange(-3, pages + 3) for _ in range(width)] for _ in range(batch)]
    lens, blocks, refs = [0] * batch, [0] * batch, [0] * pages
    for b in range(batch):
        n = rng.choice([0, 1, 127, 128, 129, rng.randrange(0, width * 128 + 1), width * 128])
        nb = min(width, pages_ref.blocks_of(n) + (rng.random() < 0.3))
        share = rng.randrange(batch)
        for j in range(nb):
            if share < b and (j + 1) * 128 <= min(lens[share], n) and rng.random() < 0.9:
                p = table[share][j]
            elif len(order) > (1 - fill) * pages:
                p = order.pop()
            else:
                nb, n = j, min(n, j * 128)
                break
            table[b][j] = p
            refs[p] += 1
        lens[b], blocks[b] = n, nb
    return State(kt, table, lens, blocks, refs), rng


SHAPES = [(1, 1, 1), (1, 3, 5), (4, 7, 40), (9, 33, 333), (70, 20, 1500), (3, 1100, 9000),
          (1030, 3, 4099), (2048, 2, 5003)]


@pytest.mark.parametrize("batch,width,pages", SHAPES)
def test_random_sequences_of_calls(kt, batch, width, pages):
    st, rng = random_state(kt, batch + width, batch, width, pages)
    st.check()
    for _ in range(12):
        what = rng.choice(["free", "fork", "fork", "reserve", "compact"])
        if what == "free":
            st.free([rng.randrange(batch) for _ in range(rng.randint(1, max(1, batch // 3)))])
        elif what == "fork":
            n = rng.randint(1, batch)
            st.fork([rng.randrange(batch) for _ in range(n)], [rng.randrange(batch) for _ in range(n)])
        elif what == "reserve":
            st.reserve(rng.choice([None, [rng.choice([0, 1, 5, 130, 300]) for _ in range(batch)]]))
        else:
            st.compact(rng.random() < 0.5)


def test_fork_reads_the_state_before_the_call(kt):
    st = State(kt, [[3, 5, 0], [0, 0, 0], [0, 0, 0], [0, 0, 0]], [200, 0, 0, 0], [2, 0, 0, 0],
               [0, 0, 0, 1, 0, 1])
    # 1 <- 0; 2 <- 1 (empty before the call); 3 <- 3; 1 again; a slot and sources out of range
    st.fork([0, 1, 3, 0], [1, 2, 3, 1])
    st.fork([-1, 9, 0], [2, 2, 77])
    st.fork([0, 0], [2, 0])  # the second one's slot holds its own source


def test_fork_without_pages(kt):
    """Whole blocks need none; of the others the first ones get what there is."""
    st = State(kt, [[0, 1], [2, 3], [0, 0], [0, 0], [0, 0], [0, 0]], [256, 130, 0, 0, 0, 0],
               [2, 2, 0, 0, 0, 0], [1, 1, 1, 1, 0])
    moves, count = st.fork([1, 1, 0, 1], [2, 3, 4, 5])
    assert count.item() == 1 and moves[0].tolist() == [3, 4]


def test_reserve_without_pages(kt):
    st = State(kt, [[0, 9, 9, 9], [1, 9, 9, 9], [2, 9, 9, 9], [9, 9, 9, 9]], [128, 100, 128, 0],
               [1, 1, 1, 0], [1, 1, 1, 0, 0, 0, 0])
    st.reserve([128 * 2, 28, 128 * 3, 1])   # 2, 0, 3 (one too many), 1 (behind it)
    st.reserve([0, 0, 0, 1])
    st.reserve([128 * 3 + 1, -1, 0, 0])     # no room in the table, a count that makes no sense
    st.reserve([0x7fffffff, 1, 1, 1])


def test_bad_maps_are_recorded(kt):
    st = State(kt, [[0, 77], [-4, 1], [0, 0]], [256, 130, 0], [2, 2, 0], [1, 1, 0, 0])
    st.fork([0], [2])
    st.compact(False)
    st.free([0, 1, 2, 2, 1])
    # pages that nobody is said to hold; lengths and counts that do not agree
    st = State(kt, [[2, 3], [0, 1], [0, 0]], [300, 100, 0], [2, 1, 0], [0, 0, 0, 0])
    st.fork([0, 1], [2, 0])
    st.compact(False)
    st.free([1])
    st = State(kt, [[2, 3], [0, 1], [0, 0]], [100, -1, 0], [3, -1, 0], [1, 1, 1, 1])
    st.fork([0, 1], [2, 2])
    st.reserve()


def test_large_pool_and_table(kt):
    """A quarter of a million pages, packed low: the free ones are far up."""
    pages, used = 262147, 250001
    refs = [1] * used + [0] * (pages - used)
    table = [list(range(b * 8000, (b + 1) * 8000)) + [0] * 192 for b in range(8)]
    table += [[0] * 8192 for _ in range(8)]
    st = State(kt, table, [8000 * 128 - 5] * 8 + [0] * 8, [8000] * 8 + [0] * 8, refs)
    st.fork(list(range(8)), list(range(8, 16)))
    st.reserve([128 * 190] * 16)
    st.free([1, 3, 5, 7, 9, 11, 13, 15])
    st.compact(True)


# ---- copying ----------------------------------------------------------------------------
def pools_of(pages, sizes, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randint(0, 256, (pages, s), dtype=torch.uint8, device="cuda", generator=gen)
            for s in sizes]


@pytest.mark.parametrize("sizes", [[4], [16], [12, 20, 4096], [4096, 4100, 8192, 4112],
                                   [32768 * 8, 32768 * 8, 32, 1024 * 8], [36] * 256])
@pytest.mark.parametrize("n", [1, 7, 40])
def test_copy(kt, sizes, n):
    pools = pools_of(101, sizes)
    order = torch.randperm(101)
    moves = dev(torch.stack([order[:n], order[n:2 * n]], 1).tolist() + [[5, 6]] * 3)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want = [p.clone() for p in pools]
    for p in want:
        p[order[n:2 * n].cuda()] = p[order[:n].cuda()]
    kt.kt_copy_pages(kt.page_pools(pools), moves, dev([n]), ws)
    for p, w in zip(pools, want):
        assert torch.equal(p, w)
    assert kt.kt_read_device_status(ws) == kt.KT_OK
    kt.kt_copy_pages(kt.page_pools(pools), moves, dev([0]), ws)
    for p, w in zip(pools, want):
        assert torch.equal(p, w)


def test_copy_of_bad_moves(kt):
    pools = pools_of(9, [64, 12])
    want = [p.clone() for p in pools]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moves = dev([[0, 1], [-1, 2], [3, 9], [100000, 4], [5, 5], [6, 7]])
    for count, copied in ((6, ((0, 1), (6, 7))), (-3, ()), (7, ((0, 1), (6, 7)))):
        for p in want:
            for a, b in copied:
                p[b] = p[a]
        kt.kt_copy_pages(kt.page_pools(pools), moves, dev([count]), ws)
        for p, w in zip(pools, want):
            assert torch.equal(p, w)
        assert kt.kt_read_device_status(ws) == kt.KT_ERR_DEVICE_CHECK


def test_copy_past_four_gigabytes(kt):
    """Offsets that pass 32 bits."""
    pages, size = 5000, 1 << 20
    pool = torch.zeros(pages, size, dtype=torch.uint8, device="cuda")
    pool[4990] = 7
    pool[10] = 9
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kt.kt_copy_pages(kt.page_pools([pool]), dev([[4990, 3], [10, 4999]]), dev([2]), ws)
    assert bool((pool[3] == 7).all()) and bool((pool[4999] == 9).all())
    assert int(pool[:3].sum()) == 0 and bool((pool[4990] == 7).all())


def test_captured_turnover(kt):
    """Free, fork, reserve and copy captured once and replayed while lengths and sources change."""
    width, pages = 6, 60
    table = [[b * 6 + j for j in range(width)] for b in range(4)] + [[0] * width for _ in range(4)]
    st = State(kt, table, [300, 128, 1, 5 * 128] + [0] * 4, [3, 1, 1, 5] + [0] * 4,
               [1 if p % 6 < [3, 1, 1, 5][p // 6] else 0 for p in range(24)] + [0] * (pages - 24))
    pools = pools_of(pages, [4096, 12])
    src, dst = dev([0, 1, 2, 3]), dev([4, 5, 6, 7])
    moves, count = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), dev([0])
    handle = kt.page_pools(pools)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        kt.kt_free_seqs(st.map, dst, st.ws)
        kt.kt_fork_seqs(st.map, src, dst, moves, count, st.ws)
        kt.kt_reserve_pages(st.map, st.ws)
        kt.kt_copy_pages(handle, moves, count, st.ws)
    rng = random.Random(5)
    for _ in range(6):
        s = [rng.randrange(4) for _ in range(4)]
        src.copy_(dev(s))
        want = [p.clone() for p in pools]
        st.ref.free([4, 5, 6, 7])
        moved = st.ref.fork(s, [4, 5, 6, 7])
        st.ref.reserve()
        for a, b in moved:
            for p in want:
                p[b] = p[a]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        st.check()
        for p, w in zip(pools, want):
            assert torch.equal(p, w)
        for b in range(4):  # one token each
            if st.ref.lens[b] < 5 * 128:
                st.ref.lens[b] += 1
        st.lens.copy_(dev(st.ref.lens))


def test_other_stream(kt):
    st, rng = random_state(kt, 11, 40, 10, 900)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        st.free([0, 1, 2])
        st.fork([5, 6, 7], [0, 1, 2])
        st.reserve()
        st.compact(True)
    kt.kt_free_seqs(st.map, dev([3]), st.ws, stream=stream)
    st.ref.free([3])
    stream.synchronize()
    st.check()
