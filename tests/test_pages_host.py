"""Host-only checks of the calls on shared pages: every refusal is made before the device is
touched, and the reference keeps the map's invariants."""
import ctypes
import random

import pytest

import block_sparse_long_quest_gb300 as kt
import pages_ref

FAKE, FAR, FAR2, FAR3 = 0x100000, 0x10000000, 0x20000000, 0x30000000  # never dereferenced
BIG = 1 << 40


def fake_map(**kw):
    m = kt.PageMap(FAKE, FAKE, FAKE, FAR3, 4, 128, 16, 100)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


def by(x):
    return ctypes.byref(x) if x is not None else None


CALLS = {
    "free": lambda m, ws=FAKE, n=BIG: kt.lib.kt_free_seqs(by(m), FAKE, 2, ws, n, None),
    "fork": lambda m, ws=FAKE, n=BIG: kt.lib.kt_fork_seqs(by(m), FAKE, FAKE, 2, FAKE, FAKE, ws, n,
                                                          None),
    "reserve": lambda m, ws=FAKE, n=BIG: kt.lib.kt_reserve_pages(by(m), None, ws, n, None),
    "compact": lambda m, ws=FAKE, n=BIG: kt.lib.kt_compact_pages(by(m), None, None, FAKE, FAKE, ws,
                                                                 n, None),
    "bytes": lambda m, ws=FAKE, n=BIG: kt.lib.kt_page_workspace_bytes(
        by(m), by(ctypes.c_size_t(0)) if ws == FAKE else None),
}


@pytest.mark.parametrize("call", list(CALLS))
def test_map_refusals(call):
    f = CALLS[call]
    assert f(None) == kt.KT_ERR_INVALID_ARG
    for field in ("block_table", "seq_lens", "num_blocks", "page_refs"):
        assert f(fake_map(**{field: None})) == kt.KT_ERR_INVALID_ARG
        assert f(fake_map(**{field: FAKE + 4})) == kt.KT_ERR_INVALID_ARG
    for field in ("batch", "max_blocks_per_seq", "num_pages"):
        assert f(fake_map(**{field: 0})) == kt.KT_ERR_INVALID_ARG
        assert f(fake_map(**{field: -5})) == kt.KT_ERR_INVALID_ARG
    assert f(fake_map(block_size=64)) == kt.KT_ERR_UNSUPPORTED
    assert f(fake_map(batch=2049)) == kt.KT_ERR_UNSUPPORTED
    assert f(fake_map(max_blocks_per_seq=1 << 24)) == kt.KT_ERR_UNSUPPORTED
    assert f(fake_map(num_pages=0x7FFFFFFF)) == kt.KT_ERR_UNSUPPORTED
    assert f(fake_map(), ws=None) == kt.KT_ERR_INVALID_ARG
    if call != "bytes":
        assert f(fake_map(), ws=FAKE + 8) == kt.KT_ERR_INVALID_ARG
        need = kt.kt_page_workspace_bytes(fake_map())
        assert f(fake_map(), n=need - 1) == kt.KT_ERR_WORKSPACE_TOO_SMALL
        assert need >= 256 + 2 * 400


def test_list_refusals():
    m, L = by(fake_map()), kt.lib
    bad = kt.KT_ERR_INVALID_ARG
    for n in (0, -1):
        assert L.kt_free_seqs(m, FAKE, n, FAKE, BIG, None) == bad
    for n in (0, -1, 5):
        assert L.kt_fork_seqs(m, FAKE, FAKE, n, FAKE, FAKE, FAKE, BIG, None) == bad
    assert L.kt_free_seqs(m, None, 1, FAKE, BIG, None) == bad
    assert L.kt_free_seqs(m, FAKE + 4, 1, FAKE, BIG, None) == bad
    for hole in range(4):
        for p in (None, FAKE + 4):
            args = [FAKE] * 4
            args[hole] = p
            assert L.kt_fork_seqs(m, args[0], args[1], 1, args[2], args[3], FAKE, BIG, None) == bad
    assert L.kt_reserve_pages(m, FAKE + 4, FAKE, BIG, None) == bad
    for moves, count in ((None, FAKE), (FAKE, None), (FAKE + 8, FAKE), (FAKE, FAKE + 4)):
        assert L.kt_compact_pages(m, None, None, moves, count, FAKE, BIG, None) == bad
    for table, refs in ((FAR, None), (None, FAR), (FAR + 4, FAR2), (FAR, FAR2 + 4), (FAR, FAR),
                        (FAKE + 16, FAR2), (FAR, FAR3 + 16), (FAR3, FAR2), (FAR, FAKE)):
        assert L.kt_compact_pages(m, table, refs, FAKE, FAKE, FAKE, BIG, None) == bad


def test_copy_refusals():
    bad, L = kt.KT_ERR_INVALID_ARG, kt.lib

    def call(pools=((FAKE, 32768),), n=None, pages=10, moves=FAKE, count=FAKE, most=4, ws=FAKE,
             size=256):
        a = (kt.PagePool * max(1, len(pools)))(*[kt.PagePool(*p) for p in pools])
        return L.kt_copy_pages(a, len(pools) if n is None else n, pages, moves, count, most, ws,
                               size, None)

    assert L.kt_copy_pages(None, 1, 10, FAKE, FAKE, 4, FAKE, 256, None) == bad
    for kw in (dict(n=0), dict(n=-1), dict(pages=0), dict(moves=None), dict(count=None),
               dict(most=0), dict(most=-3), dict(ws=None), dict(size=255), dict(moves=FAKE + 8),
               dict(count=FAKE + 4), dict(ws=FAKE + 8), dict(pools=((None, 64),)),
               dict(pools=((FAKE + 8, 64),)), dict(pools=((FAKE, 0),)), dict(pools=((FAKE, -4),)),
               dict(pools=((FAKE, 6),)), dict(pools=((FAKE, 64), (FAR, 2)))):
        assert call(**kw) == bad, kw
    assert call(pools=((FAKE, 64),) * 257) == kt.KT_ERR_UNSUPPORTED
    assert call(pools=((FAKE, (1 << 32) + 4),)) == kt.KT_ERR_UNSUPPORTED


def test_binding_refuses_other_tensors():
    torch = pytest.importorskip("torch")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    m = kt.page_map(i(4, 16), i(4), i(4), i(100))
    assert (m.batch, m.max_blocks_per_seq, m.num_pages, m.block_size) == (4, 16, 100, 128)
    calls = [
        lambda: kt.page_map(i(4, 16).long(), i(4), i(4), i(100)),
        lambda: kt.page_map(i(4, 32)[:, ::2], i(4), i(4), i(100)),
        lambda: kt.page_map(i(4, 16), i(3), i(4), i(100)),
        lambda: kt.page_map(i(4, 16), i(4), i(8)[::2], i(100)),
        lambda: kt.page_map(i(4, 16), i(4), i(4), i(100).float()),
        lambda: kt.kt_free_seqs(m, i(2).long(), ws, stream=1),
        lambda: kt.kt_fork_seqs(m, i(2), i(1), i(2, 2), i(1), ws, stream=1),
        lambda: kt.kt_fork_seqs(m, i(1), i(2), i(2, 2), i(1), ws, stream=1),
        lambda: kt.kt_fork_seqs(m, i(2), i(2), i(1, 2), i(1), ws, stream=1),
        lambda: kt.kt_fork_seqs(m, i(2), i(2), i(2, 2), i(1).long(), ws, stream=1),
        lambda: kt.kt_reserve_pages(m, ws, new_tokens=i(3), stream=1),
        lambda: kt.kt_compact_pages(m, i(49, 2), i(1), ws, stream=1),
        lambda: kt.kt_compact_pages(m, i(50, 2), i(1), ws, new_table=i(3, 16), new_refs=i(100),
                                    stream=1),
        lambda: kt.kt_compact_pages(m, i(50, 2), i(1), ws, new_table=i(4, 16), new_refs=i(99),
                                    stream=1),
        lambda: kt.page_pools([]),
        lambda: kt.page_pools([torch.zeros(4, 8), torch.zeros(5, 8)]),
        lambda: kt.page_pools([torch.zeros(4, 8)[:, ::2]]),
    ]
    for i_call, f in enumerate(calls):
        with pytest.raises(kt.KtError) as e:
            f()
        assert e.value.status == kt.KT_ERR_INVALID_ARG, i_call


def test_reference_keeps_the_counts():
    rng = random.Random(3)
    m = pages_ref.Map([[0] * 12 for _ in range(9)], [0] * 9, [0] * 9, [0] * 60)
    for step in range(300):
        live = [b for b in range(9) if m.blocks[b]]
        empty = [b for b in range(9) if not m.blocks[b]]
        what = rng.choice(["free", "fork", "reserve", "compact"])
        if what == "free" and live:
            m.free(rng.sample(live, rng.randint(1, len(live))))
        elif what == "fork" and empty:
            dst = rng.sample(empty, rng.randint(1, len(empty)))
            m.fork([rng.randrange(9) for _ in dst], dst)
        elif what == "reserve":
            more = [rng.randint(0, 200) for _ in range(9)]
            m.reserve(more)
            m.lens = [min(n + k, 128 * c) for n, k, c in zip(m.lens, more, m.blocks)]
        elif what == "compact":
            _, table, refs = m.compact()
            m.table = [[p if p is not None else 0 for p in row] for row in table]
            m.refs = refs
            used = sum(r > 0 for r in refs)
            assert all(r > 0 for r in refs[:used])
        held = [0] * 60
        for row, n in zip(m.table, m.blocks):
            for p in row[:n]:
                held[p] += 1
        assert held == m.refs, (step, what)
