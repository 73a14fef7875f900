"""Sequences that share pages, as a server runs them: a prompt, samples forked from it, decode steps
(pages reserved, rows appended, attention behind the shared prefix), samples freed and others forked
in their place, the pool compacted; every step against the page reference and a plain 64-bit
softmax over each sequence's own tokens."""
import numpy as np
import pytest

import f8_ref
import pages_ref
from test_gpu_prefix import tolerance

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

B, H, G, WIDTH, PAGES, PROMPT = 8, 2, 4, 6, 41, 290
SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_long_quest_gb300 as kt
    return kt


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, kt, cache):
        self.kt, self.cache = kt, cache
        self.rng = np.random.default_rng(3)
        self.table = torch.zeros(B, WIDTH, dtype=torch.int32, device="cuda")
        self.lens, self.blocks = dev([0] * B), dev([0] * B)
        self.refs = dev([0] * PAGES)
        self.map = kt.page_map(self.table, self.lens, self.blocks, self.refs)
        self.ref = pages_ref.Map(self.table.tolist(), [0] * B, [0] * B, [0] * PAGES)
        self.page_ws = kt.page_workspace(self.map)
        shape = (PAGES, H, 128, 128)
        if cache == "f16":
            self.k, self.v = (torch.full(shape, float("nan"), dtype=torch.float16, device="cuda")
                              for _ in range(2))
            self.kv = kt.paged_kv(self.k, self.v, self.table, self.lens)
            self.pools = [self.k, self.v]
        else:
            self.k, self.v = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")
                              for _ in range(2))
            self.ks, self.vs = (torch.full((PAGES, H), float("nan"), device="cuda")
                                for _ in range(2))
            self.kv = kt.paged_kv_f8(self.k, self.ks, self.v, self.vs, self.table, self.lens)
            self.pools = [self.k, self.v, self.ks, self.vs]
        self.copies = kt.page_pools(self.pools)
        self.params = kt.sparse_params(H * G, 0, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
        make = kt.workspace if cache == "f16" else kt.workspace_f8
        self.ws = make(kt.KT_OP_PREFIX_ATTN, self.kv, self.params)
        self.cu, self.prefix = dev([0, B]), dev([0])
        self.groups = kt.prefix_groups(self.cu, self.prefix)
        self.moves, self.count = torch.zeros(PAGES, 2, dtype=torch.int32, device="cuda"), dev([0])
        self.q, self.out = None, torch.zeros(B, H * G, 128, device="cuda")
        self.tokens = [np.zeros((2, 0, H, 128))] * B  # of every sequence: K and V rows

    def same(self):
        assert self.table.tolist() == self.ref.table and self.refs.tolist() == self.ref.refs
        assert self.lens.tolist() == self.ref.lens and self.blocks.tolist() == self.ref.blocks
        assert self.kt.kt_read_device_status(self.page_ws) == self.kt.KT_OK
        assert self.kt.kt_read_device_status(self.ws) == self.kt.KT_OK

    def rows(self, n):
        x = self.rng.normal(size=(2, n, H, 128)).astype(np.float16)
        return x.astype(np.float64), torch.from_numpy(x).cuda()

    def prompt(self):
        more = [PROMPT] + [0] * (B - 1)
        self.kt.kt_reserve_pages(self.map, self.page_ws, dev(more))
        self.ref.reserve(more)
        host, x = self.rows(PROMPT)
        if self.cache == "f16":  # (what a prefill does)
            for t in range(PROMPT):
                page = self.ref.table[0][t // 128]
                self.k[page, :, t % 128], self.v[page, :, t % 128] = x[0, t], x[1, t]
            self.lens[0] = PROMPT
        else:
            self.kt.kt_append_kv_f8(self.kv, self.params, x[0], x[1], self.ws,
                                    cu_tokens=dev([0] + [PROMPT] * B))
        self.ref.lens[0] = PROMPT
        self.tokens[0] = host
        self.same()

    def fork(self, src, dst):
        n = len(src)
        self.kt.kt_fork_seqs(self.map, dev(src), dev(dst), self.moves[:n], self.count, self.page_ws)
        self.kt.kt_copy_pages(self.copies, self.moves[:n], self.count, self.page_ws)
        self.ref.fork(src, dst)
        for s, d in zip(src, dst):
            self.tokens[d] = self.tokens[s]
        self.same()

    def step_calls(self, x):
        """What a decode step launches: pages, rows, attention."""
        kt = self.kt
        kt.kt_reserve_pages(self.map, self.page_ws)
        if self.cache == "f16":
            kt.kt_append_kv(self.kv, self.params, x[0], x[1], None, self.ws)
            call = kt.kt_prefix_decode_attn
        else:
            kt.kt_append_kv_f8(self.kv, self.params, x[0], x[1], self.ws)
            call = kt.kt_prefix_decode_attn_f8
        call(self.q, self.kv, self.groups, H * G, SCALE, self.out, self.ws)

    def stepped(self, host):
        """Behind a step: the reference follows, and everything is compared."""
        self.ref.reserve(None)
        for b in range(B):
            self.ref.lens[b] += 1
            self.tokens[b] = np.concatenate([self.tokens[b], host[:, b:b + 1]], axis=1)
        self.same()
        self.check()

    def contents(self):
        """The pools' values, [pages][heads][128][128]."""
        if self.cache == "f16":
            return self.k.cpu().numpy().astype(np.float64), self.v.cpu().numpy().astype(np.float64)
        return tuple(f8_ref.decode(c.cpu().numpy()) *
                     s.cpu().numpy().astype(np.float64)[:, :, None, None]
                     for c, s in ((self.k, self.ks), (self.v, self.vs)))

    def check(self):
        pools = self.contents()
        got, q = self.out.cpu().numpy().astype(np.float64), self.q.cpu().numpy().astype(np.float64)
        for b in range(B):
            n = self.ref.lens[b]
            pages = self.ref.table[b][:-(-n // 128)]
            k, v = (x[pages].transpose(1, 0, 2, 3).reshape(H, -1, 128)[:, :n] for x in pools)
            rows = self.tokens[b].transpose(0, 2, 1, 3)
            if self.cache == "f16":
                assert np.array_equal(k, rows[0]) and np.array_equal(v, rows[1])
            else:
                # an e4m3 code next to the largest, 448, is off by 16 of its scale; codes that are
                # made anew when a scale grows, to twice as much at most, by 16, 8, ... more
                for x, y in ((k, rows[0]), (v, rows[1])):
                    for at in range(0, n, 128):
                        part = np.abs(y[:, at:at + 128])
                        step = 2 * part.max((1, 2), keepdims=True) / 448 * 32
                        assert (np.abs(x[:, at:at + 128] - y[:, at:at + 128]) <= step).all()
            for h in range(H):
                heads = slice(h * G, (h + 1) * G)
                s = q[b, heads] @ k[h].T * SCALE
                p = np.exp(s - s.max(-1, keepdims=True))
                total = p.sum(-1, keepdims=True)
                p /= total
                want = p @ v[h]
                tol = tolerance(p @ np.abs(v[h]), want,
                                (np.abs(q[b, heads]) @ np.abs(k[h]).T).max() * SCALE,
                                np.abs(v[h]).sum(0)[None] / total, -(-n // 128) + 64)
                assert (np.abs(got[b, heads] - want) <= tol).all()


@pytest.mark.parametrize("cache", ["f16", "f8"])
def test_samples_of_a_prompt(kt, cache):
    sv = Server(kt, cache)
    sv.prompt()
    sv.fork([0] * 7, list(range(1, 8)))
    sv.prefix.fill_(PROMPT // 128)
    sv.q = torch.randn(B, H * G, 128, generator=torch.Generator().manual_seed(1)).half().cuda()
    for _ in range(2):
        host, x = sv.rows(B)
        sv.step_calls(x)
        sv.stepped(host)
    # two samples end, two others take their places; each slot's page of its own is copied
    sv.kt.kt_free_seqs(sv.map, dev([2, 5]), sv.page_ws)
    sv.ref.free([2, 5])
    sv.same()
    sv.fork([7, 1], [2, 5])
    # a captured step, over the border of a page
    host, x = sv.rows(B)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        sv.step_calls(x)
    for _ in range(384 - PROMPT):
        host, new = sv.rows(B)
        x.copy_(new)
        graph.replay()
        sv.ref.reserve(None)
        for b in range(B):
            sv.ref.lens[b] += 1
            sv.tokens[b] = np.concatenate([sv.tokens[b], host[:, b:b + 1]], axis=1)
    sv.same()
    sv.check()
    assert sv.ref.lens[0] > 384
    # holes of freed sequences close; what the pages hold, and the attention, stays
    sv.kt.kt_free_seqs(sv.map, dev([0, 3, 4]), sv.page_ws)
    sv.ref.free([0, 3, 4])
    sv.same()
    before = None
    for turn in range(2):
        (kt.kt_prefix_decode_attn if cache == "f16" else kt.kt_prefix_decode_attn_f8)(
            sv.q, sv.kv, sv.groups, H * G, SCALE, sv.out, sv.ws)
        if turn == 0:
            before = sv.out.clone()
            kt.kt_compact_pages(sv.map, sv.moves[:PAGES // 2], sv.count, sv.page_ws)
            kt.kt_copy_pages(sv.copies, sv.moves[:PAGES // 2], sv.count, sv.page_ws)
            want, table, refs = sv.ref.compact()
            assert sv.count.item() == len(want) > 0
            sv.ref.table = [[o if w is None else w for w, o in zip(row, old)]
                            for row, old in zip(table, sv.ref.table)]
            sv.ref.refs = refs
            sv.same()
    assert torch.equal(sv.out, before)
    assert (sv.out[[0, 3, 4]] == 0).all() and (sv.out[[1, 2, 5, 6, 7]] != 0).any()
    used = [p for p, r in enumerate(sv.ref.refs) if r > 0]
    assert used == list(range(len(used)))
