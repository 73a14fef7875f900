"""One page map for the caches of three layers: every layer of a step appends with the map's lengths,
leaves the new ones apart and attends with those; samples forked and freed, representatives kept."""
import numpy as np
import pytest

from test_gpu_shared_sequences import PAGES, PROMPT, SCALE, B, G, H, Server, dev

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

LAYERS = 3


@pytest.fixture(scope="module", autouse=True)
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_long_quest_gb300 as kt
    return kt


class Layers:
    """A Server a layer, on the map (and its reference) of the first one."""

    def __init__(self, kt, cache, in_place):
        self.kt, self.cache, self.in_place = kt, cache, in_place
        self.sv = [Server(kt, cache) for _ in range(LAYERS)]
        self.first = f = self.sv[0]
        self.next = dev([0] * B)
        self.reps = [torch.zeros(PAGES, H, 2, 128, dtype=torch.float16, device="cuda")
                     for _ in range(LAYERS)]
        self.kv, self.kv_next = [], []
        for i, s in enumerate(self.sv):
            s.rng, s.ref, s.ws = np.random.default_rng(i), f.ref, f.ws
            for kvs, lens in ((self.kv, f.lens), (self.kv_next, self.next)):
                kvs.append(kt.paged_kv(s.k, s.v, f.table, lens) if cache == "f16" else
                           kt.paged_kv_f8(s.k, s.ks, s.v, s.vs, f.table, lens))
            s.q = torch.randn(B, H * G, 128, generator=torch.Generator().manual_seed(i)).half().cuda()
        self.copies = kt.page_pools([p for s in self.sv for p in s.pools] + self.reps)

    def prompt(self):
        kt, f = self.kt, self.first
        more = [PROMPT] + [0] * (B - 1)
        kt.kt_reserve_pages(f.map, f.page_ws, dev(more))
        f.ref.reserve(more)
        for i, s in enumerate(self.sv):
            host, x = s.rows(PROMPT)
            s.tokens[0] = host
            if self.cache == "f8":
                kt.kt_append_kv_f8(self.kv[i], s.params, x[0], x[1], f.ws, new_lens=self.next,
                                   cu_tokens=dev([0] + [PROMPT] * B), reps_pool=self.reps[i])
                continue
            for t in range(PROMPT):
                page = f.ref.table[0][t // 128]
                s.k[page, :, t % 128], s.v[page, :, t % 128] = x[0, t], x[1, t]
            self.next[0] = PROMPT
            kt.kt_build_block_reps(self.kv_next[i], s.params, 0, PROMPT // 128, self.reps[i])
        f.lens.copy_(self.next)
        f.ref.lens[0] = PROMPT
        f.same()

    def fork(self, src, dst):
        f, n = self.first, len(src)
        self.kt.kt_fork_seqs(f.map, dev(src), dev(dst), f.moves[:n], f.count, f.page_ws)
        self.kt.kt_copy_pages(self.copies, f.moves[:n], f.count, f.page_ws)
        f.ref.fork(src, dst)
        for s in self.sv:
            for a, b in zip(src, dst):
                s.tokens[b] = s.tokens[a]
        f.same()

    def step(self, rows):
        """What a decode step over the layers launches."""
        kt, f = self.kt, self.first
        kt.kt_reserve_pages(f.map, f.page_ws)
        for i, s in enumerate(self.sv):
            last = self.in_place and i == LAYERS - 1
            new = f.lens if last else self.next
            if self.cache == "f16":
                kt.kt_append_kv_lens(self.kv[i], s.params, rows[i][0], rows[i][1], new, self.reps[i],
                                     f.ws)
                call = kt.kt_prefix_decode_attn
            else:
                kt.kt_append_kv_f8(self.kv[i], s.params, rows[i][0], rows[i][1], f.ws, new_lens=new,
                                   reps_pool=self.reps[i])
                call = kt.kt_prefix_decode_attn_f8
            call(s.q, (self.kv if last else self.kv_next)[i], f.groups, H * G, SCALE, s.out, f.ws)
        if not self.in_place:
            f.lens.copy_(self.next)

    def stepped(self, hosts):
        f = self.first
        f.ref.reserve(None)
        for b in range(B):
            f.ref.lens[b] += 1
            for s, host in zip(self.sv, hosts):
                s.tokens[b] = np.concatenate([s.tokens[b], host[:, b:b + 1]], axis=1)

    def check(self):
        self.first.same()
        for i, s in enumerate(self.sv):
            s.check()
            fresh = torch.zeros_like(self.reps[i])
            build = self.kt.kt_build_block_reps if self.cache == "f16" else \
                self.kt.kt_build_block_reps_f8
            build(self.kv[i], s.params, 0, self.first.table.shape[1], fresh)
            full = sorted({p for row, n in zip(s.ref.table, s.ref.lens) for p in row[:n // 128]})
            assert len(full) >= PROMPT // 128
            assert torch.equal(self.reps[i][full], fresh[full])


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "last-in-place"])
@pytest.mark.parametrize("cache", ["f16", "f8"])
def test_layers_on_one_map(kt, cache, in_place):
    m = Layers(kt, cache, in_place)
    m.prompt()
    m.fork([0] * 7, list(range(1, 8)))
    m.first.prefix.fill_(PROMPT // 128)
    for _ in range(2):
        hosts, rows = zip(*(s.rows(B) for s in m.sv))
        m.step(rows)
        m.stepped(hosts)
        m.check()
    m.kt.kt_free_seqs(m.first.map, dev([2, 5]), m.first.page_ws)
    m.first.ref.free([2, 5])
    m.fork([7, 1], [2, 5])
    # a captured step, over the end of a block
    hosts, rows = zip(*(s.rows(B) for s in m.sv))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        m.step(rows)
    for _ in range(384 - PROMPT):
        hosts, new = zip(*(s.rows(B) for s in m.sv))
        for x, y in zip(rows, new):
            x.copy_(y)
        graph.replay()
        m.stepped(hosts)
    assert m.first.ref.lens[0] > 384
    m.check()


def test_append_with_lengths_apart(kt):
    """Lengths of sequences that grow, that have no room and that make no sense; the cache's own stay,
    and the pools become what the append in place makes of them."""
    lens = [0, 127, 128, 300, 384, -3, 5]
    table = torch.arange(21, dtype=torch.int32, device="cuda").reshape(7, 3)
    table[6, 0] = 21  # no page
    gen = torch.Generator(device="cuda").manual_seed(4)
    new = torch.randn(2, 7, 2, 128, generator=gen, device="cuda").half()
    pools = torch.randn(2, 21, 2, 128, 128, generator=gen, device="cuda").half()
    params = kt.sparse_params(4, 0, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = []
    for apart in (False, True):
        own, out, x = dev(lens), dev([77] * 7), pools.clone()
        kv = kt.paged_kv(x[0], x[1], table, own)
        reps = torch.zeros(kt.kt_reps_pool_bytes(kv, params), dtype=torch.uint8, device="cuda")
        if apart:
            kt.kt_append_kv_lens(kv, params, new[0], new[1], out, reps, ws)
            assert own.tolist() == lens
        else:
            kt.kt_append_kv(kv, params, new[0], new[1], reps, ws)
            out = own
        assert kt.kt_read_device_status(ws) == kt.KT_ERR_DEVICE_CHECK
        assert out.tolist() == [1, 128, 129, 301, 384, -3, 5]
        got.append((x, reps))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert bool((got[1][1].view(torch.float16).reshape(21, -1)[3] != 0).any())
