"""Attention behind shared prefixes on the GPU, against a plain 64-bit softmax over each
sequence's own table."""
import numpy as np
import pytest

import f8_ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_long_quest_gb300 as kt
    return kt


def tolerance(mag, want, score, all_v, steps):
    """Bound of |got - want|; mag: sum p |v|, score: the largest scale * sum |q k|, all_v: sum |v| /
    sum exp(s - max s), steps: additions that a sum may go through one after the other.

    A score is accumulated in binary32 over 8 tensor-core steps, each of which may truncate 2^-23
    of the running magnitude; its base-2 exponent (at most 1.45 * 2 * score, or 32) is rounded by
    2^-24 of it twice and the exponential errs by 2^-22; P is split into two binary16 (2^-22); P V
    runs through 16 tensor-core steps (2^-23 each), and sums of blocks and of parts add 2^-24 for
    each of `steps` additions, rescaling by an exponential (2^-22 and the rounded difference of two
    maxima, 2^-23 of at most 32 or 2.9 score) at most as often as the maximum grows, which a
    bound of 16 covers together with the joins.  Numerator and denominator both carry these.
    P in binary16 parts ends at 2^-24, half a step of which is 2^-33 of 2^8 for every token, where 2^8
    stands for a P no greater than the largest."""
    score = max(score, 11.0)
    arg = max(32.0, 2.9 * score)
    p = 8 * 2.0 ** -23 * score + 2.0 ** -23 * arg + 2 * 2.0 ** -22
    p += 16 * 2.0 ** -23 + steps * 2.0 ** -24 + 16 * (2.0 ** -22 + 2.0 ** -23 * arg)
    return 2 * p * mag + 2.0 ** -22 * np.abs(want) + 2.0 ** -33 * all_v


class Batch:
    """Groups of (members, prefix blocks, tails); pages shuffled, tails behind the prefix."""

    def __init__(self, groups, heads, group, seed=0, spare=3, sharp=1.0, before=0, after=0,
                 alone=(70,), cache="f16"):
        rng = np.random.default_rng(seed)
        lens, rows = [], []
        blocks = []
        cu = [before]
        lists = [[(0, int(alone[i % len(alone)]))] for i in range(before)]
        for prefix, tails in groups:
            lists.append([(prefix, t) for t in tails])
            cu.append(cu[-1] + len(tails))
        lists += [[(0, int(alone[i % len(alone)]))] for i in range(after)]
        pages = sum((g[0][0] if g else 0) + sum(-(-max(t, 0) // 128) for _, t in g)
                    for g in lists) + spare
        order = list(rng.permutation(pages))
        for g in lists:
            shared = [order.pop() for _ in range(g[0][0])] if g else []
            for prefix, t in g:
                n = max(0, 128 * prefix + t)
                row = (shared + [order.pop() for _ in range(-(-max(t, 0) // 128))])
                lens.append(n)
                rows.append(row)
        width = max(1, max(len(r) for r in rows))
        table = np.full((len(rows), width), -1, dtype=np.int32)
        for b, r in enumerate(rows):
            table[b, :len(r)] = r
        self.heads, self.group, self.pages = heads, group, pages
        self.lens, self.table = np.array(lens, dtype=np.int32), table
        self.cu = np.array(cu, dtype=np.int32)
        self.prefix = np.array([p for p, _ in groups], dtype=np.int32)
        self.cache = cache
        shape = (pages, heads, 128, 128)
        if cache == "f16":
            self.k = (rng.normal(size=shape) * sharp).astype(np.float16)
            self.v = rng.normal(size=shape).astype(np.float16)
        else:
            # codes around 48, one scale a page and head so that values are of unit size times sharp
            self.kc = f8_ref.encode(rng.normal(size=shape) * 48)
            self.vc = f8_ref.encode(rng.normal(size=shape) * 48)
            exp = rng.integers(-2, 2, size=(2, pages, heads))
            self.ks = (max(sharp, 2.0 ** -20) * 2.0 ** exp[0] / 64).astype(np.float32)
            self.vs = (2.0 ** exp[1] / 64).astype(np.float32)
            self.decode()
        self.q = rng.normal(size=(len(rows), heads * group, 128)).astype(np.float16)
        self.skip = set()  # (sequence, block) whose page is no page

    def decode(self):
        self.k = f8_ref.decode(self.kc) * self.ks.astype(np.float64)[:, :, None, None]
        self.v = f8_ref.decode(self.vc) * self.vs.astype(np.float64)[:, :, None, None]

    def dev(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def upload(self, kt):
        self.dq, self.dt, self.dl = self.dev(self.q), self.dev(self.table), self.dev(self.lens)
        self.dcu, self.dp = self.dev(self.cu), self.dev(self.prefix)
        if self.cache == "f16":
            self.dk, self.dv = self.dev(self.k), self.dev(self.v)
            self.kv = kt.paged_kv(self.dk, self.dv, self.dt, self.dl)
        else:
            self.dk, self.dv = self.dev(self.kc), self.dev(self.vc)
            self.dks, self.dvs = self.dev(self.ks), self.dev(self.vs)
            self.kv = kt.paged_kv_f8(self.dk, self.dks, self.dv, self.dvs, self.dt, self.dl)
        self.groups = kt.prefix_groups(self.dcu, self.dp)
        self.params = kt.sparse_params(self.heads * self.group, 0, 1, 1, kt.KT_REP_QUEST,
                                       kt.KT_HEAD_SHARED)
        make = kt.workspace if self.cache == "f16" else kt.workspace_f8
        self.ws = make(kt.KT_OP_PREFIX_ATTN, self.kv, self.params)
        self.out = torch.full(self.dq.shape, 7.0, dtype=torch.float32, device="cuda")

    def call(self, kt, scale=SCALE, stream=None):
        f = kt.kt_prefix_decode_attn if self.cache == "f16" else kt.kt_prefix_decode_attn_f8
        f(self.dq, self.kv, self.groups, self.heads * self.group, scale, self.out, self.ws,
          stream=stream)

    def check(self, scale=SCALE):
        got = self.out.cpu().numpy().astype(np.float64)
        for b, n in enumerate(self.lens):
            nb = -(-int(n) // 128)
            ids = [j for j in range(nb) if (b, j) not in self.skip]
            for h in range(self.heads):
                rows = slice(h * self.group, (h + 1) * self.group)
                if not ids:
                    assert (got[b, rows] == 0).all()
                    continue
                pg = self.table[b, ids]
                left = np.concatenate([np.arange(j * 128, j * 128 + 128) for j in ids]) < n
                k = self.k[pg, h].reshape(-1, 128)[left].astype(np.float64)
                v = self.v[pg, h].reshape(-1, 128)[left].astype(np.float64)
                q = self.q[b, rows].astype(np.float64)
                s = q @ k.T * scale
                p = np.exp(s - s.max(-1, keepdims=True))
                total = p.sum(-1, keepdims=True)
                p /= total
                want = p @ v
                tol = tolerance(p @ np.abs(v), want, (np.abs(q) @ np.abs(k).T).max() * scale,
                                np.abs(v).sum(0)[None] / total, nb + 64)
                err = np.abs(got[b, rows] - want)
                assert (err <= tol).all(), (b, h, float((err / tol).max()))


def run(kt, batch, want=None, **kw):
    batch.upload(kt)
    batch.call(kt, **kw)
    assert kt.kt_read_device_status(batch.ws) == (kt.KT_OK if want is None else want)
    batch.check(kw.get("scale", SCALE))


SHAPES = {
    "one-alone": dict(groups=[(0, [1])], heads=1, group=1),
    "one-tile": dict(groups=[(1, [5, 130])], heads=1, group=1),
    "no-tails": dict(groups=[(3, [0, 0, 0])], heads=2, group=4),
    "a-group-of-one": dict(groups=[(4, [77])], heads=2, group=3),
    "no-prefix": dict(groups=[(0, [5, 300, 128])], heads=4, group=2),
    "odd-rows": dict(groups=[(5, [1, 200, 129, 64, 7])], heads=2, group=7),
    "two-groups": dict(groups=[(9, [100, 3]), (2, [500, 0, 31])], heads=4, group=8),
    "outside": dict(groups=[(3, [40, 50])], heads=2, group=4, before=2, after=3, alone=(70, 0, 400)),
    "128-rows": dict(groups=[(6, [9] * 16)], heads=1, group=8),
    "129-rows": dict(groups=[(6, [130] * 43)], heads=1, group=3),
    "256-rows": dict(groups=[(7, [3 * i for i in range(64)])], heads=2, group=4),
    "300-rows": dict(groups=[(20, [i % 5 for i in range(100)])], heads=2, group=3),
    "600-rows": dict(groups=[(11, [i % 300 for i in range(75)]), (3, [7] * 40)], heads=2, group=8),
    "many-groups": dict(groups=[(i % 4, [i, 128 - i, 200]) for i in range(30)], heads=2, group=2),
    "long": dict(groups=[(300, [1000, 5, 40])], heads=2, group=4),
    "empty-groups": dict(groups=[(0, []), (4, [10, 20]), (0, []), (0, [3])], heads=1, group=4),
}


CACHES = pytest.mark.parametrize("cache", ["f16", "f8"])


@CACHES
@pytest.mark.parametrize("name", list(SHAPES))
def test_attention(kt, name, cache):
    run(kt, Batch(**SHAPES[name], seed=len(name), cache=cache))


@CACHES
@pytest.mark.parametrize("ctas", [1, 2, 7])
@pytest.mark.parametrize("name", ["two-groups", "300-rows", "many-groups", "outside"])
def test_few_ctas(kt, name, ctas, cache):
    kt.kt_set_max_ctas(ctas)
    try:
        run(kt, Batch(**SHAPES[name], seed=ctas, cache=cache))
    finally:
        kt.kt_set_max_ctas(0)


@CACHES
@pytest.mark.parametrize("sharp", [0.0, 8.0, 60.0])
def test_flat_and_sharp_scores(kt, sharp, cache):
    run(kt, Batch(groups=[(12, [300, 1, 128, 64]), (3, [9, 9])], heads=2, group=4, sharp=sharp,
                  cache=cache))


@CACHES
@pytest.mark.parametrize("power", [18, 22, 24, 27, 33])
def test_scores_beyond_the_steps_of_binary32(kt, power, cache):
    """One channel counts; its products are whole multiples of 2^power (exact in binary32), so each
    row's output is the mean of V over the tokens with its largest score: the largest and the next
    score are 2^power apart.  (Scores near 2^power times 200.)"""
    b = Batch(groups=[(4, [300, 20, 128]), (0, [200])], heads=2, group=4, cache=cache)
    rng = np.random.default_rng(power)
    whole = rng.integers(-8, 9, size=(b.pages, 2, 128))
    b.q[:] = 0
    b.q[..., 5] = rng.integers(1, 16, size=b.q.shape[:2]) * 2.0 ** (power // 2 - 8)
    if cache == "f16":
        b.k[:] = 0
        b.k[..., 5] = whole * 2.0 ** ((power + 1) // 2 - 8)
        scale = 2.0 ** 16
    else:
        codes = np.zeros(b.kc.shape)
        codes[..., 5] = whole
        b.kc = f8_ref.encode(codes)
        b.ks[:] = 2.0 ** ((power + 1) // 2)
        b.decode()
        scale = 2.0 ** 8
    b.upload(kt)
    b.call(kt, scale=scale)
    assert kt.kt_read_device_status(b.ws) == kt.KT_OK
    got = b.out.cpu().numpy().astype(np.float64)
    for i, n in enumerate(b.lens):
        pg = b.table[i, : -(-int(n) // 128)]
        for h in range(2):
            k = b.k[pg, h].reshape(-1, 128)[:n, 5].astype(np.float64)
            v = b.v[pg, h].reshape(-1, 128)[:n].astype(np.float64)
            for g in range(4):
                # the mean of up to n equal weights: each is a power of two, exact in one part;
                # 16 tensor-core steps a block (2^-23 each), sums of blocks and parts, a division
                top = v[k == k.max()]
                tol = (16 * 2.0 ** -23 + 2.0 ** -20) * np.abs(top).mean(0)
                assert (np.abs(got[i, h * 4 + g] - top.mean(0)) <= tol).all(), (i, h, g)


@CACHES
def test_scale(kt, cache):
    run(kt, Batch(groups=[(5, [30, 150, 260])], heads=2, group=5, cache=cache), scale=0.5)


@CACHES
def test_short_members_are_attended_alone(kt, cache):
    """Of a group with a prefix of 6 blocks: one shorter, one ending inside it, one empty."""
    b = Batch(groups=[(6, [20, 300, 0, 1, 90])], heads=2, group=4, cache=cache)
    b.lens[1], b.lens[3], b.lens[4] = 5 * 128 + 3, 0, 6 * 128 - 1
    run(kt, b)
    b.lens[:] = [100, 0, 90, 0, 6 * 128 + 1]
    run(kt, b)
    b.lens[:] = 0
    run(kt, b)


def test_groups_that_make_no_sense(kt):
    shape = dict(groups=[(4, [20, 300]), (2, [9, 40, 1])], heads=2, group=4)
    for cu in ([0, 2, 6], [-1, 2, 5], [0, 3, 2], [3, 1, 5]):
        b = Batch(**shape)
        b.cu[:] = cu
        run(kt, b, want=kt.KT_ERR_DEVICE_CHECK)
    for prefix in ([-1, 2], [4, 1000]):
        b = Batch(**shape)
        b.prefix[:] = prefix
        run(kt, b, want=kt.KT_ERR_DEVICE_CHECK)
    b = Batch(**shape)
    b.lens[0] = -7
    b.upload(kt)
    b.call(kt)
    assert kt.kt_read_device_status(b.ws) == kt.KT_ERR_DEVICE_CHECK
    b.lens[0] = 0
    b.check()


@CACHES
def test_bad_pages_are_skipped(kt, cache):
    b = Batch(groups=[(4, [20, 300, 129])], heads=2, group=4, cache=cache)
    b.table[:, 2] = 1 << 30
    b.table[1, 5] = -3
    b.table[2, 4] = b.pages
    b.skip = {(0, 2), (1, 2), (2, 2), (1, 5), (2, 4)}
    run(kt, b, want=kt.KT_ERR_DEVICE_CHECK)
    b = Batch(groups=[(1, [0, 0])], heads=1, group=2, cache=cache)
    b.table[:, 0] = -1
    b.skip = {(0, 0), (1, 0)}
    run(kt, b, want=kt.KT_ERR_DEVICE_CHECK)


@pytest.mark.parametrize("value", [0.0, -1.0, float("nan"), float("inf"), 2.0 ** 31, 2.0 ** -31])
@pytest.mark.parametrize("side", ["ks", "vs"])
def test_blocks_of_bad_scales_are_skipped(kt, side, value):
    b = Batch(groups=[(4, [20, 300, 129])], heads=1, group=4, cache="f8")
    getattr(b, side)[b.table[0, 1]] = value
    getattr(b, side)[b.table[1, 5]] = value
    b.skip = {(0, 1), (1, 1), (2, 1), (1, 5)}
    run(kt, b, want=kt.KT_ERR_DEVICE_CHECK)


@pytest.mark.parametrize("k,v", [(2.0 ** -30, 2.0 ** 30), (2.0 ** 3, 2.0 ** -30)])
def test_scales_at_their_ends(kt, k, v):
    b = Batch(groups=[(4, [20, 300, 129])], heads=1, group=4, cache="f8")
    b.ks[b.table[0, 1]] = k
    b.vs[b.table[1, 5]] = v
    b.decode()
    run(kt, b)


def test_scale_that_leaves_nothing_of_the_scores(kt):
    """The product of both scales is below binary32: every token weighs the same."""
    b = Batch([(2, [5, 77, 200])], 2, 4, seed=12, cache="f8")
    b.ks[:] = 2.0 ** -30
    b.decode()
    run(kt, b, scale=1e-42)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -65504.0])
def test_rows_behind_the_end_may_be_anything(kt, value):
    b = Batch(groups=[(3, [1, 64, 127, 130]), (0, [100])], heads=2, group=4)
    for i, n in enumerate(b.lens):
        if n % 128:
            page = b.table[i, n // 128]
            b.k[page, :, n % 128:] = value
            b.v[page, :, n % 128:] = value
    for page in set(range(b.pages)) - set(b.table.ravel().tolist()):
        b.k[page] = value
        b.v[page] = value
    run(kt, b)


@pytest.mark.parametrize("code", [0x7F, 0xFF, 0x7E])
def test_codes_behind_the_end_may_be_anything(kt, code):
    b = Batch(groups=[(3, [1, 64, 127, 130]), (0, [100])], heads=2, group=4, cache="f8")
    for i, n in enumerate(b.lens):
        if n % 128:
            page = b.table[i, n // 128]
            b.kc[page, :, n % 128:] = code
            b.vc[page, :, n % 128:] = code
    for page in set(range(b.pages)) - set(b.table.ravel().tolist()):
        b.kc[page] = code
        b.vc[page] = code
    run(kt, b)


def test_values_that_are_not_finite(kt):
    """A row of its own with an infinite or NaN value does not reach the other rows.  P is hi + lo
    with lo of either sign (or 0), so an infinite V gives inf * hi + inf * lo: inf, or NaN where lo
    is not positive."""
    b = Batch(groups=[(3, [20, 64, 127])], heads=2, group=4)
    b.upload(kt)
    b.dq[1, 2] = float("nan")
    b.dv[int(b.table[2, 3]), 0, 5, 9] = float("inf")
    b.call(kt)
    out = b.out.cpu().numpy()
    assert np.isnan(out[1, 2]).all() and not np.isfinite(out[2, :4, 9]).any()
    assert np.isfinite(np.delete(out.reshape(24, 128), [1 * 8 + 2] + list(range(16, 20)), 0)).all()
    b.out[1, 2] = 0
    ok = b.out.cpu().numpy()
    b2 = Batch(groups=[(3, [20, 64, 127])], heads=2, group=4)
    b2.upload(kt)
    b2.call(kt)
    clean = b2.out.cpu().numpy()
    keep = np.ones((3, 8), dtype=bool)
    keep[1, 2] = False
    keep[2, :4] = False
    assert np.array_equal(ok[keep], clean[keep])


@CACHES
def test_the_same_every_time_and_on_other_streams(kt, cache):
    b = Batch(groups=[(30, [20, 300, 129] * 10), (7, [5] * 20)], heads=4, group=3, cache=cache)
    run(kt, b)
    first = b.out.clone()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(20):
        b.out.fill_(3.0)
        torch.cuda.synchronize()
        b.call(kt, stream=stream if i % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(b.out, first)


def test_two_calls_at_once(kt):
    """On two streams, each with its own workspace, many calls in flight."""
    batches = [Batch(groups=[(30, [i % 5 for i in range(90)])], heads=2, group=3),
               Batch(groups=[(40, [20, 300, 129] * 5), (7, [5] * 20)], heads=4, group=4, cache="f8")]
    firsts = []
    for b in batches:
        run(kt, b)
        firsts.append(b.out.clone())
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for b in batches:
        b.out.fill_(3.0)
    torch.cuda.synchronize()
    for _ in range(200):
        for b, stream in zip(batches, streams):
            b.call(kt, stream=stream)
    torch.cuda.synchronize()
    for b, first in zip(batches, firsts):
        assert kt.kt_read_device_status(b.ws) == kt.KT_OK
        assert torch.equal(b.out, first)


@CACHES
def test_calls_in_a_row_share_a_workspace(kt, cache):
    """Other groups, lengths and outputs from one call to the next, no wait between them."""
    shapes = [[(12, [20, 300, 129, 5]), (0, [7, 900])], [(1, [2000]), (3, [1, 2, 3, 4, 5])],
              [(0, [0, 1, 128, 129, 500, 10])]]
    batches = [Batch(groups=g, heads=2, group=4, seed=i, cache=cache) for i, g in enumerate(shapes)]
    for b in batches:
        run(kt, b)
    firsts = [b.out.clone() for b in batches]
    ws = max((b.ws for b in batches), key=lambda w: w.numel())
    for b in batches:
        b.ws = ws
    for _ in range(50):
        for b in batches:
            b.call(kt)
    torch.cuda.synchronize()
    assert kt.kt_read_device_status(ws) == kt.KT_OK
    for b, first in zip(batches, firsts):
        assert torch.equal(b.out, first)


@CACHES
def test_captured_call_follows_its_inputs(kt, cache):
    """Lengths, groups and queries change between replays; a second graph shares the workspace."""
    b = Batch(groups=[(6, [20, 300, 10, 1, 90]), (2, [400, 500, 600])], heads=2, group=4,
              cache=cache)
    b.upload(kt)
    graphs = []
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            b.call(kt)
        graphs.append(graph)
    rng = np.random.default_rng(1)
    full = b.lens.copy()
    for i in range(6):
        b.lens = np.array([rng.integers(0, n + 1) if rng.random() < 0.5 else n for n in full],
                          dtype=np.int32)
        b.q = rng.normal(size=b.q.shape).astype(np.float16)
        b.prefix = np.array([rng.integers(0, 7), rng.integers(0, 3)], dtype=np.int32)
        b.dl.copy_(b.dev(b.lens))
        b.dq.copy_(b.dev(b.q))
        b.dp.copy_(b.dev(b.prefix))
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert kt.kt_read_device_status(b.ws) == kt.KT_OK
        b.check()


def test_workspace_serves_the_other_calls(kt):
    """One workspace for the decode step, dense attention and this call, in turns."""
    b = Batch(groups=[(10, [700, 300, 1200])], heads=2, group=4)
    b.upload(kt)
    params = kt.sparse_params(8, 1, 2, 4, kt.KT_REP_QUEST, kt.KT_HEAD_SEPARATE)
    ws = kt.workspace(kt.KT_OP_PREFIX_ATTN, b.kv, params)
    reps = torch.zeros(kt.kt_reps_pool_bytes(b.kv, params), dtype=torch.uint8, device="cuda")
    kt.kt_build_block_reps(b.kv, params, 0, b.table.shape[1], reps)
    sel = torch.zeros(3, 2, 4, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    step, dense = torch.zeros_like(b.out), torch.zeros_like(b.out)
    own = kt.workspace(kt.KT_OP_SPARSE_STEP, b.kv, params)
    kt.kt_sparse_decode_step(b.dq, b.kv, reps, params, sel, cnt, step, own)
    want, want_sel = step.clone(), sel.clone()
    for _ in range(4):
        b.out.fill_(9.0)
        kt.kt_prefix_decode_attn(b.dq, b.kv, b.groups, 8, SCALE, b.out, ws)
        step.fill_(9.0)
        kt.kt_sparse_decode_step(b.dq, b.kv, reps, params, sel, cnt, step, ws)
        kt.kt_dense_decode_attn(b.dq, b.kv, 8, SCALE, dense, ws)
        assert kt.kt_read_device_status(ws) == kt.KT_OK
        b.check()
        assert torch.equal(step, want) and torch.equal(sel, want_sel)
        assert float((dense - b.out).abs().max()) < 1e-2
