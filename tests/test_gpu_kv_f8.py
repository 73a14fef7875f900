"""Rotary positions and the 8-bit cache on the GPU: the quantising append, its
representatives, reading back and the attention over the codes, against a plain
64-bit reference (f8_ref), bit for bit where the definition leaves no freedom."""
import ctypes

import numpy as np
import pytest

import f8_ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_long_quest_gb300 as kt
    return kt


DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SCALE = 128 ** -0.5
def attention_tolerance(mag, want, score, all_v):
    """Bound of |got - want|; mag: sum p |v|, score: the largest SCALE * sum |q k|, all_v: sum |v| /
    sum exp(s - max s).

    A score is accumulated in binary32 over 8 tensor-core steps, each of which may truncate 2^-23
    of the running magnitude; the base-2 exponent and its argument (at most 2 * 1.45 * score, or 32)
    err by 2^-22 of it; P is split into two binary16 (2^-22); the sums over a warp's tokens and over
    warps add 2^-24 for each of fewer than 2^9 steps.  Numerator and denominator both carry these.
    2^15 P / max P in binary16 parts ends at 2^-24, half a step of which is 2^-40 of the largest P
    for every token, however small its own.  Inputs of unit size have score < 22.6 (2^8 * SCALE),
    which gives 1.2e-4."""
    score = max(score, 22.6)
    p = 8 * 2.0 ** -23 * score + 2.0 ** -22 * max(32.0, 2.9 * score) + 2.0 ** -22 + 2.0 ** -15
    return 2 * p * mag + 2.0 ** -22 * np.abs(want) + 2.0 ** -40 * all_v


@pytest.fixture(autouse=True)
def _seed():
    torch.manual_seed(1234)


def host16(t):
    """Values of a row tensor as the cache takes them: rounded to binary16 (numpy)."""
    return t.cpu().to(torch.float16).numpy()


def assert_status(kt, ws, want=None):
    assert kt.kt_read_device_status(ws) == (kt.KT_OK if want is None else want)


# ---- rotary positions -------------------------------------------------------------------
def check_rope(got, x, pos, f, amp, layout):
    x = x.float().cpu().numpy()
    want, mag = f8_ref.rotate(x, pos, f, amp, layout)
    tol = f8_ref.rope_tolerance(want, mag, pos, f, amp)
    n = 2 * len(f)
    got = got.cpu().numpy()
    err = np.abs(got.astype(np.float64) - want)
    assert (err <= tol).all(), (err - tol).max()
    # behind the rotated channels: the input's own binary16 value
    with np.errstate(over="ignore"):
        assert np.array_equal(got[..., n:], x[..., n:].astype(np.float16))


SCALINGS = [("plain", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 32.0), ("bands", 8.0)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("rot", [128, 96, 64, 32, 16, 126, 58, 6, 2])
def test_rope(kt, dtype, layout, rot):
    rng = torch.Generator().manual_seed(rot)
    for n, (tokens, hq, hk, gap) in enumerate([(1, 32, 8, 0), (5, 3, 1, 16), (613, 4, 4, 1024)]):
        scaling, factor = SCALINGS[(n + rot) % 5]
        if scaling == "ntk" and rot == 2:
            scaling, factor = "linear", 3.0
        fast = 4.0 if scaling == "bands" else 32.0
        row = (hq + hk) * 128 + gap  # a packed projection with other parts behind
        buf = torch.randn(tokens, row, generator=rng).to(DTYPES[dtype]).cuda()
        x = buf[:, :(hq + hk) * 128].unflatten(1, (hq + hk, 128))
        pos = torch.randint(-5, 1 << 20, (tokens,), generator=rng, dtype=torch.int64)
        pos[-1] = (1 << 31) - 1 if n == 1 else pos[-1]
        pos = pos.to(torch.int32)
        lay = kt.KT_ROPE_HALF if layout == "half" else kt.KT_ROPE_PAIRS
        kind = dict(plain=kt.KT_ROPE_PLAIN, linear=kt.KT_ROPE_LINEAR, ntk=kt.KT_ROPE_NTK,
                    yarn=kt.KT_ROPE_YARN, bands=kt.KT_ROPE_BANDS)[scaling]
        r = kt.rope(rot, theta=1e6, layout=lay, scaling=kind, factor=factor, original_len=8192,
                    beta_fast=fast)
        f, amp = f8_ref.frequencies(rot, 1e6, scaling, factor, 8192, fast)
        q_out = torch.full((tokens + 1, hq, 128), 7.0, dtype=torch.float16, device="cuda")
        k_out = torch.full((tokens + 1, hk, 128), 7.0, dtype=torch.float16, device="cuda")
        kt.kt_apply_rope(r, pos.cuda(), x[:, :hq], q_out[:tokens], x[:, hq:], k_out[:tokens])
        for out, part in ((q_out, x[:, :hq]), (k_out, x[:, hq:])):
            check_rope(out[:tokens], part, pos.numpy(), f, amp, layout)
            assert (out[tokens:] == 7.0).all()
        # one of the two alone gives the same rows
        alone = torch.zeros_like(k_out[:tokens])
        kt.kt_apply_rope(r, pos.cuda(), k=x[:, hq:], k_out=alone)
        assert torch.equal(alone, k_out[:tokens])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("layout,rot", [("half", 128), ("pairs", 128), ("half", 90)])
def test_rope_is_elementary_binary32(kt, dtype, layout, rot):
    """The rows are those of elementary binary32 operations (products and sum rounded) on the
    binary32 values nearest to cos and sin.

    The kernel's cos and sin err by three roundings of terms below pi/256 next to the nearest
    value's: by 3 * 2^-25 / 81.5 < 1.1e-9, at most 1.9% of the spacing 2^-24 of values in [1/2, 1),
    so fewer than 1 of 26 are not the nearest one (smaller values more often, but their products
    count less).  A result with two such products is off by about 2^-24 |x| then, and the spacing
    of binary16 is at least 2^-11 of the result: with |x| three times the result on the whole, a
    rounding changes in fewer than 2/26 * 3 * 2^-13 = 2^-15.1 of all; twice that is allowed."""
    rng = torch.Generator().manual_seed(3)
    x = torch.randn(512, 16, 128, generator=rng).to(DTYPES[dtype])
    pos = torch.randint(0, 60000, (512,), generator=rng, dtype=torch.int32)
    f, _ = f8_ref.frequencies(rot, 1e6)
    ang = np.fmod(pos.numpy().astype(np.longdouble)[:, None] * f, f8_ref.PI2).astype(np.float64)
    c, s = (torch.from_numpy(t(ang)).float()[:, None] for t in (np.cos, np.sin))
    n, y = rot // 2, x.float().clone()
    a, b = (slice(0, n), slice(n, rot)) if layout == "half" else (slice(0, rot, 2),
                                                                  slice(1, rot, 2))
    y[..., a], y[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    out = torch.empty(x.shape, dtype=torch.float16, device="cuda")
    lay = kt.KT_ROPE_HALF if layout == "half" else kt.KT_ROPE_PAIRS
    kt.kt_apply_rope(kt.rope(rot, theta=1e6, layout=lay), pos.cuda(), x.cuda(), out)
    assert (out.cpu() != y.half()).sum() <= x.numel() * 2.0 ** -14


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rot", [128, 64, 90])
def test_rope_in_place_and_without_effect(kt, layout, rot):
    x = torch.randn(77, 5, 128).half().cuda()
    pos = torch.arange(77, dtype=torch.int32).cuda() * 991
    r = kt.rope(rot, layout=layout)
    want = torch.empty_like(x)
    kt.kt_apply_rope(r, pos, x, want)
    y = x.clone()
    kt.kt_apply_rope(r, pos, y, y)
    assert torch.equal(y, want)
    kt.kt_apply_rope(r, torch.zeros_like(pos), x, y)  # position 0
    assert torch.equal(y, x)
    kt.kt_apply_rope(r, pos[:0], x[:0], y[:0])        # no tokens
    assert torch.equal(y, x)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("layout,rot", [("half", 128), ("half", 48), ("pairs", 96), ("half", 90)])
@pytest.mark.parametrize("tokens,hq,hk", [(3000, 32, 8), (2501, 13, 0), (2433, 9, 9)])
def test_rope_of_many_tokens(kt, dtype, layout, rot, tokens, hq, hk):
    """Enough tokens for a warp to take all heads of one, eight rows at a time: whole turns and a
    last one of fewer heads, that ends inside q or inside k."""
    rng = torch.Generator().manual_seed(tokens + rot)
    assert tokens >= 16 * torch.cuda.get_device_properties(0).multi_processor_count
    x = torch.randn(tokens, hq + hk, 128, generator=rng).to(DTYPES[dtype]).cuda()
    pos = torch.randint(0, 1 << 21, (tokens,), generator=rng, dtype=torch.int32)
    r = kt.rope(rot, theta=5e5, layout=kt.KT_ROPE_HALF if layout == "half" else kt.KT_ROPE_PAIRS)
    f, amp = f8_ref.frequencies(rot, 5e5)
    q, k = x[:, :hq], x[:, hq:] if hk else None
    q_out = torch.full((tokens + 1, hq, 128), 7.0, dtype=torch.float16, device="cuda")
    k_out = torch.full((tokens + 1, max(hk, 1), 128), 7.0, dtype=torch.float16, device="cuda")
    kt.kt_apply_rope(r, pos.cuda(), q, q_out[:tokens], k, k_out[:tokens] if hk else None)
    check_rope(q_out[:tokens], q, pos.numpy(), f, amp, layout)
    if hk:
        check_rope(k_out[:tokens], k, pos.numpy(), f, amp, layout)
    assert (q_out[tokens:] == 7.0).all() and (k_out[tokens if hk else 0:] == 7.0).all()
    if dtype == "f16":  # in place
        y = q.contiguous()
        kt.kt_apply_rope(r, pos.cuda(), y, y)
        assert torch.equal(y, q_out[:tokens])


def test_rope_turns_back(kt):
    """The rotation by -p undoes the rotation by p: what its transpose, and so its gradient, is."""
    x = torch.randn(50, 4, 128, dtype=torch.float32).cuda()
    pos = torch.randint(0, 1 << 20, (50,), dtype=torch.int32).cuda()
    r = kt.rope(128)
    y = torch.empty(50, 4, 128, dtype=torch.float16, device="cuda")
    z = torch.empty_like(y)
    kt.kt_apply_rope(r, pos, x, y)
    kt.kt_apply_rope(r, -pos, y, z)
    # two roundings to binary16 of values up to |x| + |y| of a pair, and their rotation
    pair = (x.abs() + x.abs().roll(64, -1)).cpu()
    assert ((z.float().cpu() - x.cpu()).abs() <= 2.0 ** -11 * 2.1 * pair + 2.0 ** -24).all()


def test_rope_non_finite_values_stay_in_their_pairs(kt):
    x = torch.randn(3, 2, 128).half().cuda()
    x[1, 0, 5], x[2, 1, 100], x[0, 0, 127] = float("inf"), float("nan"), 60000.0
    pos = torch.tensor([0, 3, 9], dtype=torch.int32).cuda()
    for layout, partner in ((0, lambda c: (c + 32) % 64), (1, lambda c: c ^ 1)):
        out = torch.empty_like(x)
        kt.kt_apply_rope(kt.rope(64, layout=layout), pos, x, out)
        bad = ~torch.isfinite(out)
        want = torch.zeros_like(bad)
        want[1, 0, 5] = want[1, 0, partner(5)] = True
        want[2, 1, 100] = True  # passes through
        assert torch.equal(bad, want)


# ---- the cache --------------------------------------------------------------------------
class Paged:
    """An 8-bit cache on the device with a shuffled table, and its host copy."""

    def __init__(self, kt, lens, H, blocks, seed, garbage=True, spare=3):
        self.kt, self.H = kt, H
        rng = np.random.default_rng(seed)
        B = len(lens)
        pages = B * blocks + spare
        fill = 0x7F if garbage else 0  # e4m3 NaN wherever nothing was written
        mk = lambda: torch.full((pages, H, 128, 128), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.k_code, self.v_code = mk(), mk()
        self.k_scale = torch.full((pages, H), float("nan"), device="cuda")
        self.v_scale = torch.full((pages, H), float("nan"), device="cuda")
        self.table = torch.from_numpy(rng.permutation(pages)[:B * blocks].reshape(B, blocks)
                                      .astype(np.int32)).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.kv = kt.paged_kv_f8(self.k_code, self.k_scale, self.v_code, self.v_scale, self.table,
                                 self.lens)
        self.host = f8_ref.Cache(self.k_code.cpu().numpy(), self.k_scale.cpu().numpy(),
                                 self.v_code.cpu().numpy(), self.v_scale.cpu().numpy(),
                                 self.table.cpu().numpy(), self.lens.cpu().numpy())

    def check(self):
        for side, code, scale in (("k", self.k_code, self.k_scale),
                                  ("v", self.v_code, self.v_scale)):
            assert np.array_equal(scale.cpu().numpy().astype(np.float64), self.host.scale[side],
                                  equal_nan=True), side
            assert f8_ref.same_codes(code.cpu().numpy(), self.host.code[side]), side
        assert np.array_equal(self.lens.cpu().numpy(), self.host.lens)


def reps_pool(kt, pg, params):
    n = kt.kt_reps_pool_bytes_f8(pg.kv, params)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def check_reps(kt, pg, pool, rep, done):
    """The reps of the blocks `done`, and nothing written for any other page."""
    pages, rows = pg.k_code.shape[0], {0: 1, 1: 1, 2: 2, 3: 4}[rep]
    a = pool.cpu().numpy().view(np.float32 if rep == 1 else np.float16)
    a = a.reshape(pages, pg.H, rows, 128)
    seen = np.zeros(pages, dtype=bool)
    for b, j in done:
        page = int(pg.host.table[b, j])
        seen[page] = True
        for h in range(pg.H):
            want = pg.host.reps(page, h, rep).astype(a.dtype)
            assert np.array_equal(a[page, h], want), (b, j, h)
    raw = pool.cpu().numpy().reshape(pages, -1)
    assert (raw[~seen] == 0xFF).all()


def rows_of(rng, tokens, H, dtype, spread=1.0):
    x = torch.randn(tokens, H, 128, generator=rng)
    x *= torch.exp2(torch.rand(tokens, 1, 1, generator=rng) * spread - spread / 2)
    return x.to(DTYPES[dtype]).cuda()


COUNTS = [  # rows of three sequences, call after call: empty ones, block borders, long chunks
    [1, 0, 127], [1, 128, 1], [126, 1, 0], [300, 2, 129], [0, 0, 0], [5, 256, 255], [1, 1, 1],
]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rep", [0, 1, 2, 3])
@pytest.mark.parametrize("H,in_place", [(1, True), (8, False)])
def test_append_ragged(kt, dtype, rep, H, in_place):
    rng = torch.Generator().manual_seed(7 * rep + H)
    pg = Paged(kt, [0, 0, 0], H, 7, 11)
    p = kt.sparse_params(H, 1, 2, 2, rep, kt.KT_HEAD_SHARED)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    pool, done = reps_pool(kt, pg, p), []
    for counts in COUNTS:
        m = sum(counts)
        k, v = rows_of(rng, m, H, dtype, 6.0), rows_of(rng, m, H, dtype, 6.0)
        cu = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
        new = None if in_place else torch.full((3,), -1, dtype=torch.int32, device="cuda")
        before = pg.lens.clone()
        kt.kt_append_kv_f8(pg.kv, p, k, v, ws, cu_tokens=cu, new_lens=new, reps_pool=pool)
        done += pg.host.append(host16(k), host16(v), counts)
        if not in_place:
            assert torch.equal(pg.lens, before)
            pg.lens.copy_(new)
        pg.check()
        check_reps(kt, pg, pool, rep, done)
        assert_status(kt, ws)
    assert (ws[:256] == 0).all()  # the header is left as it was found
    # the same reps from the finished cache
    again = reps_pool(kt, pg, p)
    kt.kt_build_block_reps_f8(pg.kv, p, 0, 7, again)
    assert torch.equal(again, pool)


@pytest.mark.parametrize("B,H", [(1, 2), (5, 3), (300, 1)])
def test_append_one_row_each(kt, B, H):
    """The decode form (no cu_tokens) over a block border, equal to the ragged form."""
    rng = torch.Generator().manual_seed(B)
    lens = [(125 + 37 * b) % 200 for b in range(B)]
    pg, other = Paged(kt, [0] * B, H, 3, 5), Paged(kt, [0] * B, H, 3, 5)
    p = kt.sparse_params(H, 1, 1, 2, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    k, v = rows_of(rng, sum(lens), H, "f16"), rows_of(rng, sum(lens), H, "f16")
    for x in (pg, other):
        kt.kt_append_kv_f8(x.kv, p, k, v, ws, cu_tokens=cu)
        x.host.append(host16(k), host16(v), lens)
        x.check()
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    pools = [reps_pool(kt, pg, p), reps_pool(kt, pg, p)]
    done = []
    for step in range(5):
        k, v = rows_of(rng, B, H, "f16", 9.0), rows_of(rng, B, H, "f16", 9.0)
        kt.kt_append_kv_f8(pg.kv, p, k, v, ws, reps_pool=pools[0])
        kt.kt_append_kv_f8(other.kv, p, k, v, ws, cu_tokens=one, reps_pool=pools[1])
        done += pg.host.append(host16(k), host16(v), [1] * B)
        pg.check()
        assert torch.equal(other.lens, pg.lens) and torch.equal(other.k_code, pg.k_code)
        assert torch.equal(other.v_code, pg.v_code) and torch.equal(pools[0], pools[1])
    check_reps(kt, pg, pools[0], 2, done)
    assert_status(kt, ws)


def test_append_range_of_values(kt):
    """Scales from 2^-15 to 2^8, codes at their borders, zeros, subnormals, infinities and NaN."""
    pg = Paged(kt, [0], 1, 4, 3)
    p = kt.sparse_params(1, 1, 1, 2, kt.KT_REP_MAX, kt.KT_HEAD_SHARED)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    every = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.float16)
    grid = torch.from_numpy(np.concatenate([f8_ref.GRID, (f8_ref.GRID[1:] + f8_ref.GRID[:-1]) / 2]))
    rows = [torch.zeros(1, 128), torch.full((1, 128), -0.0), torch.full((3, 128), 2.0 ** -24),
            torch.full((2, 128), 448 * 2.0 ** -15), torch.full((2, 128), 449 * 2.0 ** -15),
            torch.nn.functional.pad(grid, (0, 3)).reshape(-1, 128),
            torch.nn.functional.pad(-grid, (0, 3)).reshape(-1, 128),
            torch.full((1, 128), 65504.0), torch.full((1, 128), -63488.0),
            torch.tensor([61440.0, 63487.0, -65504.0, float("nan")]).repeat(32)[None],
            torch.full((1, 128), float("nan")), torch.full((1, 128), float("inf")),
            torch.full((1, 128), -float("inf"))]
    x = torch.cat([r.half() for r in rows])
    for part in (x[:5], x[5:9], x[9:], every[:128 * 100].reshape(-1, 128),
                 every[1 << 15:(1 << 15) + 128 * 100].reshape(-1, 128), every[-128:].reshape(1, -1)):
        y = part[:, None, :].contiguous().cuda()
        cu = torch.tensor([0, y.shape[0]], dtype=torch.int32, device="cuda")
        kt.kt_append_kv_f8(pg.kv, p, y, -y, ws, cu_tokens=cu)
        h = y.cpu().numpy()
        pg.host.append(h, -h, [y.shape[0]])
        pg.check()
    assert_status(kt, ws)


def test_append_grown_scale_codes_old_rows_again(kt):
    """Each row twice as large as the one before: every call shifts the rows before it."""
    pg = Paged(kt, [0], 2, 1, 3)
    p = kt.sparse_params(2, 1, 1, 2, kt.KT_REP_MAX, kt.KT_HEAD_SHARED)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    x = torch.randn(1, 2, 128).cuda()
    for e in range(-14, 12):
        y = (x * 2.0 ** e).half()
        kt.kt_append_kv_f8(pg.kv, p, y, -y, ws)
        h = y.cpu().numpy()
        pg.host.append(h, -h, [1])
        pg.check()


@pytest.mark.parametrize("layout,rot", [(0, 128), (0, 64), (1, 128), (1, 34), (0, 50)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_append_rotated_equals_rotation_then_append(kt, dtype, layout, rot):
    """From one packed projection: q, k rotated in the call, equal to kt_apply_rope's rows."""
    rng = torch.Generator().manual_seed(rot)
    lens, counts, H, G = [90, 3, 128], [200, 1, 61], 2, 4
    pg, other = Paged(kt, [0] * 3, H, 4, 5), Paged(kt, [0] * 3, H, 4, 5)
    p = kt.sparse_params(H * G, 1, 1, 2, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    r = kt.rope(rot, theta=1e5, layout=layout)
    k0, v0 = rows_of(rng, sum(lens), H, dtype), rows_of(rng, sum(lens), H, dtype)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    for x in (pg, other):
        kt.kt_append_kv_f8(x.kv, p, k0, v0, ws, cu_tokens=cu)
    cu = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
    qkv = rows_of(rng, sum(counts), H * G + 2 * H, dtype, 4.0)
    q, k, v = qkv[:, :H * G], qkv[:, H * G:H * G + H], qkv[:, H * G + H:]
    pos = torch.cat([torch.arange(n, n + m) for n, m in zip(lens, counts)]).to(torch.int32).cuda()
    q1, k1 = (torch.empty(sum(counts), h, 128, dtype=torch.float16, device="cuda")
              for h in (H * G, H))
    kt.kt_apply_rope(r, pos, q, q1, k, k1)
    pools = [reps_pool(kt, pg, p), reps_pool(kt, pg, p)]
    kt.kt_append_kv_f8(other.kv, p, k1, v.half().contiguous(), ws, cu_tokens=cu,
                       reps_pool=pools[1])
    q2 = torch.empty_like(q1)
    kt.kt_append_kv_f8(pg.kv, p, k, v, ws, rope=r, q=q, q_out=q2, cu_tokens=cu,
                       reps_pool=pools[0])
    assert torch.equal(q1, q2) and torch.equal(pools[0], pools[1])
    for a in ("k_code", "v_code", "lens"):
        assert torch.equal(getattr(pg, a), getattr(other, a)), a
    assert torch.equal(torch.nan_to_num(pg.k_scale), torch.nan_to_num(other.k_scale))
    # without a rotation q is only rounded
    kt.kt_append_kv_f8(pg.kv, p, k, v, ws, q=q, q_out=q2, cu_tokens=cu)
    assert torch.equal(q2, q.half())
    assert_status(kt, ws)


HEADS_A_CTA = [  # KV heads, query heads a KV head, K heads a CTA, cached lengths and new rows
    (8, 4, 4, [80], [9900]),
    (8, 8, 4, [(53 * b) % 300 for b in range(30)], [(71 * b) % 150 for b in range(30)]),
    (5, 1, 3, [(53 * b) % 300 for b in range(40)], [(37 * b) % 130 for b in range(40)]),
    (3, 2, 2, [(29 * b) % 200 for b in range(50)], [(41 * b) % 140 for b in range(50)]),
    (8, 1, 2, [(53 * b) % 300 for b in range(20)], [(91 * b) % 170 for b in range(20)]),
]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("case", range(len(HEADS_A_CTA)))
def test_append_with_several_heads_a_cta(kt, dtype, case):
    """Rotated appends of so many blocks that a CTA takes several K heads of one, the last group
    fewer: codes, scales, representatives and q, bit for bit, from begun blocks whose scale grows
    and into blocks that the call completes."""
    H, G, heads, lens, counts = HEADS_A_CTA[case]
    n = case + list(DTYPES).index(dtype)
    layout, rot = [("half", 128), ("pairs", 64), ("half", 90)][n % 3]
    rep, stride = [(0, 1), (1, 1), (2, 1), (3, 8)][n % 4]
    B, m = len(lens), sum(counts)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per = min(4, (m // 128 + 2 * B) * H // sms)
    groups = -(-H // per)
    assert -(-H // groups) == heads  # the launch takes as many heads a CTA as meant here
    rng = torch.Generator().manual_seed(case)
    blocks = max(-(-(a + c) // 128) for a, c in zip(lens, counts))
    pg, other = Paged(kt, [0] * B, H, blocks, 15), Paged(kt, [0] * B, H, blocks, 15)
    p = kt.sparse_params(H * G, 1, 1, 2, rep, kt.KT_HEAD_SHARED, fix_stride=stride)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    k, v = rows_of(rng, sum(lens), H, "f16", 6.0), rows_of(rng, sum(lens), H, "f16", 6.0)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    for x in (pg, other):
        kt.kt_append_kv_f8(x.kv, p, k, v, ws, cu_tokens=cu)
    pg.host.append(host16(k), host16(v), lens)
    qkv = rows_of(rng, m, H * G + 2 * H, dtype, 8.0)
    q, k, v = qkv[:, :H * G], qkv[:, H * G:H * G + H], qkv[:, H * G + H:]
    pos = torch.cat([torch.arange(a, a + c) for a, c in zip(lens, counts)]).to(torch.int32)
    r = kt.rope(rot, theta=1e5, layout=kt.KT_ROPE_HALF if layout == "half" else kt.KT_ROPE_PAIRS)
    q1, k1 = (torch.empty(m, h, 128, dtype=torch.float16, device="cuda") for h in (H * G, H))
    kt.kt_apply_rope(r, pos.cuda(), q, q1, k, k1)
    f, amp = f8_ref.frequencies(rot, 1e5)
    check_rope(k1, k, pos.numpy(), f, amp, layout)
    check_rope(q1, q, pos.numpy(), f, amp, layout)
    cu = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
    pools = [reps_pool(kt, pg, p), reps_pool(kt, pg, p)]
    q2 = torch.zeros_like(q1)
    kt.kt_append_kv_f8(pg.kv, p, k, v, ws, rope=r, q=q, q_out=q2, cu_tokens=cu,
                       reps_pool=pools[0])
    assert torch.equal(q1, q2)
    done = pg.host.append(host16(k1), host16(v), counts)
    pg.check()
    # representatives: as an unrotated append of the rotated rows builds them, a head a CTA
    kt.kt_append_kv_f8(other.kv, p, k1, v.half().contiguous(), ws, cu_tokens=cu,
                       reps_pool=pools[1])
    assert torch.equal(pools[0], pools[1]) and torch.equal(other.k_code, pg.k_code)
    rows = {0: 1, 1: 1, 2: 2, 3: 128 // stride}[rep]
    got = pools[0].cpu().numpy().view(np.float32 if rep == 1 else np.float16)
    got = got.reshape(-1, H, rows, 128)
    assert done
    for b, j in done:
        page = int(pg.host.table[b, j])
        for h in range(H):
            assert np.array_equal(got[page, h],
                                  pg.host.reps(page, h, rep, stride).astype(got.dtype)), (b, j, h)
    assert_status(kt, ws)
    assert (ws[:256] == 0).all()


def test_append_refuses_on_the_device(kt):
    """A negative length, no room, rows outside the call, a page outside the pool and a scale that
    is no power of two: recorded, and the other sequences are served."""
    H = 2
    p = kt.sparse_params(H, 1, 1, 2, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    k, v = torch.randn(12, H, 128).half().cuda(), torch.randn(12, H, 128).half().cuda()
    h, g = host16(k), host16(v)
    cu = torch.tensor([0, 4, 8, 12], dtype=torch.int32, device="cuda")

    def fresh(lens):
        pg = Paged(kt, lens, H, 2, 9)
        return pg, kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)

    for bad in (-1, 253, 1 << 30):
        for in_place in (True, False):
            pg, ws = fresh([0, bad, 0])
            new = None if in_place else torch.zeros(3, dtype=torch.int32, device="cuda")
            kt.kt_append_kv_f8(pg.kv, p, k, v, ws, cu_tokens=cu, new_lens=new)
            assert_status(kt, ws, kt.KT_ERR_DEVICE_CHECK)
            pg.host.lens[1] = 0
            pg.host.append(np.concatenate([h[:4], h[8:]]), np.concatenate([g[:4], g[8:]]),
                           [4, 0, 4])
            pg.host.lens[1] = bad
            if not in_place:
                pg.lens.copy_(new)
            pg.check()
    for cu_bad, counts in (([0, 4, 8, 13], [4, 4, 0]), ([-1, 4, 8, 12], [0, 4, 4])):
        pg, ws = fresh([0, 0, 0])
        kt.kt_append_kv_f8(pg.kv, p, k, v, ws, cu_tokens=torch.tensor(cu_bad, dtype=torch.int32,
                                                                      device="cuda"))
        assert_status(kt, ws, kt.KT_ERR_DEVICE_CHECK)
        rows = slice(0, 8) if counts[0] else slice(4, 12)
        pg.host.append(h[rows], g[rows], counts)
        pg.check()
    for page in (-1, 9, 1 << 30):  # the pool has 9 pages
        for in_place in (True, False):
            pg, ws = fresh([126, 0, 0])
            pg.k_scale.fill_(1.0), pg.v_scale.fill_(1.0)
            before = pg.k_code.clone()
            pg.table[0, 1] = page
            new = None if in_place else torch.zeros(3, dtype=torch.int32, device="cuda")
            kt.kt_append_kv_f8(pg.kv, p, k, v, ws, cu_tokens=cu, new_lens=new)
            assert_status(kt, ws, kt.KT_ERR_DEVICE_CHECK)
            assert (pg.lens if in_place else new).tolist() == [126, 4, 4]
            first = int(pg.table[0, 0])
            assert torch.equal(pg.k_code[first, :, :126], before[first, :, :126])
    pg, ws = fresh([5, 0, 0])
    pg.k_scale.fill_(1.5), pg.v_scale.fill_(float("nan"))
    kt.kt_append_kv_f8(pg.kv, p, k, v, ws, cu_tokens=cu)
    assert_status(kt, ws, kt.KT_ERR_DEVICE_CHECK)
    page = int(pg.table[0, 0])
    for x, code, scale in ((h, pg.k_code, pg.k_scale), (g, pg.v_code, pg.v_scale)):
        for i in range(H):
            s = f8_ref.block_scale(np.abs(x[:4, i].astype(np.float64)).max())
            assert float(scale[page, i]) == s
            assert f8_ref.same_codes(code[page, i, 5:9].cpu().numpy(),
                                     f8_ref.code_rows(x[:4, i], s))
    # no tokens at all: lengths pass through
    new = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    kt.kt_append_kv_f8(pg.kv, p, k[:0], v[:0], ws, cu_tokens=torch.zeros_like(cu), new_lens=new)
    assert torch.equal(new, pg.lens)


def test_long_spans_of_pages_are_checked(kt):
    """A bad page far inside a long chunk keeps the length; a good chunk of the same size not."""
    H, n = 1, 128 * 200 + 17
    p = kt.sparse_params(H, 1, 1, 2, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    x = torch.randn(n + 3, H, 128).half().cuda()
    cu = torch.tensor([0, n, n + 3], dtype=torch.int32, device="cuda")
    for bad in (False, True):
        pg = Paged(kt, [0, 0], H, 202, 4)
        ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
        if bad:
            pg.table[0, 170] = pg.k_code.shape[0]
        kt.kt_append_kv_f8(pg.kv, p, x, x, ws, cu_tokens=cu)
        assert pg.lens.tolist() == [0 if bad else n, 3]
        assert_status(kt, ws, kt.KT_ERR_DEVICE_CHECK if bad else kt.KT_OK)


@pytest.mark.parametrize("tokens", [40, 4000])  # q beside the tiles, and ahead of them
@pytest.mark.parametrize("rotated", [False, True])
def test_append_of_a_padded_batch(kt, tokens, rotated):
    """Rows in front of the first sequence and behind the last are of no sequence: not appended,
    and their rows of q_out stay as they were."""
    H, Hq, lo, hi = 2, 4, 3, tokens - 11
    rng = torch.Generator().manual_seed(tokens)
    p = kt.sparse_params(Hq, 1, 1, 2, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    q, k, v = (rows_of(rng, tokens, h, "f16") for h in (Hq, H, H))
    rope = kt.rope(64) if rotated else None
    got = []
    for a, b in ((0, tokens), (lo, hi)):
        pg = Paged(kt, [100, 0, 7], H, 34, 17, garbage=False)
        pg.k_scale.fill_(1.0)
        pg.v_scale.fill_(1.0)
        ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
        q_out = torch.full_like(q, 9.0)
        rows = slice(0, tokens) if a else slice(lo, hi)
        cu = torch.tensor([0, 1, 1, hi - lo], dtype=torch.int32, device="cuda") + a
        kt.kt_append_kv_f8(pg.kv, p, k[rows], v[rows], ws, rope=rope, q=q[rows],
                           q_out=q_out[rows], cu_tokens=cu)
        assert pg.lens.tolist() == [101, 0, 7 + hi - lo - 1]
        assert_status(kt, ws)
        got.append((q_out, pg.k_code, pg.v_code, pg.k_scale, pg.v_scale))
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert (got[1][0][:lo] == 9.0).all() and (got[1][0][hi:] == 9.0).all()
    assert (got[1][0][lo:hi] != 9.0).any(-1).all()


@pytest.mark.parametrize("B", [32, 33, 257, 1500])
def test_many_sequences(kt, B):
    """Ragged rows of many sequences, most of them short or empty: appended, then read back."""
    rng = np.random.default_rng(B)
    counts = [int(c) for c in rng.choice([0, 0, 1, 2, 130], B, p=[.3, .1, .4, .17, .03])]
    m = sum(counts)
    gen = torch.Generator().manual_seed(B)
    pg = Paged(kt, [0] * B, 1, 2, B)
    p = kt.sparse_params(1, 1, 1, 2, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    k, v = rows_of(gen, m, 1, "f16"), rows_of(gen, m, 1, "f16")
    q = rows_of(gen, m, 1, "f16")
    q_out, want = torch.empty_like(q), torch.empty_like(q)
    cu = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
    r = kt.rope(128)
    pos = torch.cat([torch.arange(c) for c in counts]).to(torch.int32).cuda()
    kr = torch.empty_like(k)
    kt.kt_apply_rope(r, pos, q, want, k, kr)
    kt.kt_append_kv_f8(pg.kv, p, k, v, ws, rope=r, q=q, q_out=q_out, cu_tokens=cu)
    pg.host.append(host16(kr), host16(v), counts)
    pg.check()
    assert torch.equal(q_out, want)
    back = torch.empty_like(k)
    kt.kt_read_kv_f8(pg.kv, cu, back, None, ws)
    exact = np.concatenate([pg.host.values("k", int(pg.host.table[b, t // 128]), 0)[t % 128][None]
                            for b in range(B) for t in range(counts[b])])
    assert np.array_equal(back[:, 0].double().cpu().numpy(), exact)
    assert_status(kt, ws)


def test_long_append_rotates_q_ahead(kt):
    """More rows than ride along with the tiles: q in a launch of its own, lengths in place."""
    counts, H, G = [1700, 0, 900, 1], 2, 2
    gen = torch.Generator().manual_seed(5)
    qkv = rows_of(gen, sum(counts), H * G + 2 * H, "bf16")
    q, k, v = qkv[:, :H * G], qkv[:, H * G:H * G + H], qkv[:, H * G + H:]
    cu = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
    p = kt.sparse_params(H * G, 1, 1, 2, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    r = kt.rope(128)
    pos = torch.cat([torch.arange(c) for c in counts]).to(torch.int32).cuda()
    want, kr = (torch.empty(sum(counts), h, 128, dtype=torch.float16, device="cuda")
                for h in (H * G, H))
    kt.kt_apply_rope(r, pos, q, want, k, kr)
    for rope in (r, None):
        pg = Paged(kt, [0] * 4, H, 14, 5)
        ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
        q_out = torch.empty_like(want)
        for _ in range(3):  # back to back: each call reads the lengths the one before left
            pg.lens.zero_()
            kt.kt_append_kv_f8(pg.kv, p, k, v, ws, rope=rope, q=q, q_out=q_out, cu_tokens=cu)
        pg.host.append(host16(kr if rope else k), host16(v), counts)
        pg.check()
        assert torch.equal(q_out, want if rope else q.half())
        # captured: the two launches of a call keep their order with what surrounds them
        again = Paged(kt, [0] * 4, H, 14, 5)
        side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            for _ in range(3):
                again.lens.zero_()
                q_out.zero_()
                kt.kt_append_kv_f8(again.kv, p, k, v, ws, rope=rope, q=q, q_out=q_out,
                                   cu_tokens=cu)
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(3):
            g.replay()
        assert torch.equal(again.lens, pg.lens) and torch.equal(again.k_code, pg.k_code)
        assert torch.equal(q_out, want if rope else q.half())
        assert_status(kt, ws)


# ---- reading back -----------------------------------------------------------------------
def filled(kt, lens, H, seed, blocks=None, params=None, spread=5.0):
    blocks = max(1, -(-max(lens) // 128)) if blocks is None else blocks
    pg = Paged(kt, [0] * len(lens), H, blocks, seed)
    p = params or kt.sparse_params(H, 1, 1, 2, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    rng = torch.Generator().manual_seed(seed)
    m = sum(lens)
    k, v = rows_of(rng, m, H, "f16", spread), rows_of(rng, m, H, "f16", spread)
    # blocks of very different size, so that scales differ from block to block
    size = torch.exp2(torch.randint(-3, 4, (len(lens), blocks), generator=rng).float())
    f = torch.cat([size[b].repeat_interleave(128)[:n] for b, n in enumerate(lens)])
    v = (v * f[:, None, None].cuda()).half()
    cu = torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device="cuda")
    kt.kt_append_kv_f8(pg.kv, p, k, v, ws, cu_tokens=cu)
    pg.host = f8_ref.Cache(pg.k_code.cpu().numpy(), pg.k_scale.cpu().numpy(),
                           pg.v_code.cpu().numpy(), pg.v_scale.cpu().numpy(),
                           pg.table.cpu().numpy(), pg.lens.cpu().numpy())
    assert pg.lens.tolist() == list(lens)
    assert_status(kt, ws)
    return pg


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H", [1, 3, 8])
def test_read_back(kt, dtype, H):
    lens, first, counts = [300, 1, 700, 129], [37, 0, 127, 128], [263, 0, 520, 1]
    pg = filled(kt, lens, H, 21)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    m = sum(counts)
    cu = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
    fst = torch.tensor(first, dtype=torch.int32, device="cuda")
    outs = [torch.full((m + 2, H, 128), 3.0, dtype=DTYPES[dtype], device="cuda") for _ in "kv"]
    kt.kt_read_kv_f8(pg.kv, cu, outs[0][:m], outs[1][:m], ws, first=fst)
    for side, out in zip("kv", outs):
        want = np.concatenate([
            np.stack([pg.host.values(side, int(pg.host.table[b, t // 128]), h)[t % 128]
                      for h in range(H)])[None]
            for b in range(4) for t in range(first[b], first[b] + counts[b])])
        assert np.array_equal(out[:m].double().cpu().numpy(), want)
        assert (out[m:] == 3.0).all()
    alone = torch.zeros_like(outs[1][:m])
    kt.kt_read_kv_f8(pg.kv, cu, None, alone, ws, first=fst)
    assert torch.equal(alone, outs[1][:m])
    alone.zero_()
    kt.kt_read_kv_f8(pg.kv, cu, alone, None, ws, first=fst)
    assert torch.equal(alone, outs[0][:m])
    kt.kt_read_kv_f8(pg.kv, cu * 0, alone[:0], None, ws)  # nothing
    assert_status(kt, ws)


def test_read_outside_is_left_alone(kt):
    pg = filled(kt, [200, 130], 2, 22)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda")

    def read(first, cu=cu, n=20):
        out = torch.full((n, 2, 128), 9.0, dtype=torch.float32, device="cuda")
        kt.kt_read_kv_f8(pg.kv, cu, out, None, ws,
                         first=torch.tensor(first, dtype=torch.int32, device="cuda"))
        return (out != 9.0).any(-1).any(-1).cpu()

    touched = read([195, 0])
    assert touched.tolist() == [True] * 5 + [False] * 5 + [True] * 10
    assert_status(kt, ws, kt.KT_ERR_DEVICE_CHECK)
    touched = read([-4, (1 << 31) - 5])
    assert touched.tolist() == [False] * 4 + [True] * 6 + [False] * 10
    assert_status(kt, ws, kt.KT_ERR_DEVICE_CHECK)
    # rows of no sequence are no error
    touched = read([0, 0], torch.tensor([2, 4, 15], dtype=torch.int32, device="cuda"))
    assert touched.tolist() == [False] * 2 + [True] * 13 + [False] * 5
    assert_status(kt, ws)
    pg.table[1, 0] = 77
    touched = read([0, 120])
    assert touched.tolist() == [True] * 10 + [False] * 8 + [True] * 2
    assert_status(kt, ws, kt.KT_ERR_DEVICE_CHECK)
    touched = read([0, 128])  # the second sequence ends after two of its rows
    assert touched.tolist() == [True] * 12 + [False] * 8
    assert_status(kt, ws, kt.KT_ERR_DEVICE_CHECK)
    read([190, 128], torch.tensor([0, 10, 12], dtype=torch.int32, device="cuda"), 12)
    assert_status(kt, ws)


# ---- attention --------------------------------------------------------------------------
def check_attention(pg, q, out, blocks_of, G):
    """out against the reference; blocks_of(b, h): the blocks of sequence b and KV head h."""
    q, out = q.cpu().numpy(), out.cpu().numpy().astype(np.float64)
    for b in range(len(pg.host.lens)):
        for h in range(pg.H):
            sl = slice(h * G, h * G + G)
            blocks = blocks_of(b, h)
            if pg.host.lens[b] == 0 or not len(blocks):
                assert (out[b, sl] == 0).all()
                continue
            want, mag, score, all_v = pg.host.attend(q[b, sl], b, h, blocks, SCALE)
            err = np.abs(out[b, sl] - want)
            tol = attention_tolerance(mag, want, score, all_v)
            assert (err <= tol).all(), (b, h, (err / tol).max())


@pytest.mark.parametrize("G", [1, 3, 4, 8])
@pytest.mark.parametrize("H,lens", [(1, [1]), (2, [0, 17, 128, 129, 0, 255]), (8, [1500, 3, 640]),
                                    (4, [127]), (1, [40000])])
def test_dense_attention(kt, G, H, lens):
    pg = filled(kt, lens, H, 31 + G)
    q = torch.randn(len(lens), H * G, 128).half().cuda()
    out = torch.full((len(lens), H * G, 128), float("nan"), device="cuda")
    p = kt.sparse_params(H * G, 0, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    ws = kt.workspace_f8(kt.KT_OP_DENSE_ATTN, pg.kv, p)
    for _ in range(2):
        kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, out, ws)
        check_attention(pg, q, out, lambda b, h: range(-(-int(pg.host.lens[b]) // 128)), G)
    assert_status(kt, ws)
    first = out.clone()
    for ctas in (1, 2, 7):  # another split of the long axis, the same answer within rounding
        kt.kt_set_max_ctas(ctas)
        kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, out, ws)
        kt.kt_set_max_ctas(0)
        check_attention(pg, q, out, lambda b, h: range(-(-int(pg.host.lens[b]) // 128)), G)
    kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, out, ws)
    assert torch.equal(out, first)


@pytest.mark.parametrize("G,H,lens", [
    (4, 8, [20000, 3, 0, 9000, 129, 12345, 128 * 11]),  # one list of blocks over all SMs
    (8, 2, [70000, 128, 60001]),
    (2, 1, [(37 * b) % 300 for b in range(400)]),       # more segments than SMs, empty ones too
    (1, 1, [0] * 200),
])
def test_dense_attention_shares_the_blocks_out(kt, G, H, lens):
    """Enough blocks for every CTA to take an equal part of all segments' blocks: pieces of a
    segment in several CTAs, several segments in a CTA."""
    pg = filled(kt, lens, H, 37)
    q = torch.randn(len(lens), H * G, 128).half().cuda()
    p = kt.sparse_params(H * G, 0, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    ws = kt.workspace_f8(kt.KT_OP_DENSE_ATTN, pg.kv, p)
    first = None
    for ctas in (0, 0, 0, 3, 50):
        out = torch.full((len(lens), H * G, 128), float("nan"), device="cuda")
        kt.kt_set_max_ctas(ctas)
        kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, out, ws)
        kt.kt_set_max_ctas(0)
        if first is None or ctas:
            check_attention(pg, q, out, lambda b, h: range(-(-int(pg.host.lens[b]) // 128)), G)
            first = out if first is None else first
        else:
            assert torch.equal(out, first)  # the order of the sums is the CTAs', not their timing
    assert_status(kt, ws)


def segment_counters(ws, segments):
    """The counters of the segments' parts: behind the workspace's header, zero between calls."""
    return ws[256:256 + 4 * segments]


# more segments than SMs, most of them empty: (KV heads, lengths of 32 or more sequences)
PADDED = [
    (8, [200] + [0] * 31),
    (8, [0] * 31 + [1000]),
    (8, [300, 300] + [0] * 30),
    (8, [0, 200, 0, 0, 641] + [0] * 25 + [200, 1]),
    (4, [200] + [0] * 39),
    (8, [0] * 13 + [1000, 0, 1000, 257] + [0] * 14 + [1024]),
    (1, [0] * 100 + [5] + [0] * 99),
]


@pytest.mark.parametrize("ctas", [0, 40, 7])
@pytest.mark.parametrize("H,lens", PADDED)
def test_padded_batches_of_more_segments_than_ctas(kt, H, lens, ctas):
    """Few live sequences in a batch of many slots: fewer blocks in all than CTAs.  Every segment is
    written, the workspace's counters are back at zero, and calls of other lengths on the same
    workspace, and the binary16 dense call, are right too."""
    G = 4
    B = len(lens)
    pg = filled(kt, lens, H, 41)
    q = torch.randn(B, H * G, 128).half().cuda()
    p = kt.sparse_params(H * G, 1, 1, 3, kt.KT_REP_QUEST, kt.KT_HEAD_SEPARATE)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    every = lambda b, h: range(-(-int(pg.host.lens[b]) // 128))  # noqa: E731
    out = torch.empty(B, H * G, 128, device="cuda")

    def run(call, blocks_of):
        out.fill_(float("nan"))
        kt.kt_set_max_ctas(ctas)
        call()
        kt.kt_set_max_ctas(0)
        check_attention(pg, q, out, blocks_of, G)
        assert (segment_counters(ws, B * H) == 0).all()

    sel = torch.full((B, H, 3), -1, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(B, H, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(5)
    for b, n in enumerate(lens):  # any choice of the Context blocks: 1 .. nb - 2
        nb = -(-n // 128)
        for h in range(H):
            ids = np.sort(rng.permutation(max(0, nb - 2))[:rng.integers(0, 4)]) + 1
            sel[b, h, :len(ids)] = torch.from_numpy(ids.astype(np.int32))
            cnt[b, h] = len(ids)
    hs, hc = sel.cpu(), cnt.cpu()
    picked = lambda b, h: chosen(kt, pg, hs, hc, p, b, h)  # noqa: E731
    dense = lambda: kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, out, ws)  # noqa: E731
    sparse = lambda: kt.kt_sparse_decode_attn_f8(q, pg.kv, p, sel, cnt, out, ws)  # noqa: E731
    for _ in range(2):
        run(dense, every)
        run(sparse, picked)
    kv16, _k, _v = paged16(kt, pg)
    out.fill_(float("nan"))
    kt.kt_dense_decode_attn(q, kv16, H * G, SCALE, out, ws)
    check_attention(pg, q, out, every, G)
    # the lengths one block shorter
    pg.lens.copy_(torch.clamp(pg.lens - 128, min=0))
    pg.host.lens = pg.lens.cpu().numpy()
    run(dense, every)
    assert_status(kt, ws)


@pytest.mark.parametrize("live", [{0: 300}, {7: 1000, 30: 200}, {3: 700, 4: 1024, 17: 1, 31: 257}])
@pytest.mark.parametrize("mode", [0, 1])
def test_padded_step_in_two_launches(kt, mode, live):
    """The step and the layer call over a batch of 32 slots with few live sequences."""
    H, G, B = 8, 4, 32
    lens = [live.get(b, 0) for b in range(B)]
    p = kt.sparse_params(H * G, 1, 1, 3, kt.KT_REP_QUEST, mode)
    pg = filled(kt, lens, H, 43, params=p)
    kv16 = kt.PagedKV(pg.k_code.data_ptr(), pg.v_code.data_ptr(), pg.table.data_ptr(),
                      pg.lens.data_ptr(), B, H, 128, 128, pg.table.shape[1], pg.k_code.shape[0])
    assert kt.kt_sparse_decode_step_kernels(kv16, p) == 2
    q = torch.randn(B, H * G, 128).half().cuda()
    pool = reps_pool(kt, pg, p)
    kt.kt_build_block_reps_f8(pg.kv, p, 0, 100, pool)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    U = 1 if mode == kt.KT_HEAD_SHARED else H
    hist = torch.zeros(1, B, U, 3, dtype=torch.int32, device="cuda")
    cnts = torch.full((1, B, U), -1, dtype=torch.int32, device="cuda")
    out = torch.empty(B, H * G, 128, device="cuda")
    pol = kt.reuse_policy(1, dense_layer_num=0)
    assert kt.kt_decode_layer_action(pol, 0, 0) == (kt.KT_LAYER_SELECT, 0)
    for layer in (False, True, False):
        out.fill_(float("nan"))
        if layer:
            kt.kt_decode_layer_f8(pol, 0, 0, q, pg.kv, pool, p, hist, cnts, out, ws)
        else:
            kt.kt_sparse_decode_step_f8(q, pg.kv, pool, p, hist[0], cnts[0], out, ws)
        hs, hc = hist[0].cpu(), cnts[0].cpu()
        for b, n in enumerate(lens):
            assert (hc[b] == min(3, max(0, -(-n // 128) - 2))).all()
        check_attention(pg, q, out, lambda b, h: chosen(kt, pg, hs, hc, p, b, h), G)
        assert (segment_counters(ws, B * H) == 0).all()
    assert_status(kt, ws)


def test_captured_batch_that_empties_and_fills(kt):
    """Sequences of a captured batch of more segments than SMs end and begin between replays: each
    replay gives what eager calls on a workspace of their own give, to the bit."""
    H, G, B = 8, 4, 32
    full = [128 * 9 + 5 * b for b in range(B)]
    p = kt.sparse_params(H * G, 1, 2, 3, kt.KT_REP_QUEST, kt.KT_HEAD_SEPARATE)
    pg = filled(kt, full, H, 45, params=p)
    q = torch.randn(B, H * G, 128).half().cuda()
    pool = reps_pool(kt, pg, p)
    kt.kt_build_block_reps_f8(pg.kv, p, 0, 100, pool)

    def buffers():
        return (kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p),
                torch.zeros(B, H, 3, dtype=torch.int32, device="cuda"),
                torch.zeros(B, H, dtype=torch.int32, device="cuda"),
                torch.empty(B, H * G, 128, device="cuda"), torch.empty(B, H * G, 128, device="cuda"))

    def run(ws, sel, cnt, step, dense):
        kt.kt_sparse_decode_step_f8(q, pg.kv, pool, p, sel, cnt, step, ws)
        kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, dense, ws)

    a, c = buffers(), buffers()
    run(*a)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        run(*a)
    torch.cuda.current_stream().wait_stream(side)
    for live in ({}, {3: 200}, None, {0: 1000, 31: 1}, {b: 5 for b in range(B)}, {17: 1237}, None):
        lens = full if live is None else [live.get(b, 0) for b in range(B)]
        pg.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for x in (a, c):
            x[3].fill_(float("nan")), x[4].fill_(float("nan"))
        g.replay()
        run(*c)
        assert torch.equal(a[3], c[3]) and torch.equal(a[4], c[4]) and torch.equal(a[2], c[2])
        assert torch.isfinite(a[3]).all() and torch.isfinite(a[4]).all()
        pg.host.lens = np.array(lens)
        check_attention(pg, q, a[4], lambda b, h: range(-(-lens[b] // 128)), G)
        assert (segment_counters(a[0], B * H) == 0).all()
    assert_status(kt, a[0])


def chosen(kt, pg, sel, cnt, p, b, h):
    u = 0 if p.head_mode == kt.KT_HEAD_SHARED else h
    nb = -(-int(pg.host.lens[b]) // 128)
    c0 = min(p.initial_blocks, nb)
    c1 = max(c0, nb - p.local_blocks)
    return list(range(c0)) + sel[b, u, :int(cnt[b, u])].tolist() + list(range(c1, nb))


def paged16(kt, pg):
    """The cache's values in binary16 pools (exact), for the framework's binary16 calls."""
    c = [torch.from_numpy(f8_ref.decode(x.cpu().numpy())) for x in (pg.k_code, pg.v_code)]
    s = [x.cpu().double()[:, :, None, None] for x in (pg.k_scale, pg.v_scale)]
    k, v = (torch.nan_to_num(a * b).half().cuda() for a, b in zip(c, s))
    return kt.paged_kv(k, v, pg.table, pg.lens), k, v


@pytest.mark.parametrize("G,H", [(4, 2), (1, 1), (8, 4), (3, 2)])
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("rep", [0, 1, 2, 3])
def test_step_and_its_parts(kt, rep, mode, G, H):
    """The step's selection is that of the binary16 calls over the same representatives; its
    attention, and that over the given selection, are the reference's."""
    lens = [128 * 30 + 77, 128 * 9, 128 * 5 + 1, 90]
    p = kt.sparse_params(H * G, 1, 2, 5, rep, mode)
    pg = filled(kt, lens, H, 51, params=p)
    q = torch.randn(len(lens), H * G, 128).half().cuda()
    pool = reps_pool(kt, pg, p)
    kt.kt_build_block_reps_f8(pg.kv, p, 0, 1 << 20, pool)
    check_reps(kt, pg, pool, rep, [(b, j) for b, n in enumerate(lens) for j in range(n // 128)])
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    U = 1 if mode == kt.KT_HEAD_SHARED else H
    mk = lambda: torch.full((4, U, 5), -1, dtype=torch.int32, device="cuda")  # noqa: E731
    sel, sel2, sel3 = mk(), mk(), mk()
    cnt, cnt2, cnt3 = (torch.full((4, U), -1, dtype=torch.int32, device="cuda") for _ in "abc")
    out = torch.full((4, H * G, 128), float("nan"), device="cuda")
    kt.kt_sparse_decode_step_f8(q, pg.kv, pool, p, sel, cnt, out, ws)
    kv16, _k, _v = paged16(kt, pg)
    kt.kt_score_select_blocks(q, kv16, pool, p, sel2, cnt2, None, ws)
    kt.kt_score_select_blocks_f8(q, pg.kv, pool, p, sel3, cnt3, None, ws)
    assert torch.equal(cnt, cnt2) and torch.equal(cnt, cnt3) and torch.equal(sel2, sel3)
    sel16, cnt16, out16 = mk(), cnt.clone(), torch.empty_like(out)
    kt.kt_sparse_decode_step(q, kv16, pool, p, sel16, cnt16, out16, ws)
    assert torch.equal(sel, sel16)
    hs, hc = sel.cpu(), cnt.cpu()
    check_attention(pg, q, out, lambda b, h: chosen(kt, pg, hs, hc, p, b, h), G)
    kt.kt_sparse_decode_attn_f8(q, pg.kv, p, sel, cnt, out, ws)
    check_attention(pg, q, out, lambda b, h: chosen(kt, pg, hs, hc, p, b, h), G)
    assert_status(kt, ws)


@pytest.mark.parametrize("batch", [1, 60])
def test_step_in_one_and_in_two_launches(kt, batch):
    """One launch for few segments; 480 segments take the selection and the attention apart."""
    H, G, rep, mode = 8, 4, 2, 1
    lens = [128 * 12 + 5 + b for b in range(batch)]
    p = kt.sparse_params(H * G, 1, 2, 3, rep, mode)
    pg = filled(kt, lens, H, 53, params=p)
    kv16 = kt.PagedKV(pg.k_code.data_ptr(), pg.v_code.data_ptr(), pg.table.data_ptr(),
                      pg.lens.data_ptr(), batch, H, 128, 128, pg.table.shape[1],
                      pg.k_code.shape[0])
    assert kt.kt_sparse_decode_step_kernels(kv16, p) == (1 if batch == 1 else 2)
    q = torch.randn(batch, H * G, 128).half().cuda()
    pool = reps_pool(kt, pg, p)
    kt.kt_build_block_reps_f8(pg.kv, p, 0, 100, pool)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    sel = torch.zeros(batch, H, 3, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(batch, H, dtype=torch.int32, device="cuda")
    out = torch.empty(batch, H * G, 128, device="cuda")
    for _ in range(3):
        kt.kt_sparse_decode_step_f8(q, pg.kv, pool, p, sel, cnt, out, ws)
        hs, hc = sel.cpu(), cnt.cpu()
        assert (hc == 3).all()
        check_attention(pg, q, out, lambda b, h: chosen(kt, pg, hs, hc, p, b, h), G)
    assert_status(kt, ws)


def test_scales_from_elsewhere(kt):
    """Scales that are no powers of two serve the attention; zeros, NaN and infinities are
    recorded and their block is left out."""
    H, G, lens = 2, 4, [128 * 6 + 9]
    pg = filled(kt, lens, H, 61)
    rng = np.random.default_rng(1)
    for t in (pg.k_scale, pg.v_scale):
        t.copy_(torch.from_numpy(rng.uniform(0.01, 1.0, t.shape).astype(np.float32)))
    pg.host.scale = {"k": pg.k_scale.cpu().double().numpy(), "v": pg.v_scale.cpu().double().numpy()}
    q = torch.randn(1, H * G, 128).half().cuda()
    out = torch.empty(1, H * G, 128, device="cuda")
    p = kt.sparse_params(H * G, 0, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    ws = kt.workspace_f8(kt.KT_OP_DENSE_ATTN, pg.kv, p)
    kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, out, ws)
    check_attention(pg, q, out, lambda b, h: range(7), G)
    assert_status(kt, ws)
    # V scales 2^-30 and 2^30 beside one another
    page = [int(x) for x in pg.table[0].cpu()]
    pg.v_scale[page[1]], pg.v_scale[page[2]] = 2.0 ** -30, 2.0 ** 30
    pg.host.scale["v"] = pg.v_scale.cpu().double().numpy()
    kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, out, ws)
    check_attention(pg, q, out, lambda b, h: range(7), G)
    assert_status(kt, ws)
    for which, value in ((pg.k_scale, 0.0), (pg.v_scale, float("nan")), (pg.k_scale, float("inf")),
                         (pg.v_scale, -1.0)):
        keep = which.clone()
        which[page[3]] = value
        kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, out, ws)
        assert_status(kt, ws, kt.KT_ERR_DEVICE_CHECK)
        check_attention(pg, q, out, lambda b, h: [0, 1, 2, 4, 5, 6], G)
        which.copy_(keep)
    # a page outside the pool
    pg.table[0, 4] = pg.k_code.shape[0]
    kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, out, ws)
    assert_status(kt, ws, kt.KT_ERR_DEVICE_CHECK)
    check_attention(pg, q, out, lambda b, h: [0, 1, 2, 3, 5, 6], G)


@pytest.mark.parametrize("G", [1, 3, 4, 8])
@pytest.mark.parametrize("exps", [[17], [20], [23], [24], [26], [30], [30, -30, 8, 22, 0]])
def test_large_scores(kt, G, exps):
    """K scales up to 2^30: scores so large that one token takes all of the weight.

    A score errs by 8 * 2^-23 of sum |q k| (eight truncated steps of the tensor core), one of
    them and the maximum by 2^-24 each where they are rounded; where the best is ahead of the next by
    64 more than twice that (in base 2), the others' weights are below 2^-64 and the output is the
    best token's V: a product in units of the block's scale (exact, P in two parts 2^-22), and one
    division, 2^-20 in all.  Elsewhere it stays among the values of V."""
    H, lens = 2, [128 * 7 + 9, 300]
    pg = filled(kt, lens, H, 63)
    for b in range(2):
        for j in range(8):
            pg.k_scale[int(pg.host.table[b, j])] = 2.0 ** exps[j % len(exps)]
    pg.host.scale["k"] = pg.k_scale.cpu().double().numpy()
    q = torch.randn(2, H * G, 128).half().cuda()
    p = kt.sparse_params(H * G, 8, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SEPARATE)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    pool = reps_pool(kt, pg, p)
    kt.kt_build_block_reps_f8(pg.kv, p, 0, 8, pool)
    sel = torch.zeros(2, H, 1, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(2, H, dtype=torch.int32, device="cuda")
    dense, step, given = (torch.empty(2, H * G, 128, device="cuda") for _ in "abc")
    kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, dense, ws)
    kt.kt_sparse_decode_step_f8(q, pg.kv, pool, p, sel, cnt, step, ws)  # every block is Initial
    kt.kt_sparse_decode_attn_f8(q, pg.kv, p, sel, cnt, given, ws)
    assert (cnt == 0).all()
    assert_status(kt, ws)
    clear = 0
    for out in (dense, step, given):
        got = out.cpu().double().numpy()
        for b, n in enumerate(lens):
            for h in range(H):
                k, v = (np.concatenate([pg.host.values(s, int(pg.host.table[b, j]), h)
                                        for j in range(-(-n // 128))])[:n] for s in "kv")
                for i in range(h * G, h * G + G):
                    x = q[b, i].cpu().double().numpy()
                    base2 = SCALE * 1.4426950408889634
                    s, err = k @ x * base2, np.abs(k) @ np.abs(x) * base2 * 10 * 2.0 ** -23
                    best = s.argmax()
                    assert (np.abs(got[b, i]) <= np.abs(v).max(0) * (1 + 2.0 ** -20)).all()
                    if (s[best] - err[best] - np.delete(s + err, best)).min() >= 64:
                        clear += 1
                        assert (np.abs(got[b, i] - v[best]) <= np.abs(v[best]) * 2.0 ** -20 +
                                np.abs(v).max(0) * 2.0 ** -50).all(), (b, i)
    assert clear >= (3 * 2 * H * G * 3) // 4


@pytest.mark.parametrize("rep,stride", [(0, 1), (1, 1), (2, 1), (3, 1), (3, 16), (3, 128)])
def test_reps_of_scales_from_elsewhere(kt, rep, stride):
    """Representatives of blocks whose scales the append does not write, from 2^-30 to 2^30: those
    of the values read back (code * scale in binary32), bit for bit, saturating in binary16; the
    Mean rounded once.  The step over such blocks selects as the selection call does."""
    H, G, blocks = 2, 4, 24
    p = kt.sparse_params(H * G, 1, 1, 4, rep, kt.KT_HEAD_SEPARATE, fix_stride=stride)
    pg = filled(kt, [128 * blocks], H, 62, params=p)
    rng = np.random.default_rng(3)
    scale = 2.0 ** rng.uniform(-30, 30, pg.k_scale.shape)
    own = [0.3, 2.0 ** -30, 2.0 ** -26, 2.0 ** -15, 1.0, 256.0, 512.0, 65520.0, 2.0 ** 30, 146.25]
    scale[[int(x) for x in pg.table[0, :len(own)].cpu()]] = np.array(own)[:, None]
    scale = scale.astype(np.float32)
    pg.k_scale.copy_(torch.from_numpy(scale))
    pg.k_code[int(pg.table[0, 5])] = 0  # zeros under 256, and under 2^30
    pg.k_code[int(pg.table[0, 8]), 0] = 0
    pool = reps_pool(kt, pg, p)
    kt.kt_build_block_reps_f8(pg.kv, p, 0, blocks, pool)
    rows = {0: 1, 1: 1, 2: 2, 3: 128 // stride}[rep]
    got = pool.cpu().numpy().view(np.float32 if rep == 1 else np.float16)
    got = got.reshape(pg.k_code.shape[0], H, rows, 128)
    code = pg.k_code.cpu().numpy()
    back = torch.empty(128 * blocks, H, 128, dtype=torch.float32, device="cuda")
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    kt.kt_read_kv_f8(pg.kv, torch.tensor([0, 128 * blocks], dtype=torch.int32, device="cuda"),
                     back, None, ws)
    back = back.cpu().numpy().reshape(blocks, 128, H, 128)
    for j in range(blocks):
        page = int(pg.host.table[0, j])
        for h in range(H):
            x = f8_ref.decode(code[page, h]).astype(np.float32) * scale[page, h]
            assert np.array_equal(x, back[j, :, h])
            if rep == 1:  # the sum is exact in 64 bits, and so is its product with the scale
                s = f8_ref.decode(code[page, h]).sum(0) / 128.0 * np.float64(scale[page, h])
                want = s.astype(np.float32)[None]
            else:
                x = {0: x.max(0, keepdims=True), 2: np.stack([x.min(0), x.max(0)]),
                     3: x[::stride]}[rep]
                want = np.clip(x, -65504.0, 65504.0).astype(np.float16)
            assert np.array_equal(got[page, h], want), (j, h)
    assert np.isfinite(got[[int(x) for x in pg.host.table[0]]]).all()
    # the step, with scales of one order
    scale = rng.uniform(0.01, 0.011, scale.shape).astype(np.float32)
    pg.k_scale.copy_(torch.from_numpy(scale))
    kt.kt_build_block_reps_f8(pg.kv, p, 0, blocks, pool)
    q = torch.randn(1, H * G, 128).half().cuda()
    sel = torch.zeros(1, H, 4, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(1, H, dtype=torch.int32, device="cuda")
    out = torch.empty(1, H * G, 128, device="cuda")
    kt.kt_sparse_decode_step_f8(q, pg.kv, pool, p, sel, cnt, out, ws)
    sel16, cnt16 = torch.zeros_like(sel), torch.zeros_like(cnt)
    kt.kt_score_select_blocks_f8(q, pg.kv, pool, p, sel16, cnt16, None, ws)
    assert torch.equal(sel.sort(-1)[0], sel16.sort(-1)[0]) and (cnt == 4).all()
    pg.host.code["k"], pg.host.scale["k"] = code, scale.astype(np.float64)
    hs, hc = sel.cpu(), cnt.cpu()
    check_attention(pg, q, out, lambda b, h: chosen(kt, pg, hs, hc, p, b, h), G)
    assert_status(kt, ws)


@pytest.mark.parametrize("rep,stride", [(0, 1), (1, 1), (2, 1), (3, 8), (3, 128)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_reps_of_nan_keys(kt, rep, stride, dtype):
    """A channel with a NaN key has NaN for its representative (Fix: the row's own), whether the
    append builds it, over one call or two, or kt_build_block_reps_f8; other channels, heads and
    sequences are as without it, and their attention is."""
    H, G, lens = 2, 4, [128 * 6 + 5, 128 * 4]
    p = kt.sparse_params(H * G, 1, 1, 2, rep, kt.KT_HEAD_SEPARATE, fix_stride=stride)
    rng = torch.Generator().manual_seed(9)
    m = sum(lens)
    k, v = rows_of(rng, m, H, dtype, 4.0), rows_of(rng, m, H, dtype, 4.0)
    k[3, 0, 7] = float("nan")                   # one value, in the block's first warp
    k[127, 0, 64] = -float("nan")               # and in its last
    k[128:256, 0, 9] = float("nan")             # a channel through a block
    k[256 + 40, 0] = float("nan")               # a row
    k[lens[0] + 200, 0, 1] = float("inf")       # no NaN: the largest code
    for first in (0, 128 * 2 + 40):             # in one call, and split inside a block
        pg = Paged(kt, [0, 0], H, 7, 12)
        ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
        pool, done = reps_pool(kt, pg, p), []
        parts = [[0, 0], lens] if first == 0 else [[first, 0], [lens[0] - first, lens[1]]]
        at = [0, lens[0]]
        for counts in parts:
            rows = torch.cat([torch.arange(a, a + n) for a, n in zip(at, counts)]).cuda()
            at = [a + n for a, n in zip(at, counts)]
            cu = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
            kt.kt_append_kv_f8(pg.kv, p, k[rows], v[rows], ws, cu_tokens=cu, reps_pool=pool)
            done += pg.host.append(host16(k[rows]), host16(v[rows]), counts)
        pg.check()
        again = reps_pool(kt, pg, p)
        kt.kt_build_block_reps_f8(pg.kv, p, 0, 7, again)
        rows = {0: 1, 1: 1, 2: 2, 3: 128 // stride}[rep]
        for t in (pool, again):
            got = t.cpu().numpy().view(np.float32 if rep == 1 else np.float16)
            got = got.reshape(-1, H, rows, 128)
            assert len(done) == 10
            for b, j in done:
                page = int(pg.host.table[b, j])
                for h in range(H):
                    want = pg.host.reps(page, h, rep, stride).astype(got.dtype)
                    assert np.array_equal(got[page, h], want, equal_nan=True), (b, j, h)
        if rep != 3:
            page = int(pg.host.table[0, 0])
            assert np.isnan(got[page, 0]).sum() == 2 * rows
    q = torch.randn(2, H * G, 128).half().cuda()
    sel = torch.zeros(2, H, 2, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(2, H, dtype=torch.int32, device="cuda")
    out = torch.empty(2, H * G, 128, device="cuda")
    kt.kt_sparse_decode_step_f8(q, pg.kv, pool, p, sel, cnt, out, ws)
    hs, hc = sel.cpu(), cnt.cpu()
    assert (hc == 2).all()
    assert torch.isnan(out[0, :G]).all()        # block 0 is an Initial one
    out[0, :G] = 0.0
    check_attention(pg, q, out, lambda b, h: chosen(kt, pg, hs, hc, p, b, h) if b or h else [], G)
    assert_status(kt, ws)


def test_offsets_beyond_32_bits(kt):
    """Pools of 5.2 GB, the sequence's pages at their end."""
    H, G, pages = 8, 2, 40000
    code = [torch.zeros(pages, H, 128, 128, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.ones(pages, H, device="cuda") for _ in "kv"]
    table = torch.tensor([[39999, 3, 39990, 32770]], dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = kt.paged_kv_f8(code[0], scale[0], code[1], scale[1], table, lens)
    p = kt.sparse_params(H * G, 1, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, kv, p)
    n = 400
    k, v = torch.randn(n, H, 128).half().cuda(), torch.randn(n, H, 128).half().cuda()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pool = torch.zeros(kt.kt_reps_pool_bytes_f8(kv, p), dtype=torch.uint8, device="cuda")
    kt.kt_append_kv_f8(kv, p, k, v, ws, cu_tokens=cu, reps_pool=pool)
    small = Paged(kt, [0], H, 4, 3)
    small.host.append(host16(k), host16(v), [n])
    back = [torch.empty(n, H, 128, dtype=torch.float16, device="cuda") for _ in "kv"]
    kt.kt_read_kv_f8(kv, cu, back[0], back[1], ws)
    for side, out in zip("kv", back):
        want = np.concatenate([
            np.stack([small.host.values(side, int(small.host.table[0, j]), h)
                      for h in range(H)], 1) for j in range(4)])[:n]
        assert np.array_equal(out.double().cpu().numpy(), want)
    q = torch.randn(1, H * G, 128).half().cuda()
    out = torch.empty(1, H * G, 128, device="cuda")
    kt.kt_dense_decode_attn_f8(q, kv, H * G, SCALE, out, ws)
    check_attention(small, q, out, lambda b, h: range(4), G)
    sel = torch.zeros(1, 1, 1, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    kt.kt_sparse_decode_step_f8(q, kv, pool, p, sel, cnt, out, ws)
    hs, hc = sel.cpu(), cnt.cpu()
    check_attention(small, q, out, lambda b, h: chosen(kt, small, hs, hc, p, b, h), G)
    reps = pool.view(torch.float16).reshape(pages, H, 2, 128)
    for j in range(3):
        for h in range(H):
            want = small.host.reps(int(small.host.table[0, j]), h, 2).astype(np.float16)
            assert np.array_equal(reps[int(table[0, j]), h].cpu().numpy(), want)
    assert_status(kt, ws)


# ---- together ---------------------------------------------------------------------------
class Loop:
    """A decode loop over the 8-bit cache: rotate and append, then the step or the dense layer."""

    def __init__(self, kt, prompt, steps, seed, H=2, G=4, rep=2, mode=1):
        self.kt, self.H, self.G, self.B = kt, H, G, len(prompt)
        self.p = kt.sparse_params(H * G, 1, 1, 3, rep, mode)
        self.pg = Paged(kt, [0] * self.B, H, -(-(max(prompt) + steps) // 128), seed)
        self.ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, self.pg.kv, self.p)
        self.pool = reps_pool(kt, self.pg, self.p)
        self.pool.zero_()
        self.rope = kt.rope(128, theta=1e6)
        rng = torch.Generator().manual_seed(seed)
        self.prompt = list(prompt)
        self.first = rows_of(rng, sum(prompt), (G + 2) * H, "bf16")
        self.rows = [rows_of(rng, self.B, (G + 2) * H, "bf16") for _ in range(steps)]
        self.x = torch.empty_like(self.rows[0])
        self.q = torch.empty(self.B, H * G, 128, dtype=torch.float16, device="cuda")
        U = 1 if mode == 0 else H
        self.sel = torch.zeros(self.B, U, 3, dtype=torch.int32, device="cuda")
        self.cnt = torch.zeros(self.B, U, dtype=torch.int32, device="cuda")
        self.out = torch.empty(self.B, H * G, 128, device="cuda")
        self.dense = torch.empty_like(self.out)

    def split(self, x):
        n = self.H * self.G
        return x[:, :n], x[:, n:n + self.H], x[:, n + self.H:]

    def prefill(self):
        q, k, v = self.split(self.first)
        cu = torch.tensor(np.cumsum([0] + self.prompt), dtype=torch.int32, device="cuda")
        self.kt.kt_append_kv_f8(self.pg.kv, self.p, k, v, self.ws, rope=self.rope, cu_tokens=cu,
                                reps_pool=self.pool)

    def step(self):
        kt, pg = self.kt, self.pg
        q, k, v = self.split(self.x)
        kt.kt_append_kv_f8(pg.kv, self.p, k, v, self.ws, rope=self.rope, q=q, q_out=self.q,
                           reps_pool=self.pool)
        kt.kt_sparse_decode_step_f8(self.q, pg.kv, self.pool, self.p, self.sel, self.cnt, self.out,
                                    self.ws)
        kt.kt_dense_decode_attn_f8(self.q, pg.kv, self.H * self.G, SCALE, self.dense, self.ws)

    def state(self):
        return [self.out.clone(), self.dense.clone(), self.sel.clone(), self.q.clone(),
                self.pg.lens.clone(), self.pg.k_code.clone(), self.pool.clone()]


def test_decode_loop(kt):
    """From prompts of one token to several blocks, over block borders; every step against the
    reference over the cache as read on the host, every tenth in full."""
    lp = Loop(kt, [700, 1, 255, 640], 135, 71)
    lp.prefill()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    f, amp = f8_ref.frequencies(128, 1e6)
    for t, row in enumerate(lp.rows):
        lp.x.copy_(row)
        lp.step()
        n = [m + t + 1 for m in lp.prompt]
        assert lp.pg.lens.tolist() == n
        if t % 10 and t + 1 < len(lp.rows):
            continue
        pg = lp.pg
        pos = np.array(n) - 1
        check_rope(lp.q, lp.split(row)[0], pos, f, amp, "half")
        pg.host = f8_ref.Cache(pg.k_code.cpu().numpy(), pg.k_scale.cpu().numpy(),
                               pg.v_code.cpu().numpy(), pg.v_scale.cpu().numpy(),
                               pg.table.cpu().numpy(), pg.lens.cpu().numpy())
        hs, hc = lp.sel.cpu(), lp.cnt.cpu()
        check_attention(pg, lp.q, lp.out, lambda b, h: chosen(kt, pg, hs, hc, lp.p, b, h), lp.G)
        check_attention(pg, lp.q, lp.dense, lambda b, h: range(-(-n[b] // 128)), lp.G)
        # the newest token's V, read back, is its row within half a step of its block's scale
        cu = torch.arange(lp.B + 1, dtype=torch.int32, device="cuda")
        back = torch.empty(lp.B, lp.H, 128, dtype=torch.float16, device="cuda")
        kt.kt_read_kv_f8(pg.kv, cu, None, back, ws, first=pg.lens - 1)
        v = lp.split(row)[2].half().float()
        for b in range(lp.B):
            s = pg.v_scale[int(pg.host.table[b, pos[b] // 128])][:, None]
            assert ((back[b].float() - v[b]).abs() <= v[b].abs() * 2.0 ** -4 + s * 2.0 ** -10).all()
    check_reps_of_loop(kt, lp)
    assert_status(kt, lp.ws)
    assert_status(kt, ws)


def check_reps_of_loop(kt, lp):
    want = reps_pool(kt, lp.pg, lp.p)
    want.zero_()
    kt.kt_build_block_reps_f8(lp.pg.kv, lp.p, 0, 100, want)
    assert torch.equal(want, lp.pool)


def test_decode_loop_captured(kt):
    """A captured step replayed over a block border gives the eager loop's results; a second
    captured loop with a workspace of its own, replayed in turn, does not disturb it."""
    a, b, c = (Loop(kt, [250, 130], 12, s) for s in (81, 82, 81))
    a.prefill(), b.prefill(), c.prefill()
    graphs = []
    for lp in (a, b):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            lp.step()
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(g)
    for t in range(12):
        for lp, g in zip((a, b), graphs):
            lp.x.copy_(lp.rows[t])
            g.replay()
        c.x.copy_(c.rows[t])
        c.step()
        for x, y in zip(a.state(), c.state()):
            assert torch.equal(x, y)
    assert a.pg.lens.tolist() == [262, 142]
    for lp in (a, b, c):
        assert_status(kt, lp.ws)


def test_two_streams(kt):
    """Two loops on two streams at once, each with its cache and workspace."""
    loops = [Loop(kt, [300, 64], 8, s) for s in (91, 92)]
    want = []
    for s in (91, 92):
        lp = Loop(kt, [300, 64], 8, s)
        lp.prefill()
        for row in lp.rows:
            lp.x.copy_(row)
            lp.step()
        want.append(lp.state())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lp, st in zip(loops, streams):
        with torch.cuda.stream(st):
            lp.prefill()
    for t in range(8):
        for lp, st in zip(loops, streams):
            with torch.cuda.stream(st):
                lp.x.copy_(lp.rows[t])
                lp.step()
    torch.cuda.synchronize()
    for lp, w in zip(loops, want):
        for x, y in zip(lp.state(), w):
            assert torch.equal(x, y)


def test_decode_layer(kt):
    """The layer call makes the dense, selecting and reusing calls' results."""
    H, G, lens = 2, 4, [128 * 9 + 3, 500]
    p = kt.sparse_params(H * G, 1, 1, 2, kt.KT_REP_MEAN, kt.KT_HEAD_SEPARATE)
    pg = filled(kt, lens, H, 95, params=p)
    pool = reps_pool(kt, pg, p)
    kt.kt_build_block_reps_f8(pg.kv, p, 0, 100, pool)
    pol = kt.reuse_policy(4, dense_layer_num=1, layer_step=2, token_step=2)
    slots = kt.kt_decode_history_slots(pol)
    hist = torch.zeros(slots, 2, H, 2, dtype=torch.int32, device="cuda")
    cnts = torch.zeros(slots, 2, H, dtype=torch.int32, device="cuda")
    ws = kt.workspace_f8(kt.KT_OP_SPARSE_STEP, pg.kv, p)
    for token in range(3):
        for layer in range(4):
            q = torch.randn(2, H * G, 128).half().cuda()
            out, want = torch.empty(2, H * G, 128, device="cuda"), torch.empty(2, H * G, 128,
                                                                               device="cuda")
            action, slot = kt.kt_decode_layer_action(pol, token, layer)
            old = hist[slot].clone()
            kt.kt_decode_layer_f8(pol, token, layer, q, pg.kv, pool, p, hist, cnts, out, ws)
            if action == kt.KT_LAYER_DENSE:
                kt.kt_dense_decode_attn_f8(q, pg.kv, H * G, SCALE, want, ws)
            elif action == kt.KT_LAYER_SELECT:
                sel, cnt = torch.zeros_like(old), torch.zeros_like(cnts[0])
                kt.kt_sparse_decode_step_f8(q, pg.kv, pool, p, sel, cnt, want, ws)
                assert torch.equal(sel, hist[slot]) and torch.equal(cnt, cnts[slot])
            else:
                kt.kt_sparse_decode_attn_f8(q, pg.kv, p, hist[slot], cnts[slot], want, ws)
                assert torch.equal(old, hist[slot])
            assert torch.equal(out, want)
    assert_status(kt, ws)


def test_status_of_the_c_calls(kt):
    """The C entry points return their status; nothing is written where they refuse."""
    pg = filled(kt, [10], 1, 97)
    before = pg.k_code.clone()
    r = kt.rows(torch.zeros(1, 1, 128, dtype=torch.float16, device="cuda"))
    p = kt.sparse_params(1, 1, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    st = kt.lib.kt_append_kv_f8(ctypes.byref(pg.kv), ctypes.byref(p), None, None, None,
                                ctypes.byref(r), ctypes.byref(r), None, 2, None, None,
                                pg.lens.data_ptr(), 256, None)
    assert st == kt.KT_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(pg.k_code, before) and pg.lens.tolist() == [10]
