"""Host-only checks of the rotary positions and the 8-bit cache: the table of
frequencies against its formulas, and the refusals of every call (made before
the device is touched).  The reference implementation is checked here too."""
import ctypes
import math

import numpy as np
import pytest

import block_sparse_long_quest_gb300 as kt
import f8_ref

FAKE = 0x100000  # aligned, never dereferenced: validation fails before any launch
FAR = 0x10000000  # another one, far from it


# ---- the reference itself ---------------------------------------------------------------
def test_reference_codes_are_the_e4m3_grid():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, f8_ref.TABLE, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=5000) * 10.0 ** rng.uniform(-4, 2, 5000), f8_ref.GRID,
                        (f8_ref.GRID[1:] + f8_ref.GRID[:-1]) / 2, [-0.0, 448.0, -448.0]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    ok = np.abs(x) <= 448
    assert np.array_equal(f8_ref.encode(x)[ok], want[ok])
    assert f8_ref.encode(np.array([1e9, -np.inf, np.nan])).tolist() == [0x7E, 0xFE, 0x7F]


def test_reference_scale_is_the_least():
    for a in (0.0, 1e-7, 0.0136, 0.01368, 447.9, 448.0, 448.25, 57344.0, 65504.0):
        s = f8_ref.block_scale(a)
        assert a <= 448 * s or s == 256
        assert s == 2.0 ** -15 or a > 448 * s / 2


# ---- frequencies ------------------------------------------------------------------------
SCALINGS = {"plain": kt.KT_ROPE_PLAIN, "linear": kt.KT_ROPE_LINEAR, "ntk": kt.KT_ROPE_NTK,
            "yarn": kt.KT_ROPE_YARN, "bands": kt.KT_ROPE_BANDS}


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("rot,theta", [(128, 1e4), (128, 5e7), (64, 1e6), (6, 2.0), (4, 1e4)])
def test_frequencies(scaling, rot, theta):
    factor = 1.0 if scaling == "plain" else 8.0
    fast = 4.0 if scaling == "bands" else 32.0
    r = kt.rope(rot, theta=theta, scaling=SCALINGS[scaling], factor=factor, original_len=8192,
                beta_fast=fast, beta_slow=1.0, layout=kt.KT_ROPE_PAIRS)
    f, amp = f8_ref.frequencies(rot, theta, scaling, factor, 8192, fast, 1.0)
    want = (f / f8_ref.PI2 * np.longdouble(2.0) ** 64).astype(np.float64)
    got = np.array([float(v) for v in r.phase], dtype=np.float64)
    assert (np.abs(got[:rot // 2] - want) <= np.abs(want) * 2.0 ** -49 + 1).all()
    assert (got[rot // 2:] == 0).all()
    assert r.rotary_dim == rot and r.layout == kt.KT_ROPE_PAIRS
    assert abs(r.amplitude - amp) <= 2.0 ** -23 * amp


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=130), dict(rotary_dim=-2),
    dict(theta=1.0), dict(theta=math.nan), dict(theta=math.inf), dict(theta=-5.0),
    dict(factor=2.0), dict(scaling=kt.KT_ROPE_LINEAR, factor=0.5),
    dict(scaling=kt.KT_ROPE_LINEAR, factor=math.nan), dict(layout=2), dict(scaling=9),
    dict(scaling=kt.KT_ROPE_NTK, rotary_dim=2, factor=2.0),
    dict(scaling=kt.KT_ROPE_YARN, factor=2.0, original_len=0),
    dict(scaling=kt.KT_ROPE_YARN, factor=2.0, original_len=4096, beta_slow=0.0),
    dict(scaling=kt.KT_ROPE_BANDS, factor=2.0, original_len=4096, beta_fast=1.0),
    dict(scaling=kt.KT_ROPE_BANDS, factor=2.0, original_len=4096, beta_fast=math.inf),
])
def test_rope_init_refuses(kw):
    with pytest.raises(kt.KtError) as e:
        kt.rope(**{"rotary_dim": 128, **kw})
    assert e.value.status == kt.KT_ERR_INVALID_ARG


def test_rope_init_refuses_null():
    assert kt.lib.kt_rope_init(None, ctypes.byref(kt.Rope())) == kt.KT_ERR_INVALID_ARG
    assert kt.lib.kt_rope_init(ctypes.byref(kt.RopeParams()), None) == kt.KT_ERR_INVALID_ARG


# ---- refusals ---------------------------------------------------------------------------
def rows(data=FAKE, heads=8, stride=None, dtype=kt.KT_F16):
    return kt.Rows(data, heads * 128 if stride is None else stride, heads, dtype)


def ref(x):
    return None if x is None else ctypes.byref(x)


def apply(rope=None, pos=FAKE, tokens=4, q="default", q_out=FAR, k=None, k_out=None):
    rope = kt.rope() if rope is None else rope
    q = rows() if q == "default" else q
    return kt.lib.kt_apply_rope(ref(rope), pos, tokens, ref(q), q_out, ref(k), k_out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(pos=None), kt.KT_ERR_INVALID_ARG),
    (dict(pos=FAKE + 4), kt.KT_ERR_INVALID_ARG),
    (dict(tokens=-1), kt.KT_ERR_INVALID_ARG),
    (dict(q=None, q_out=None), kt.KT_ERR_INVALID_ARG),
    (dict(q_out=None), kt.KT_ERR_INVALID_ARG),
    (dict(q=None), kt.KT_ERR_INVALID_ARG),
    (dict(q_out=FAR + 8), kt.KT_ERR_INVALID_ARG),
    (dict(q=rows(data=FAKE + 2)), kt.KT_ERR_INVALID_ARG),
    (dict(q=rows(heads=0, stride=128)), kt.KT_ERR_INVALID_ARG),
    (dict(q=rows(heads=5000)), kt.KT_ERR_UNSUPPORTED),
    (dict(q=rows(stride=8 * 128 - 8)), kt.KT_ERR_INVALID_ARG),
    (dict(q=rows(stride=8 * 128 + 4)), kt.KT_ERR_INVALID_ARG),
    (dict(q=rows(dtype=3)), kt.KT_ERR_INVALID_ARG),
    (dict(k=rows(FAKE + (1 << 20)), k_out=FAR), kt.KT_ERR_INVALID_ARG),         # same output
    (dict(k=rows(FAKE + (1 << 20), dtype=kt.KT_F32), k_out=FAR + (1 << 20)),
     kt.KT_ERR_INVALID_ARG),                                                    # two types
    (dict(k=rows(FAR), k_out=FAR + (1 << 20)), kt.KT_ERR_INVALID_ARG),          # q_out is k
    (dict(q_out=FAKE + 256), kt.KT_ERR_INVALID_ARG),                            # shifted overlap
    (dict(q=rows(dtype=kt.KT_BF16), q_out=FAKE), kt.KT_ERR_INVALID_ARG),        # in place, bf16
    (dict(q=rows(stride=2048), q_out=FAKE), kt.KT_ERR_INVALID_ARG),             # in place, packed
    (dict(tokens=0), kt.KT_OK),
])
def test_apply_rope_refuses(kw, status):
    assert apply(**kw) == status


def test_apply_rope_refuses_a_broken_table():
    for field, value in (("rotary_dim", 0), ("rotary_dim", 7), ("rotary_dim", 256), ("layout", 5),
                         ("amplitude", math.nan)):
        r = kt.rope()
        setattr(r, field, value)
        assert apply(rope=r) == kt.KT_ERR_INVALID_ARG
    assert kt.lib.kt_apply_rope(None, FAKE, 1, ref(rows()), FAR, None, None, None) == \
        kt.KT_ERR_INVALID_ARG


def cache(**kw):
    d = dict(k_code=FAKE, k_scale=FAKE, v_code=FAKE, v_scale=FAKE, table=FAKE, lens=FAKE, batch=2,
             H_kv=8, head_dim=128, block=128, max_blocks=64, pages=128)
    d.update(kw)
    return kt.PagedKVF8(*d.values())


def params(**kw):
    d = dict(num_q_heads=32, initial_blocks=1, local_blocks=4, top_k=8, rep=kt.KT_REP_QUEST,
             head_mode=kt.KT_HEAD_SHARED)
    d.update(kw)
    return kt.sparse_params(**d)


BAD_CACHE = [
    (dict(k_code=None), kt.KT_ERR_INVALID_ARG), (dict(v_code=None), kt.KT_ERR_INVALID_ARG),
    (dict(k_scale=None), kt.KT_ERR_INVALID_ARG), (dict(v_scale=None), kt.KT_ERR_INVALID_ARG),
    (dict(k_scale=FAKE + 4), kt.KT_ERR_INVALID_ARG), (dict(k_code=FAKE + 8), kt.KT_ERR_INVALID_ARG),
    (dict(table=None), kt.KT_ERR_INVALID_ARG), (dict(lens=None), kt.KT_ERR_INVALID_ARG),
    (dict(batch=0), kt.KT_ERR_INVALID_ARG), (dict(head_dim=64), kt.KT_ERR_UNSUPPORTED),
    (dict(block=64), kt.KT_ERR_UNSUPPORTED), (dict(batch=300), kt.KT_ERR_UNSUPPORTED),
    (dict(pages=0), kt.KT_ERR_INVALID_ARG),
]


def append(c="default", p="default", rope=None, q=None, q_out=None, k="default", v="default", cu=FAKE,
           tokens=4, new_lens=FAR, reps=None, ws=FAKE, ws_bytes=256):
    c = cache() if c == "default" else c
    p = params() if p == "default" else p
    k = rows() if k == "default" else k
    v = rows() if v == "default" else v
    return kt.lib.kt_append_kv_f8(ref(c), ref(p), ref(rope), ref(q), q_out, ref(k), ref(v), cu,
                                  tokens, new_lens, reps, ws, ws_bytes, None)


def every_call(c, p):
    n = ctypes.c_size_t(0)
    L = kt.lib
    big = 1 << 40
    return {
        "bytes": lambda: L.kt_workspace_bytes_f8(kt.KT_OP_SPARSE_STEP, ref(c), ref(p),
                                                 ctypes.byref(n)),
        "reps": lambda: L.kt_build_block_reps_f8(ref(c), ref(p), 0, 1, FAKE, None),
        "append": lambda: append(c, p),
        "read": lambda: L.kt_read_kv_f8(ref(c), None, FAKE, 4, kt.KT_F16, FAR, None, FAKE, 256,
                                        None),
        "sparse": lambda: L.kt_sparse_decode_attn_f8(FAKE, ref(c), ref(p), FAKE, FAKE, FAKE, FAKE,
                                                     big, None),
        "dense": lambda: L.kt_dense_decode_attn_f8(FAKE, ref(c), 32, 0.1, FAKE, FAKE, big, None),
        "select": lambda: L.kt_score_select_blocks_f8(FAKE, ref(c), FAKE, ref(p), FAKE, FAKE,
                                                      None, FAKE, big, None),
        "step": lambda: L.kt_sparse_decode_step_f8(FAKE, ref(c), FAKE, ref(p), FAKE, FAKE, FAKE,
                                                   FAKE, big, None),
        "layer": lambda: L.kt_decode_layer_f8(ctypes.byref(kt.reuse_policy(4)), 0, 1, FAKE, ref(c),
                                              FAKE, ref(p), FAKE, FAKE, FAKE, FAKE, big, None),
    }


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_every_call_refuses_a_bad_cache(kw, status):
    for name, call in every_call(cache(**kw), params()).items():
        assert call() == status, name


def test_every_call_refuses_no_cache():
    for name, call in every_call(None, params()).items():
        assert call() == kt.KT_ERR_INVALID_ARG, name


@pytest.mark.parametrize("kw,status", [
    (dict(num_q_heads=30), kt.KT_ERR_INVALID_ARG), (dict(num_q_heads=72), kt.KT_ERR_UNSUPPORTED),
    (dict(top_k=0), kt.KT_ERR_INVALID_ARG), (dict(local_blocks=0), kt.KT_ERR_UNSUPPORTED),
])
def test_every_call_refuses_bad_parameters(kw, status):
    for name, call in every_call(cache(), params(**kw)).items():
        if name in ("read", "dense"):
            continue
        want = kt.KT_ERR_INVALID_ARG if name == "layer" and kw.get("top_k") == 0 else status
        assert call() == want, name


def test_dynamic_reps_are_refused():
    p = params(rep=kt.KT_REP_DYNAMIC)
    calls = every_call(cache(), p)
    for name in ("reps", "select", "step", "layer"):
        assert calls[name]() == kt.KT_ERR_INVALID_ARG, name
    assert kt.kt_reps_pool_bytes_f8(cache(), p) == 0
    n = ctypes.c_size_t(0)
    for op in (kt.KT_OP_DYNAMIC_REPS, kt.KT_OP_PRESELECT):
        assert kt.lib.kt_workspace_bytes_f8(op, ref(cache()), ref(params()), ctypes.byref(n)) == \
            kt.KT_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), kt.KT_ERR_INVALID_ARG), (dict(v=None), kt.KT_ERR_INVALID_ARG),
    (dict(k=rows(heads=4)), kt.KT_ERR_INVALID_ARG), (dict(v=rows(heads=16)), kt.KT_ERR_INVALID_ARG),
    (dict(v=rows(dtype=kt.KT_F32)), kt.KT_ERR_INVALID_ARG),
    (dict(k=rows(data=FAKE + 4)), kt.KT_ERR_INVALID_ARG),
    (dict(k=rows(stride=100)), kt.KT_ERR_INVALID_ARG),
    (dict(q=rows(heads=32)), kt.KT_ERR_INVALID_ARG), (dict(q_out=FAR), kt.KT_ERR_INVALID_ARG),
    (dict(q=rows(heads=16), q_out=FAR), kt.KT_ERR_INVALID_ARG),
    (dict(q=rows(heads=32, dtype=kt.KT_BF16), q_out=FAR), kt.KT_ERR_INVALID_ARG),
    (dict(q=rows(heads=32), q_out=FAR + 4), kt.KT_ERR_INVALID_ARG),
    (dict(q=rows(FAR, heads=32), q_out=FAKE), kt.KT_ERR_INVALID_ARG),      # q_out over k and v
    (dict(q=rows(FAR, heads=32), q_out=FAR + 16), kt.KT_ERR_INVALID_ARG),  # shifted overlap
    (dict(ws=None), kt.KT_ERR_INVALID_ARG), (dict(ws_bytes=255), kt.KT_ERR_INVALID_ARG),
    (dict(ws=FAKE + 8), kt.KT_ERR_INVALID_ARG), (dict(cu=FAKE + 4), kt.KT_ERR_INVALID_ARG),
    (dict(new_lens=FAR + 4), kt.KT_ERR_INVALID_ARG), (dict(reps=FAR + 4), kt.KT_ERR_INVALID_ARG),
    (dict(tokens=-1), kt.KT_ERR_INVALID_ARG), (dict(cu=None), kt.KT_ERR_INVALID_ARG),
    (dict(c=cache(batch=16), new_lens=FAKE + 16), kt.KT_ERR_INVALID_ARG),  # half over seq_lens
])
def test_append_refuses(kw, status):
    assert append(**kw) == status


def test_append_refuses_a_broken_table():
    r = kt.rope()
    r.rotary_dim = 1
    assert append(rope=r) == kt.KT_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(cu=None), dict(cu=FAKE + 4), dict(first=FAKE + 4), dict(tokens=-1), dict(dtype=3),
    dict(k=None, v=None), dict(k=FAR + 8), dict(v=FAR + 8), dict(ws=None), dict(ws_bytes=64),
    dict(ws=FAKE + 2), dict(v=FAR + 1024), dict(v=FAR),
])
def test_read_refuses(kw):
    d = dict(c=cache(), first=None, cu=FAKE, tokens=4, dtype=kt.KT_F16, k=FAR, v=FAR + (1 << 20),
             ws=FAKE, ws_bytes=256)
    d.update(kw)
    assert kt.lib.kt_read_kv_f8(ref(d["c"]), d["first"], d["cu"], d["tokens"], d["dtype"], d["k"],
                                d["v"], d["ws"], d["ws_bytes"], None) == kt.KT_ERR_INVALID_ARG


def test_attention_refuses():
    L, c, p, big = kt.lib, ref(cache()), ref(params()), 1 << 40
    inv, small = kt.KT_ERR_INVALID_ARG, kt.KT_ERR_WORKSPACE_TOO_SMALL
    assert L.kt_sparse_decode_attn_f8(None, c, p, FAKE, FAKE, FAKE, FAKE, big, None) == inv
    assert L.kt_sparse_decode_attn_f8(FAKE, c, p, None, FAKE, FAKE, FAKE, big, None) == inv
    assert L.kt_sparse_decode_attn_f8(FAKE, c, p, FAKE, None, FAKE, FAKE, big, None) == inv
    assert L.kt_sparse_decode_attn_f8(FAKE, c, p, FAKE, FAKE, None, FAKE, big, None) == inv
    assert L.kt_sparse_decode_attn_f8(FAKE, c, p, FAKE, FAKE, FAKE, None, big, None) == inv
    assert L.kt_sparse_decode_attn_f8(FAKE, c, p, FAKE, FAKE, FAKE, FAKE, 512, None) == small
    assert L.kt_dense_decode_attn_f8(FAKE + 2, c, 32, 0.1, FAKE, FAKE, big, None) == inv
    assert L.kt_dense_decode_attn_f8(FAKE, c, 33, 0.1, FAKE, FAKE, big, None) == inv
    assert L.kt_dense_decode_attn_f8(FAKE, c, 32, 0.0, FAKE, FAKE, big, None) == inv
    assert L.kt_dense_decode_attn_f8(FAKE, c, 32, math.inf, FAKE, FAKE, big, None) == inv
    assert L.kt_dense_decode_attn_f8(FAKE, c, 32, 0.1, FAKE, FAKE, 512, None) == small
    assert L.kt_sparse_decode_step_f8(FAKE, c, None, p, FAKE, FAKE, FAKE, FAKE, big, None) == inv
    assert L.kt_sparse_decode_step_f8(FAKE, c, FAKE, p, FAKE, FAKE, FAKE, FAKE, 512, None) == small
    assert L.kt_build_block_reps_f8(c, p, -1, 1, FAKE, None) == inv
    assert L.kt_build_block_reps_f8(c, p, 0, -1, FAKE, None) == inv
    assert L.kt_build_block_reps_f8(c, p, 0, 1, None, None) == inv
    assert L.kt_build_block_reps_f8(c, p, 0, 0, FAKE, None) == kt.KT_OK
    assert L.kt_build_block_reps_f8(c, p, 64, 5, FAKE, None) == kt.KT_OK  # behind the table


def test_attention_refuses_more_blocks_than_it_counts():
    wide = cache(batch=16, H_kv=8, max_blocks=(1 << 23))
    calls = every_call(wide, params())
    for name in ("sparse", "dense", "step"):
        assert calls[name]() == kt.KT_ERR_UNSUPPORTED, name


def test_sizes_are_those_of_the_binary16_cache():
    c, p = cache(), params()
    same = kt.PagedKV(FAKE, FAKE, FAKE, FAKE, 2, 8, 128, 128, 64, 128)
    for op in (kt.KT_OP_SCORE_SELECT, kt.KT_OP_SPARSE_ATTN, kt.KT_OP_DENSE_ATTN,
               kt.KT_OP_SPARSE_STEP):
        assert kt.kt_workspace_bytes_f8(op, c, p) == kt.kt_workspace_bytes(op, same, p)
    assert kt.kt_reps_pool_bytes_f8(c, p) == kt.kt_reps_pool_bytes(same, p)


def test_binding_refuses_other_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8, 128, dtype=torch.float16)
    pos = torch.zeros(4, dtype=torch.int32)
    r = kt.rope()
    for q, out in ((x[..., :64], x), (x.transpose(0, 1), x), (x[..., ::2], x), (x, x[:, :4]),
                   (x[:3], x[:3]), (x, x.transpose(1, 2))):
        with pytest.raises(kt.KtError):
            kt.kt_apply_rope(r, pos, q, out, stream=0)
    with pytest.raises(kt.KtError):
        kt.kt_apply_rope(r, pos, x.double(), x, stream=0)
    with pytest.raises(kt.KtError):
        kt.kt_apply_rope(r, pos.long(), x, x, stream=0)
    with pytest.raises(kt.KtError):
        kt.kt_apply_rope(r, pos, x, x.bfloat16(), stream=0)
    with pytest.raises(kt.KtError):
        kt.kt_append_kv_f8(cache(), params(), x, x, x, cu_tokens=pos.long(), stream=0)
    with pytest.raises(kt.KtError):
        kt.kt_append_kv_f8(cache(), params(), x, x, x, new_lens=pos.float(), stream=0)
    with pytest.raises(kt.KtError):
        kt.kt_read_kv_f8(cache(), pos, x, None, x, first=pos.long(), stream=0)
    with pytest.raises(kt.KtError):
        kt.kt_read_kv_f8(cache(), pos, x.double(), None, x, stream=0)
    with pytest.raises(kt.KtError):
        kt.kt_append_kv_f8(cache(), params(), x, x[:3], x, stream=0)
    with pytest.raises(kt.KtError):
        kt.kt_read_kv_f8(cache(), pos, None, None, x, stream=0)
    with pytest.raises(kt.KtError):
        kt.kt_read_kv_f8(cache(), pos, x[:, :4], None, x, stream=0)


def test_binding_refuses_short_and_strided_index_tensors():
    """The kernels read batch + 1 offsets and batch lengths one behind the other: a tensor with
    fewer, or with gaps, is refused; a longer one (a padded buffer) is not."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8, 128, dtype=torch.float16)
    c, p, r = cache(batch=2), params(), kt.rope()
    ints = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731

    def refused(call):
        with pytest.raises(kt.KtError) as e:
            call()
        return e.value.status == kt.KT_ERR_INVALID_ARG

    assert refused(lambda: kt.kt_apply_rope(r, ints(8)[::2], x, x, stream=0))
    assert refused(lambda: kt.kt_apply_rope(r, ints(1).expand(4), x, x, stream=0))
    for bad in (ints(2), ints(6)[::2], ints(1).expand(3), ints(0)):
        assert refused(lambda: kt.kt_append_kv_f8(c, p, x, x, x, cu_tokens=bad, stream=0))
        assert refused(lambda: kt.kt_read_kv_f8(c, bad, x, None, x, stream=0))
    assert refused(lambda: kt.kt_read_kv_f8(c, None, x, None, x, stream=0))
    for bad in (ints(1), ints(4)[::2], ints(1).expand(2), ints(0)):
        assert refused(lambda: kt.kt_append_kv_f8(c, p, x, x, x, cu_tokens=ints(3), new_lens=bad,
                                                  stream=0))
        assert refused(lambda: kt.kt_read_kv_f8(c, ints(3), x, None, x, first=bad, stream=0))
    kt._check_int32(ints(9), 3, "a call")
    kt._check_int32(None, 3, "a call")


def test_binding_refuses_prepared_rows():
    """A kt_rows does not hold its number of tokens, which the calls check: only tensors are taken,
    and a kt_rows is refused like any other wrong argument."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8, 128, dtype=torch.float16)
    pos = torch.zeros(4, dtype=torch.int32)
    r, c, p = kt.rope(), cache(batch=4), params(num_q_heads=8)
    y = kt.rows(x)
    assert (y.stride, y.heads, y.dtype) == (8 * 128, 8, kt.KT_F16)
    for call in (lambda: kt.rows(y), lambda: kt.kt_apply_rope(r, pos, y, x, stream=0),
                 lambda: kt.kt_apply_rope(r, pos, k=y, k_out=x, stream=0),
                 lambda: kt.kt_append_kv_f8(c, p, y, x, x, stream=0),
                 lambda: kt.kt_append_kv_f8(c, p, x, y, x, stream=0),
                 lambda: kt.kt_append_kv_f8(c, p, x, x, x, q=y, q_out=x, stream=0)):
        with pytest.raises(kt.KtError) as e:
            call()
        assert e.value.status == kt.KT_ERR_INVALID_ARG
