"""Host-only checks of attention behind shared prefixes: every refusal is made before the device is
touched."""
import ctypes
import math

import pytest

import block_sparse_long_quest_gb300 as kt

FAKE = 0x100000  # aligned, never dereferenced
BIG = 1 << 40


def fake_kv(f8, **kw):
    shape = dict(batch=4, num_kv_heads=2, head_dim=128, block_size=128, max_blocks_per_seq=16,
                 num_pages=100)
    pools = ("k_code", "k_scale", "v_code", "v_scale") if f8 else ("k_pool", "v_pool")
    f = dict({n: FAKE for n in pools + ("block_table", "seq_lens")}, **shape)
    f.update(kw)
    kv = (kt.PagedKVF8 if f8 else kt.PagedKV)()
    for k, v in f.items():
        setattr(kv, k, v)
    return kv


def by(x):
    return None if x is None else ctypes.byref(x)


def need(f8, kv, heads=8):
    params = kt.sparse_params(heads, 0, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    return (kt.kt_workspace_bytes_f8 if f8 else kt.kt_workspace_bytes)(kt.KT_OP_PREFIX_ATTN, kv,
                                                                       params)


@pytest.fixture(params=[False, True], ids=["f16", "f8"])
def f8(request):
    return request.param


def call(f8, kv="", groups="", q=FAKE, heads=8, scale=0.1, out=FAKE, ws=FAKE, n=BIG):
    f = kt.lib.kt_prefix_decode_attn_f8 if f8 else kt.lib.kt_prefix_decode_attn
    kv = fake_kv(f8) if kv == "" else kv
    groups = kt.PrefixGroups(FAKE, FAKE, 3) if groups == "" else groups
    return f(q, by(kv), by(groups), heads, scale, out, ws, n, None)


def test_pointers(f8):
    assert call(f8, kv=None) == kt.KT_ERR_INVALID_ARG
    assert call(f8, groups=None) == kt.KT_ERR_INVALID_ARG
    for name in ("q", "out", "ws"):
        assert call(f8, **{name: None}) == kt.KT_ERR_INVALID_ARG
        assert call(f8, **{name: FAKE + 8}) == kt.KT_ERR_INVALID_ARG
    for i in range(2):
        for bad in (None, FAKE + 4):
            p = [FAKE, FAKE]
            p[i] = bad
            assert call(f8, groups=kt.PrefixGroups(*p, 3)) == kt.KT_ERR_INVALID_ARG
    pools = ("k_code", "k_scale", "v_code", "v_scale") if f8 else ("k_pool", "v_pool")
    for name in pools + ("block_table", "seq_lens"):
        assert call(f8, kv=fake_kv(f8, **{name: None})) == kt.KT_ERR_INVALID_ARG


def test_sizes(f8):
    for n in (0, -1):
        assert call(f8, groups=kt.PrefixGroups(FAKE, FAKE, n)) == kt.KT_ERR_INVALID_ARG
    assert call(f8, groups=kt.PrefixGroups(FAKE, FAKE, 2049)) == kt.KT_ERR_UNSUPPORTED
    for name in ("batch", "num_kv_heads", "max_blocks_per_seq", "num_pages"):
        assert call(f8, kv=fake_kv(f8, **{name: 0})) == kt.KT_ERR_INVALID_ARG
    assert call(f8, kv=fake_kv(f8, head_dim=64)) == kt.KT_ERR_UNSUPPORTED
    assert call(f8, kv=fake_kv(f8, block_size=64)) == kt.KT_ERR_UNSUPPORTED
    assert call(f8, kv=fake_kv(f8, batch=2049)) == kt.KT_ERR_UNSUPPORTED
    # blocks of all (sequence, head) beyond 2^30
    assert call(f8, kv=fake_kv(f8, batch=2048, num_kv_heads=8,
                               max_blocks_per_seq=65535)) == kt.KT_ERR_UNSUPPORTED
    for heads in (0, -8, 7):
        assert call(f8, heads=heads) == kt.KT_ERR_INVALID_ARG
    assert call(f8, heads=18) == kt.KT_ERR_UNSUPPORTED  # nine heads per KV head
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(f8, scale=scale) == kt.KT_ERR_INVALID_ARG


@pytest.mark.parametrize("batch,kv_heads,heads", [(1, 1, 1), (4, 2, 8), (64, 8, 32), (2048, 1, 8)])
def test_workspace(f8, batch, kv_heads, heads):
    kv = fake_kv(f8, batch=batch, num_kv_heads=kv_heads)
    size = need(f8, kv, heads)
    # the rows of every sequence, once behind a prefix and once behind their own blocks
    assert size >= 256 + 2 * batch * heads * 130 * 4
    assert call(f8, kv=kv, heads=heads, n=256) == kt.KT_ERR_WORKSPACE_TOO_SMALL
    assert call(f8, kv=kv, heads=heads, n=0) == kt.KT_ERR_WORKSPACE_TOO_SMALL


def test_binding_checks(f8):
    torch = pytest.importorskip("torch")
    good = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(kt.KtError):
        kt.prefix_groups(good[:3], good[:3])  # one bound too few
    with pytest.raises(kt.KtError):
        kt.prefix_groups(good.long(), good[:3])
    with pytest.raises(kt.KtError):
        kt.prefix_groups(torch.zeros(8, dtype=torch.int32)[::2], good[:3])
    g = kt.prefix_groups(good, good[:3])
    assert g.groups == 3 and g.cu_groups == good.data_ptr()
