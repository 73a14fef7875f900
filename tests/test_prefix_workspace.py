"""The workspace of attention behind shared prefixes: its region lies behind all state that the other
calls keep whatever their parameters, so workspaces of theirs are refused and one of its own serves
them."""
import random

import pytest

import block_sparse_long_quest_gb300 as kt
from test_prefix_host import call, fake_kv, need

OTHERS = (kt.KT_OP_SCORE_SELECT, kt.KT_OP_SPARSE_ATTN, kt.KT_OP_DENSE_ATTN, kt.KT_OP_SPARSE_STEP)


@pytest.fixture(params=[False, True], ids=["f16", "f8"])
def f8(request):
    return request.param


def bytes_of(f8, op, kv, params):
    return (kt.kt_workspace_bytes_f8 if f8 else kt.kt_workspace_bytes)(op, kv, params)


def some_params(rng, heads, blocks):
    return kt.sparse_params(heads, rng.choice([0, 1, 4]), rng.choice([1, 2, 9]),
                            rng.choice([1, 2, 32, 100, 255, 256, 1024]), kt.KT_REP_QUEST,
                            rng.choice([kt.KT_HEAD_SHARED, kt.KT_HEAD_SEPARATE]))


@pytest.mark.parametrize("batch", [1, 2, 3, 4, 8, 16])
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (8, 4), (2, 8)])
def test_workspaces_of_other_calls_are_refused(f8, batch, kv_heads, group):
    for blocks in (1, 16, 1024, 8192):
        kv = fake_kv(f8, batch=batch, num_kv_heads=kv_heads, max_blocks_per_seq=blocks)
        heads = kv_heads * group
        for op in OTHERS:
            for top_k in (1, 32, 1024):
                for mode in (kt.KT_HEAD_SHARED, kt.KT_HEAD_SEPARATE):
                    p = kt.sparse_params(heads, 0, 1, top_k, kt.KT_REP_QUEST, mode)
                    n = bytes_of(f8, op, kv, p)
                    assert call(f8, kv=kv, heads=heads, n=n) == kt.KT_ERR_WORKSPACE_TOO_SMALL
        n = need(f8, kv, heads)
        assert call(f8, kv=kv, heads=heads, n=n - 1) == kt.KT_ERR_WORKSPACE_TOO_SMALL


def test_its_region_is_behind_all_others(f8):
    """Of any shape and any parameters the size leaves room for at least the parts behind the
    regions of the decode step."""
    rng = random.Random(1)
    for _ in range(400):
        kv_heads, group = rng.choice([1, 2, 4, 8, 64]), rng.randint(1, 8)
        batch = rng.choice([1, 2, 5, 16, 2048 // kv_heads])
        blocks = rng.choice([1, 9, 300, 1024, 8191, 65000])
        if batch * kv_heads * (blocks + 2) > 0x3FFFFFFF:
            continue
        heads = kv_heads * group
        kv = fake_kv(f8, batch=batch, num_kv_heads=kv_heads, max_blocks_per_seq=blocks)
        size = need(f8, kv, heads)
        rows = 2 * 192 * min(batch * group, 128) + 2 * batch * heads
        for _ in range(6):
            p = some_params(rng, heads, blocks)
            assert bytes_of(f8, kt.KT_OP_PREFIX_ATTN, kv, p) == size
            assert size >= bytes_of(f8, kt.KT_OP_SPARSE_STEP, kv, p) + rows * 130 * 4


@pytest.mark.gpu
@pytest.mark.parametrize("top_k", [1, 16, 1024])
@pytest.mark.parametrize("batch", [1, 2, 3])
def test_steps_in_turn(batch, top_k):
    """A workspace sized with another top_k serves the decode step in turn with the attention behind
    prefixes, dense attention and (where it is large enough) the preselection."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_gpu_prefix import SCALE, Batch
    b = Batch(groups=[(20, [700, 300, 1200][:batch])], heads=2, group=4)
    b.upload(kt)
    p = kt.sparse_params(8, 1, 2, top_k, kt.KT_REP_QUEST, kt.KT_HEAD_SEPARATE)
    other = kt.sparse_params(8, 1, 2, 32, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    shared = kt.workspace(kt.KT_OP_PREFIX_ATTN, b.kv, other)
    large = torch.zeros(max(kt.kt_workspace_bytes(kt.KT_OP_PRESELECT, b.kv, p, 4), shared.numel()),
                        dtype=torch.uint8, device="cuda")
    reps = torch.zeros(kt.kt_reps_pool_bytes(b.kv, p), dtype=torch.uint8, device="cuda")
    kt.kt_build_block_reps(b.kv, p, 0, b.table.shape[1], reps)
    q_local = torch.randn(batch, 4, 8, 128, generator=torch.Generator().manual_seed(2)).half().cuda()
    words = kt.kt_preselect_mask_words(b.kv)

    def step(ws):
        sel = torch.zeros(batch, 2, top_k, dtype=torch.int32, device="cuda")
        cnt = torch.zeros(batch, 2, dtype=torch.int32, device="cuda")
        out, dense = torch.zeros_like(b.out), torch.zeros_like(b.out)
        kt.kt_sparse_decode_step(b.dq, b.kv, reps, p, sel, cnt, out, ws)
        kt.kt_dense_decode_attn(b.dq, b.kv, 8, SCALE, dense, ws)
        return out, sel, cnt, dense

    def preselect(ws):
        mask = torch.zeros(batch, 2, words, dtype=torch.int32, device="cuda")
        count = torch.zeros(batch, 2, dtype=torch.int32, device="cuda")
        kt.kt_preselect_blocks(b.kv, p, q_local, 4, 5, 6, mask, count, ws)
        return mask, count

    want = step(kt.workspace(kt.KT_OP_SPARSE_STEP, b.kv, p))
    want_mask, want_count = preselect(kt.workspace(kt.KT_OP_PRESELECT, b.kv, p, 4))
    for ws in (shared, large):
        for _ in range(5):
            b.out.fill_(9.0)
            kt.kt_prefix_decode_attn(b.dq, b.kv, b.groups, 8, SCALE, b.out, ws)
            got = step(ws)
            b.check()
            assert kt.kt_read_device_status(ws) == kt.KT_OK
            for x, y in zip(got, want):
                assert torch.equal(x, y)
            if ws is large:
                mask, count = preselect(ws)
                assert torch.equal(mask, want_mask) and torch.equal(count, want_count)
