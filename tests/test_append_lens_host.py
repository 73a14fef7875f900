"""Host-only checks of the append with lengths apart: refusals before the device is touched."""
import pytest

import block_sparse_long_quest_gb300 as kt
from test_prefix_host import BIG, FAKE, by, fake_kv

FAR = 0x10000000


def call(kv="", p="", k=FAKE, v=FAKE, lens=FAR, reps=None, ws=FAKE, n=BIG):
    kv = fake_kv(False) if kv == "" else kv
    p = kt.sparse_params(8, 0, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED) if p == "" else p
    return kt.lib.kt_append_kv_lens(by(kv), by(p), k, v, lens, reps, ws, n, None)


def test_refusals():
    bad = kt.KT_ERR_INVALID_ARG
    for name in ("k", "v", "lens", "ws"):
        assert call(**{name: None}) == bad and call(**{name: FAR + 4}) == bad
    assert call(reps=FAKE + 8) == bad and call(n=255) == bad
    assert call(kv=None) == bad and call(p=None) == bad
    assert call(kv=fake_kv(False, batch=0)) == bad
    for at in (FAKE + 16, FAKE - 16):  # overlaps the five lengths at FAKE, and is not those
        assert call(kv=fake_kv(False, batch=5), lens=at) == bad


def test_binding():
    torch = pytest.importorskip("torch")
    kv, p = fake_kv(False), kt.sparse_params(8, 0, 1, 1, kt.KT_REP_QUEST, kt.KT_HEAD_SHARED)
    ws, x = torch.zeros(256, dtype=torch.uint8), torch.zeros(4, 2, 128, dtype=torch.float16)
    for lens in (None, torch.zeros(3, dtype=torch.int32), torch.zeros(4), torch.zeros(4).long(),
                 torch.zeros(8, dtype=torch.int32)[::2]):
        with pytest.raises(kt.KtError) as e:
            kt.kt_append_kv_lens(kv, p, x, x, lens, None, ws, stream=1)
        assert e.value.status == kt.KT_ERR_INVALID_ARG
