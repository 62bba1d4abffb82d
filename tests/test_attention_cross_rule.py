"""Which launches cross attention takes, by rows, heads, keys and the cache's type (no GPU needed)."""
import ctypes
import random

import pytest

import tensor_transformer_mlp_tmem_gb300 as tp
from test_attention_host import hooks  # noqa: F401

E4M3 = tp.TPMLP_FLAG_KV_E4M3
ROWS, OPEN, APART = 1, 2, 4  # the row kernel, the tile kernel, a join of the tile kernel's parts


@pytest.fixture
def path(hooks):  # noqa: F811
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    hooks.tpmlp_test_cross_path.argtypes = [vp, i64, i64, i64]
    hooks.tpmlp_test_cross_room.argtypes, hooks.tpmlp_test_cross_room.restype = [vp], i64

    def of(Hq, Hkv, D, flags, B, T, keys):
        c = hooks.tpmlp_test_attn_context(Hq, Hkv, D, 64, 0, flags)
        got = hooks.tpmlp_test_cross_path(c, B, T, keys), hooks.tpmlp_test_cross_room(c)
        hooks.tpmlp_destroy(c)
        return got

    return of


@pytest.mark.parametrize("Hq,Hkv,D,B,rows,keys,bf16,e4m3", [
    (12, 12, 64, 16, 4, 577, ROWS | OPEN, ROWS | OPEN),       # beams: which of the two, they find on the device
    (12, 12, 64, 5, 1, 511, ROWS, ROWS),                      # few in all: no sequence can have many
    (8, 8, 128, 1, 8, 9000, ROWS, ROWS),
    (8, 8, 128, 2, 9, 9000, OPEN | APART, ROWS),              # bf16's row kernel takes 8 to a kv head, e4m3's 18 in all
    (32, 32, 128, 1, 17, 9000, OPEN | APART, OPEN | APART),   # 32 items on 152 SMs: 4 to each
    (96, 96, 128, 4, 1024, 4096, OPEN, OPEN),                 # more items than SMs
    (12, 12, 64, 2, 300, 9000, OPEN | APART, OPEN),           # 4 SMs to an item: e4m3 with heads of 64 wants 9
    (8, 8, 64, 3, 200, 5000, OPEN | APART, OPEN),             # 6
    (16, 16, 64, 1, 256, 4096, OPEN | APART, OPEN | APART),   # 9
    (16, 16, 64, 1, 256, 2047, OPEN, OPEN),                   # tables of fewer keys than a join is worth
    (8, 1, 64, 1, 64, 30000, OPEN | APART, OPEN | APART),     # 76
])
def test_the_faster_launches(path, Hq, Hkv, D, B, rows, keys, bf16, e4m3):
    assert path(Hq, Hkv, D, 0, B, B * rows, keys)[0] == bf16
    assert path(Hq, Hkv, D, E4M3, B, B * rows, keys)[0] == e4m3


def test_a_join_of_parts_has_room(path):
    """Results that wait for the join lie in the context's own memory: no call has more than it holds."""
    r, met = random.Random(6), 0
    for _ in range(4000):
        D, flags, Hkv = r.choice([64, 128]), r.choice([0, E4M3]), r.choice([1, 1, 2, 3, 5, 8, 16, 37])
        Hq = Hkv * r.choice([1, 2, 3, 5, 8, 16, 43, 64, 128])
        B, T = r.choice([1, 1, 2, 3, 7, 40]), int(2 ** r.uniform(0, 14))
        got, room = path(Hq, Hkv, D, flags, B, T, 1 << 20)
        assert got & (ROWS | OPEN)
        if got & APART:
            met += 1
            assert T * Hq <= room, (Hq, Hkv, D, flags, B, T)
    assert met > 200
