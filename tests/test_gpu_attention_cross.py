"""Attention of tokens to all keys of another sequence on the GPU against the definition in fp64."""
import math

import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from test_gpu_attention import check_rows, ok, on_device, queries

pytestmark = pytest.mark.gpu


def starts(new, first=0):
    return torch.tensor([first + sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32).cuda()


def all_keys(lens, new, first=0):
    return [(r, b, 0, lens[b]) for r, b in enumerate((b for b, n in enumerate(new) for _ in range(n)), first)]


SHAPES = [  # Hq, Hkv, D, page, keys, rows
    (4, 4, 128, 16, [61], [61]),
    (12, 12, 64, 16, [577, 1, 0, 300], [4, 4, 3, 17]),       # beams; a sequence without keys
    (8, 2, 128, 64, [257, 64, 5, 128], [129, 64, 2, 0]),     # one without rows
    (36, 3, 128, 32, [200, 33], [90, 33]),                   # 12 query heads to a kv head
    (40, 1, 64, 128, [150], [70]),
    (6, 2, 64, 16, [3, 50], [50, 5]),                        # more rows than keys
    (128, 1, 128, 32, [130, 15], [5, 1]),                    # the widest group
    (2, 2, 64, 256, [600], [600]),
    (7, 7, 128, 64, [63, 64, 65, 127, 128, 129], [1, 1, 1, 1, 1, 1]),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,new", SHAPES)
def test_matches_definition(lib, kv, Hq, Hkv, D, page, lens, new):
    c = ref.make(Hkv, D, page, kv, lens, seed=Hq + D + 1)  # NaN behind every sequence's last key
    first, T = 2, sum(new) + 5  # two rows before the first sequence and three behind the last: of none
    q = queries(T, Hq, D, page)
    cu = starts(new, first)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache = on_device(c, attn)
        wide = torch.zeros((T, Hq * D + 24), dtype=torch.bfloat16, device="cuda")
        wide[:, :Hq * D] = q.cuda()
        out = torch.full((T, Hq * D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        got, lse = attn.cross(wide[:, :Hq * D], cu, cache, out=out[:, :Hq * D], return_lse=True)
        ok(attn)
        assert bool((out[:, Hq * D:] == 7.0).all()) and bool((out[-3:] == 7.0).all()) and bool((out[:2] == 7.0).all())
        again = attn.cross(q.cuda(), cu, cache)
        ok(attn)
        assert torch.equal(again[2:-3], got[2:-3])
    check_rows(c, q, got, lse, all_keys(lens, new, first), Hq, D, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,new", [
    (8, 2, 128, 64, [9001], [3]),                  # few rows, many keys: split and joined
    (4, 1, 64, 16, [20011, 5, 0, 129], [40, 2, 3, 129]),
    (5, 5, 128, 128, [7000, 6999], [300, 17]),
    (20, 1, 128, 32, [5003], [1]),
    (8, 1, 64, 64, [30000], [64]),                 # many contributors: joined by a launch of its own
    (32, 8, 128, 64, [9000, 0, 40], [20, 30, 3]),
    (6, 2, 64, 16, [4001, 2047, 130], [200, 1, 77]),
])
def test_long_sequences_are_split(lib, kv, Hq, Hkv, D, page, lens, new):
    c = ref.make(Hkv, D, page, kv, lens, seed=17)
    q = queries(sum(new), Hq, D, 17) * 2
    cu = starts(new)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache = on_device(c, attn)
        got, lse = attn.cross(q.cuda(), cu, cache, return_lse=True)
        ok(attn)
        for _ in range(3):  # deterministic, and the counters are back at 0
            assert torch.equal(attn.cross(q.cuda(), cu, cache), got)
        # rows of no sequence, before and behind the others, stay as they are
        wide = torch.cat([q[:1].expand(2, -1), q, q[:1].expand(3, -1)]).cuda()
        out = torch.full_like(wide, 7.0)
        again, lse2 = attn.cross(wide, cu + 2, cache, out=out, return_lse=True)
        assert bool((out[:2] == 7.0).all()) and bool((out[-3:] == 7.0).all())
        ok(attn)
    rows = all_keys(lens, new)
    check_rows(c, q, got, lse, rows[:6] + rows[6::23] + rows[-3:], Hq, D, 1.0 / math.sqrt(D))
    # (more rows may be another kernel's)
    check_rows(c, wide.cpu(), again, lse2, all_keys(lens, new, 2)[::23], Hq, D, 1.0 / math.sqrt(D))


FEW = [  # Hq, Hkv, D, page, keys, rows: few rows to a sequence, up to two blocks of 8 or 16 with their heads
    (12, 12, 64, 16, [577, 1, 0, 300], [4, 4, 3, 4]),
    (8, 8, 128, 32, [40, 129, 1000], [1, 16, 0]),               # two blocks of 8
    (6, 2, 128, 64, [40, 129, 1000, 7], [2, 5, 0, 1]),          # three heads to a kv head
    (5, 5, 64, 16, [5 + b for b in range(40)], [(3 * b) % 7 for b in range(40)]),
    (4, 1, 64, 128, [100, 0, 31], [0, 0, 2]),
    (4, 4, 128, 64, [9001, 20], [3, 1]),                        # split and joined
    (16, 2, 64, 32, [3000, 70], [4, 1]),
    (3, 3, 128, 16, [200, 100, 50], [1, 17, 1]),                # one sequence with too many: the other kernel
    (3, 3, 64, 16, [31] * 50, [1] * 49 + [40]),
    (2, 1, 64, 16, [100] * 3, [0, 0, 0]),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,new", FEW)
def test_few_rows(lib, kv, Hq, Hkv, D, page, lens, new):
    test_matches_definition(lib, kv, Hq, Hkv, D, page, lens, new)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (128, 256)])
def test_lengths_about_the_parts_of_a_block(lib, kv, D, page):
    lens = [x + d for x in (0, 16, 64, 96, 112, 128, 192, 224, 256) for d in (-1, 0, 1) if x + d >= 0]
    new = [(70, 1, 130)[b % 3] for b in range(len(lens))]
    test_matches_definition(lib, kv, 3, 3, D, page, lens, new)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_rise_from_block_to_block(lib, kv, D):
    """Scores of some hundreds: rows' references move in block after block, in some rows of a tile only."""
    Hq, Hkv, lens, new = 4, 2, [1500, 333, 7000], [150, 40, 130]
    c = ref.make(Hkv, D, 64, kv, lens, seed=31)
    q = queries(sum(new), Hq, D, 31)
    with tp.Attention(Hq, Hkv, D, 64, kv_dtype=kv) as attn:
        got, lse = attn.cross(q.cuda(), starts(new), on_device(c, attn), scale=4.0, return_lse=True)
        ok(attn)
    check_rows(c, q, got, lse, all_keys(lens, new)[::7], Hq, D, 4.0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_replays_change_from_few_rows_to_many(lib, kv):
    """A captured call follows the rows that the offsets name at each replay, whichever kernel has them."""
    Hq, Hkv, D, page, lens = 4, 4, 128, 32, [300, 70, 129]
    c = ref.make(Hkv, D, page, kv, lens, seed=29)
    q = queries(20, Hq, D, 29)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache, qd, cu = on_device(c, attn), q.cuda(), starts([7, 6, 7])
        out = torch.empty_like(qd)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attn.cross(qd, cu, cache, out=out)
        for new in ([7, 6, 7], [20, 0, 0], [0, 16, 4], [1, 2, 17]):
            cu.copy_(starts(new))
            out.fill_(7.0)
            graph.replay()
            ok(attn)
            want, lse = attn.cross(qd, cu, cache, return_lse=True)
            ok(attn)
            assert torch.equal(out, want)
            check_rows(c, q, out, lse, all_keys(lens, new), Hq, D, D ** -0.5)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_many_items(lib, kv):
    """More items than a block tabulates."""
    lens, new = [500, 50, 1033], [3000, 50, 699]
    Hq, Hkv, D = 96, 12, 64
    c = ref.make(Hkv, D, 32, kv, lens, seed=18)
    q = queries(sum(new), Hq, D, 18)
    with tp.Attention(Hq, Hkv, D, 32, kv_dtype=kv) as attn:
        got, lse = attn.cross(q.cuda(), starts(new), on_device(c, attn), return_lse=True)
        ok(attn)
    rows = all_keys(lens, new)
    check_rows(c, q, got, lse, rows[:2] + rows[1::401] + rows[-2:], Hq, D, 0.125)


@pytest.mark.parametrize("one", [0, 30])
def test_many_sequences(lib, one):
    """More sequences than the work list's table has entries, of 0 to 40 keys and 0 to 2 rows, or one of
    more (the other kernel)."""
    lens, new = [(7 * b) % 41 for b in range(700)], [b % 3 for b in range(700)]
    new[601] += one
    c = ref.make(1, 64, 16, "bf16", lens, seed=4)
    q = queries(sum(new), 3, 64, 4)
    with tp.Attention(3, 1, 64, 16) as attn:
        got, lse = attn.cross(q.cuda(), starts(new), on_device(c, attn), return_lse=True)
        ok(attn)
    check_rows(c, q, got, lse, all_keys(lens, new), 3, 64, 0.125)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_one_row_to_a_sequence_is_decode(lib, kv):
    lens = [300, 1, 77, 0]
    c = ref.make(2, 128, 32, kv, lens, seed=6)
    q = queries(4, 6, 128, 6)
    with tp.Attention(6, 2, 128, 32, kv_dtype=kv) as attn:
        cache = on_device(c, attn)
        a, la = attn.cross(q.cuda(), starts([1] * 4), cache, return_lse=True)
        b, lb = attn.decode(q.cuda(), cache, return_lse=True)
        ok(attn)
    spans = [(r, r, 0, n) for r, n in enumerate(lens)]
    check_rows(c, q, a, la, spans, 6, 128, 128 ** -0.5)
    check_rows(c, q, b, lb, spans, 6, 128, 128 ** -0.5)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,new", [([260, 140, 90], [30, 150, 9]), ([9000, 140, 90], [3, 2, 9])])
def test_values_that_are_not_finite_stay_in_their_sequence(lib, kv, lens, new):
    Hq, Hkv, D, page = 4, 2, 64, 16
    c = ref.make(Hkv, D, page, kv, lens, seed=23)
    bad = math.nan if kv == "e4m3" else math.inf
    c["V"].view(torch.uint8 if kv == "e4m3" else c["V"].dtype)  # (indexing below is in the pool's type)
    pg = int(c["table"][1, 3])
    pools = {n: c[n].float() for n in ("K", "V")}
    pools["V"][pg, 1, 5, 7] = bad       # key 53 of sequence 1, kv head 1, dimension 7
    c["V"] = pools["V"].to(c["V"].dtype)
    q = queries(sum(new), Hq, D, 23)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        got, lse = attn.cross(q.cuda(), starts(new), on_device(c, attn), return_lse=True)
        ok(attn)
    out = got.cpu().float().view(-1, Hq, D)
    off = ~out.isfinite()
    want = torch.zeros_like(off)
    want[new[0]:new[0] + new[1], 2:, 7] = True
    assert torch.equal(off, want)
    assert bool((out[off].isnan() if kv == "e4m3" else out[off] == math.inf).all())
    assert bool(lse.isfinite().all())
    rest = [s for s in all_keys(lens, new) if s[1] != 1]
    check_rows(c, q, got, lse, rest[:4] + rest[-2:], Hq, D, 0.125)


def test_bad_pages_are_left_out_and_reported(lib):
    """A page outside the pool: its keys are left out. A length behind the table counts as the table's."""
    Hq, Hkv, D, page = 4, 2, 128, 32
    lens, new = [200, 70], [9, 3]
    c = ref.make(Hkv, D, page, "bf16", lens, seed=12)
    q = queries(12, Hq, D, 12)
    kept = dict(c, table=c["table"].clone(), lens=c["lens"].clone())
    c["table"][0, 2] = 10 ** 6
    with tp.Attention(Hq, Hkv, D, page) as attn:
        got, lse = attn.cross(q.cuda(), starts(new), on_device(c, attn), return_lse=True)
        torch.cuda.synchronize()
        assert attn.status()[0] == tp.TPMLP_ERR_BAD_PAGE
        # the same keys without that page
        short = dict(kept, table=torch.cat([kept["table"][:, :2], kept["table"][:, 3:]], 1),
                     lens=torch.tensor([200 - page, 70], dtype=torch.int32))
        short["table"][1] = kept["table"][1, :short["table"].shape[1]]
        check_rows(short, q, got, lse, [(r, 0, 0, 200 - page) for r in range(9)] + [(r, 1, 0, 70) for r in (9, 10, 11)],
                   Hq, D, 128 ** -0.5)
        kept["lens"][1] = 10 ** 6
        kept["table"][1] = kept["table"][0]
        got, lse = attn.cross(q.cuda(), starts(new), on_device(kept, attn), return_lse=True)
        torch.cuda.synchronize()
        assert attn.status()[0] == tp.TPMLP_ERR_BAD_PAGE
    full = kept["table"].shape[1] * page
    assert full == 224  # rows behind the sequence's last key hold NaN
    assert bool(got[9:].isnan().any()) and bool(got[:9].isfinite().all())


def test_replay_reads_lengths_and_rows_anew(lib):
    lens, new = [400, 90, 1], [5, 1, 7]
    c = ref.make(2, 128, 32, "bf16", lens, seed=5)
    q = queries(13, 4, 128, 5)
    with tp.Attention(4, 2, 128, 32) as attn:
        cache = on_device(c, attn)
        qd, out = q.cuda(), torch.empty((13, 512), dtype=torch.bfloat16, device="cuda")
        cu = starts(new)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attn.cross(qd, cu, cache, out=out)
        for now, rows in ((lens, new), ([33, 0, 1], [1, 2, 10]), ([256, 90, 0], [0, 13, 0])):
            cache.lens.copy_(torch.tensor(now, dtype=torch.int32))
            cu.copy_(starts(rows))
            graph.replay()
            ok(attn)
            want, lse = attn.cross(qd, cu, cache, return_lse=True)
            ok(attn)
            assert torch.equal(out, want)
            check_rows(c, q, out, lse, all_keys(now, rows), 4, 128, 128 ** -0.5)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = attn.cross(qd, cu, cache, stream=side)
        side.synchronize()
        assert torch.equal(got, out)


def test_arguments(lib):
    with tp.Attention(4, 2, 64, 16) as attn:
        table = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
        cache = attn.new_cache(1, table, torch.ones(2, dtype=torch.int32, device="cuda"))
        q = torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda")
        cu = torch.zeros(3, dtype=torch.int32, device="cuda")
        for args in ((q.float(), cu), (q[:, :128], cu), (q, cu.long()), (q, cu[:2]), (q.cpu(), cu)):
            with pytest.raises((TypeError, ValueError)):
                attn.cross(*args, cache)
        with pytest.raises(tp.TpmlpError):
            attn.cross(q, cu, cache, scale=0.0)
        assert attn.cross(q[:0], cu, cache).shape == (0, 256)
