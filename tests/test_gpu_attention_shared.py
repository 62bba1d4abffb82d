"""Decode of sequences behind shared prefixes on the GPU against the definition in fp64."""
import math

import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from test_gpu_attention import ok, on_device, queries
from test_gpu_attention_cross import starts

pytestmark = pytest.mark.gpu


def split(c, attn, P):
    """The first P sequences of a made cache as the prefixes, the others as the batch."""
    both = on_device(c, attn)
    table, lens = both.page_table, both.lens
    return (tp.PagedCache(attn, both.K, both.V, table[P:], lens[P:].clone()),
            tp.PagedCache(attn, both.K, both.V, table[:P], lens[:P].clone()))


def attend(c, q, p, b, P, prefix, lens, scale):
    """As attention_ref.attend, over prefix p (None: none) and then sequence b's own keys."""
    n, m = 0 if p is None else prefix[p], lens[b]
    Hq, D = q.shape
    if n + m == 0:
        return ref.attend(c, 0, q, 0, 0, scale)
    G = Hq // c["K"].shape[1]
    k, v = (torch.cat(([ref.rows_of(c, which, p, n)] if n else []) + ([ref.rows_of(c, which, P + b, m)] if m else []))
            .repeat_interleave(G, 1) for which in ("K", "V"))
    s = torch.einsum("hd,jhd->hj", q, k) * scale
    big = torch.einsum("hd,jhd->hj", q.abs(), k.abs()).amax(1) * scale
    w = torch.softmax(s, 1)
    return (torch.einsum("hj,jhd->hd", w, v), torch.logsumexp(s, 1), torch.einsum("hj,jhd->hd", w, v.abs()), big)


def prefix_of(cu, b):
    return next((p for p in range(len(cu) - 1) if cu[p] <= b < cu[p + 1]), None)


def check(c, q, got, lse, prefix, lens, cu, rows, Hq, D, scale):
    """Each part is computed like any other attention, and their join (two powers, two products and a
    quotient in fp32, of logs below 2^7) adds 2^-16 at most: inside out_tolerance's margin of 2^-13."""
    out, lse, P = got.cpu().double().view(-1, Hq, D), lse.cpu().double(), len(prefix)
    for b in rows:
        p = prefix_of(cu, b)
        o, l, spread, big = attend(c, q[b].double().view(Hq, D), p, b, P, prefix, lens, scale)
        tol = ref.out_tolerance(o, spread, c["kv"])
        err = (out[b] - o).abs()
        assert bool((err <= tol).all()), (b, p, float((err / tol).max()))
        if lens[b] + (0 if p is None else prefix[p]) == 0:
            assert bool((lse[b] == -math.inf).all())
        else:
            assert bool(((lse[b] - l).abs() <= ref.lse_tolerance(l, big, D)).all()), b


SHAPES = [  # Hq, Hkv, D, page, prefixes, first sequence with one, sequences of each, own keys
    (4, 4, 128, 16, [100], 0, [5], [1, 0, 17, 300, 16]),
    (12, 12, 64, 16, [511], 0, [3], [65, 1, 40]),
    (32, 8, 128, 64, [129, 0, 64], 2, [3, 2, 1], [1, 129, 128, 127, 2, 0, 515, 9, 1, 0]),  # some without prefix
    (8, 1, 64, 32, [31, 33], 0, [0, 3], [1000, 31, 33]),         # a prefix of no sequence
    (36, 3, 128, 32, [700, 9], 0, [40, 2], [5 + b for b in range(42)]),   # 12 query heads to a kv head
    (40, 1, 128, 128, [260], 1, [1], [260, 1, 0]),
    (18, 2, 64, 256, [1], 0, [2], [511, 3]),                     # 9
    (128, 1, 64, 128, [300, 40], 0, [3, 1], [300, 5, 0, 128]),   # the widest group
    (17, 1, 128, 32, [2000], 0, [2], [20, 2000]),
    (16, 16, 128, 64, [65], 0, [300], [(7 * b) % 41 for b in range(300)]),
    (33, 1, 64, 16, [64, 64], 0, [2, 2], [1, 1, 1, 0]),
    # few rows to a prefix (the row kernel), some of two blocks, and one prefix with too many among few
    (12, 12, 64, 16, [77, 0, 129, 5], 1, [4, 2, 0, 1], [3, 0, 17, 1, 40, 9, 0, 300, 2]),
    (4, 4, 128, 32, [300, 40], 0, [12, 3], [b for b in range(15)]),
    (6, 2, 128, 16, [9001], 2, [2], [5, 0, 3, 70, 1]),
    (2, 2, 128, 64, [100] * 40, 0, [b % 3 for b in range(40)], [b % 5 for b in range(45)]),
    (2, 2, 64, 64, [100] * 40, 3, [1] * 39 + [30], [b % 5 for b in range(80)]),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,prefix,first,members,lens", SHAPES)
def test_matches_definition(lib, kv, Hq, Hkv, D, page, prefix, first, members, lens):
    P, B = len(prefix), len(lens)
    c = ref.make(Hkv, D, page, kv, prefix + lens, seed=Hq + D)
    q = queries(B, Hq, D, page)
    cu = starts(members, first)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache, shared = split(c, attn, P)
        wide = torch.zeros((B, Hq * D + 16), dtype=torch.bfloat16, device="cuda")
        wide[:, :Hq * D] = q.cuda()
        out = torch.full((B, Hq * D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        got, lse = attn.decode_shared(wide[:, :Hq * D], cache, shared, cu, out=out[:, :Hq * D], return_lse=True)
        ok(attn)
        assert bool((out[:, Hq * D:] == 7.0).all())
        again, lse2 = attn.decode_shared(q.cuda(), cache, shared, cu, return_lse=True)
        ok(attn)
        assert torch.equal(again, got) and torch.equal(lse, lse2)  # deterministic
    check(c, q, got, lse, prefix, lens, cu.tolist(), range(0, B, max(1, B // 50)), Hq, D, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,prefix,members,lens", [
    (8, 2, 128, [20001], [2], [3, 9001]),
    (20, 1, 64, [9001, 300], [30, 3], [5] * 32 + [7000]),
    (6, 6, 64, [15000], [70], [1] * 70),
])
def test_long_ones_are_split_and_joined(lib, kv, Hq, Hkv, D, prefix, members, lens):
    c = ref.make(Hkv, D, 64, kv, prefix + lens, seed=9)
    q = queries(len(lens), Hq, D, 9) * 3  # peaked weights: one part outweighs the other
    cu = starts(members)
    with tp.Attention(Hq, Hkv, D, 64, kv_dtype=kv) as attn:
        cache, shared = split(c, attn, len(prefix))
        got, lse = attn.decode_shared(q.cuda(), cache, shared, cu, return_lse=True)
        for _ in range(3):
            assert torch.equal(attn.decode_shared(q.cuda(), cache, shared, cu), got)
        ok(attn)
    rows = sorted({0, 1, len(lens) // 2, len(lens) - 1})
    check(c, q, got, lse, prefix, lens, cu.tolist(), rows, Hq, D, D ** -0.5)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_is_decode_over_the_same_keys(lib, kv):
    """A prefix of whole pages in front of every sequence's own pages: plain decode of one page table."""
    Hq, Hkv, D, page, prefix, lens = 8, 2, 128, 32, 320, [1, 64, 300]
    c = ref.make(Hkv, D, page, kv, [prefix] + lens, seed=3)
    q = queries(3, Hq, D, 3)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache, shared = split(c, attn, 1)
        a = attn.decode_shared(q.cuda(), cache, shared, starts([3]))
        table = torch.cat([shared.page_table.expand(3, -1)[:, :prefix // page], cache.page_table], 1).contiguous()
        b = attn.decode(q.cuda(), tp.PagedCache(attn, cache.K, cache.V, table, cache.lens + prefix))
        none = tp.PagedCache(attn, cache.K, cache.V, shared.page_table[:0], shared.lens[:0])
        d = attn.decode_shared(q.cuda(), cache, none, torch.zeros(1, dtype=torch.int32, device="cuda"))
        assert torch.equal(d, attn.decode(q.cuda(), cache))  # without prefixes: decode itself
        ok(attn)
    # both within their tolerance of the definition: weights and output, 2^-8 or 2^-11 and 2^-8
    scale = c["V"].float()[~c["V"].float().isnan()].abs().max() * float(c["vs"].max())
    assert float((a.float() - b.float()).abs().max()) <= 2 * float(scale) * (ref.P_HALF_STEP[kv] + 2.0 ** -8)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (36, 1)])
def test_values_that_are_not_finite_reach_who_sees_them(lib, kv, Hq, Hkv):
    D, page, prefix, members, lens = 64, 16, [90, 40], [3, 2], [9, 100, 0, 33, 20]
    c = ref.make(Hkv, D, page, kv, prefix + lens, seed=31)
    bad = math.nan if kv == "e4m3" else math.inf
    V = c["V"].float()
    V[int(c["table"][1, 1]), 0, 2, 7] = bad        # key 18 of prefix 1
    V[int(c["table"][2 + 1, 3]), 0, 2, 9] = bad    # key 50 of sequence 1's own
    c["V"] = V.to(c["V"].dtype)
    q = queries(5, Hq, D, 31)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache, shared = split(c, attn, 2)
        got = attn.decode_shared(q.cuda(), cache, shared, starts(members))
        ok(attn)
    off = ~got.cpu().float().view(5, Hq, D).isfinite()
    want = torch.zeros_like(off)
    want[3:, :Hq // Hkv, 7] = True
    want[1, :Hq // Hkv, 9] = True
    assert torch.equal(off, want)


def test_bad_pages_and_offsets(lib):
    """Pages outside the pool are left out and reported; offsets behind the batch are held to it."""
    Hq, Hkv, D, page, prefix, lens = 4, 2, 64, 16, [48], [20, 5, 33]
    c = ref.make(Hkv, D, page, "bf16", prefix + lens, seed=2)
    q = queries(3, Hq, D, 2)
    with tp.Attention(Hq, Hkv, D, page) as attn:
        cache, shared = split(c, attn, 1)
        far = torch.tensor([0, 10 ** 9], dtype=torch.int32, device="cuda")
        got, lse = attn.decode_shared(q.cuda(), cache, shared, far, return_lse=True)
        ok(attn)
        check(c, q, got, lse, prefix, lens, [0, 3], range(3), Hq, D, 0.125)
        under = torch.tensor([-5, 2], dtype=torch.int32, device="cuda")
        got, lse = attn.decode_shared(q.cuda(), cache, shared, under, return_lse=True)
        ok(attn)
        check(c, q, got, lse, prefix, lens, [0, 2], range(3), Hq, D, 0.125)
        shared.page_table[0, 2] = -7
        got, lse = attn.decode_shared(q.cuda(), cache, shared, starts([3]), return_lse=True)
        torch.cuda.synchronize()
        assert attn.status()[0] == tp.TPMLP_ERR_BAD_PAGE
        check(c, q, got, lse, [32], lens, [0, 3], range(3), Hq, D, 0.125)


@pytest.mark.parametrize("Hq", [4, 40])
def test_graphs_share_and_outlive_the_workspace(lib, Hq):
    """Two graphs of one context, the second captured after the workspace grew: each replays as an eager
    call does, with lengths, offsets and queries read anew. A capture that would have to grow it is
    refused."""
    Hkv, D, page = 2 if Hq == 4 else 1, 128, 32
    prefix, lens = [300, 77], [(11 * b) % 50 for b in range(40)]
    c = ref.make(Hkv, D, page, "bf16", prefix + lens, seed=7)
    q = queries(40, Hq, D, 7).cuda()
    with tp.Attention(Hq, Hkv, D, page) as attn:
        cache, shared = split(c, attn, 2)
        few = tp.PagedCache(attn, cache.K, cache.V, cache.page_table[:5], cache.lens[:5])
        cu = starts([2, 3])
        with pytest.raises(tp.TpmlpError, match="reserve"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                attn.decode_shared(q[:5], few, shared, cu, out=torch.empty_like(q[:5]))
        attn.reserve(5)
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        o1, o2, cu2 = torch.empty_like(q[:5]), torch.empty_like(q), starts([11, 29])
        with torch.cuda.graph(g1):
            attn.decode_shared(q[:5], few, shared, cu, out=o1)
        attn.reserve(40)
        with torch.cuda.graph(g2):
            attn.decode_shared(q, cache, shared, cu2, out=o2)
        for step in range(3):
            cache.lens.copy_(torch.tensor([max(0, n - 3 * step) for n in lens], dtype=torch.int32))
            cu.copy_(starts([step, 5 - step]))
            for g in (g1, g2, g1, g2):
                g.replay()
            ok(attn)
            want, lse = attn.decode_shared(q, cache, shared, cu2, return_lse=True)
            assert torch.equal(o2, want)
            assert torch.equal(o1, attn.decode_shared(q[:5], few, shared, cu))
            ok(attn)
            check(c, q.cpu(), o2, lse, prefix, cache.lens.tolist(), cu2.tolist(), (0, 10, 11, 39), Hq, D, D ** -0.5)


def test_streams(lib):
    """A side stream gives the same; calls back to back with others of the context do not disturb it."""
    Hq, Hkv, D, page, prefix, lens = 8, 8, 64, 16, [2000], [40, 7, 300, 1]
    c = ref.make(Hkv, D, page, "bf16", prefix + lens, seed=13)
    q = queries(4, Hq, D, 13).cuda()
    with tp.Attention(Hq, Hkv, D, page) as attn:
        cache, shared = split(c, attn, 1)
        cu = starts([4])
        want = attn.decode_shared(q, cache, shared, cu)
        plain = attn.decode(q, cache)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = attn.decode_shared(q, cache, shared, cu, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        outs = []
        for _ in range(20):
            outs += [attn.decode_shared(q, cache, shared, cu), attn.decode(q, cache)]
        ok(attn)
        assert all(torch.equal(o, want if i % 2 == 0 else plain) for i, o in enumerate(outs))


def test_queries_written_just_before(lib):
    """Keys appended and queries written by the calls before, without a pause: the second launch starts
    early, and must still see them."""
    Hq, Hkv, D, page, prefix = 8, 2, 128, 16, [200]
    B = 6
    c = ref.make(Hkv, D, page, "bf16", prefix + [64] * B, seed=19)
    g = torch.Generator().manual_seed(19)
    rounds = [(torch.randn((B, (Hq + 2 * Hkv) * D), generator=g)).bfloat16().cuda() for _ in range(12)]
    pos = torch.full((B,), 63, dtype=torch.int32, device="cuda")
    with tp.Attention(Hq, Hkv, D, page) as attn:
        cache, shared = split(c, attn, 1)
        cu = starts([B])

        def step(x):
            q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], dim=1)
            return attn.decode_shared(attn.append(q, k, v, cache, pos), cache, shared, cu)

        slow = []
        for x in rounds:
            slow.append(step(x))
            torch.cuda.synchronize()
        fast = [step(x) for x in rounds]
        ok(attn)
    assert all(torch.equal(a, b) for a, b in zip(slow, fast))


def test_arguments(lib):
    with tp.Attention(4, 2, 64, 16) as attn, tp.Attention(4, 2, 64, 32) as other:
        table = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
        cache = attn.new_cache(1, table, torch.ones(3, dtype=torch.int32, device="cuda"))
        prefix = attn.new_cache(1, table[:1], torch.ones(1, dtype=torch.int32, device="cuda"))
        wrong = other.new_cache(1, table[:1], torch.ones(1, dtype=torch.int32, device="cuda"))
        q = torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda")
        cu = torch.zeros(2, dtype=torch.int32, device="cuda")
        for args in ((q.float(), cache, prefix, cu), (q[:2], cache, prefix, cu), (q, cache, wrong, cu),
                     (q, cache, prefix, cu.long()), (q, cache, prefix, cu[:1]), (q, cache, cache, cu)):
            with pytest.raises((TypeError, ValueError)):
                attn.decode_shared(*args)
        with pytest.raises(tp.TpmlpError):
            attn.decode_shared(q, cache, prefix, cu, scale=-1.0)
