"""Attention over caches with entries that name no page, over pools and tables with strides, and
prompts of groups so wide that a tile holds one token."""
import math

import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from test_gpu_attention import check_rows, ok, on_device, prompt_spans, queries

pytestmark = pytest.mark.gpu


def attend_without(c, b, q, hi, lo, scale, there):
    """ref.attend over the keys [lo, hi) that are there (bool [keys])."""
    Hq, D = q.shape
    G = Hq // c["K"].shape[1]
    keys = torch.arange(lo, hi)[there[lo:hi]]
    if not len(keys):
        return (torch.zeros(Hq, D).double(), torch.full((Hq,), -math.inf).double(), torch.zeros(Hq, D).double(),
                torch.zeros(Hq).double())
    k = ref.rows_of(c, "K", b, hi)[keys].repeat_interleave(G, 1)
    v = ref.rows_of(c, "V", b, hi)[keys].repeat_interleave(G, 1)
    s = torch.einsum("hd,jhd->hj", q, k) * scale
    big = torch.einsum("hd,jhd->hj", q.abs(), k.abs()).amax(1) * scale
    p = torch.softmax(s, 1)
    return (torch.einsum("hj,jhd->hd", p, v), torch.logsumexp(s, 1), torch.einsum("hj,jhd->hd", p, v.abs()), big)


def check_without(c, q, got, lse, spans, Hq, D, scale, there):
    out, lse = got.cpu().double().view(-1, Hq, D), lse.cpu().double()
    for r, b, lo, hi in spans:
        o, l, spread, big = attend_without(c, b, q[r].double().view(Hq, D), hi, lo, scale, there[b])
        tol = ref.out_tolerance(o, spread, c["kv"])
        assert bool(((out[r] - o).abs() <= tol).all()), (r, b, lo, hi)
        if bool(l.isinf().all()):
            assert bool((lse[r] == -math.inf).all()) and bool((out[r] == 0).all()), (r, b, lo, hi)
        else:
            assert bool(((lse[r] - l).abs() <= ref.lse_tolerance(l, big, D)).all()), (r, b, lo, hi)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("G,D,window", [(2, 128, 0), (12, 128, 0), (40, 64, 0), (2, 64, 700), (24, 64, 0)])
def test_bad_pages_in_the_middle(lib, kv, page, G, D, window):
    """A long sequence, split over the GPU, and short ones, with entries in their middle that name no
    page: single ones, whole blocks of 128 keys and more, all of a sequence. Decode and prompt leave
    those keys out and report them."""
    lens, new, Hkv = [6001, 300, 70, 513], [17, 300, 3, 40], 2
    Hq = G * Hkv
    c = ref.make(Hkv, D, page, kv, lens, seed=91)
    table, there = c["table"].clone(), []
    many = c["K"].shape[0]
    for b, n in enumerate(lens):
        pages = -(-n // page)
        bad = {0: [0, 5 % pages, pages // 2, pages - 1] + list(range(pages // 3, pages // 3 + 320 // page + 1)),
               1: [pages // 2], 2: range(pages), 3: [pages - 1, 0]}[b]
        keys = torch.ones(n, dtype=torch.bool)
        for i, e in enumerate(bad):
            table[b, e] = [-1, many, 1 << 30, -(1 << 31)][i % 4]
            keys[e * page:(e + 1) * page] = False
        there.append(keys)
    T = sum(new)
    q = queries(T, Hq, D, 91)
    cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32).cuda()
    scale = 1.0 / math.sqrt(D)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache = on_device(dict(c, table=table), attn)
        got, lse = attn.decode(q[:4].cuda(), cache, window=window, return_lse=True)
        torch.cuda.synchronize()
        assert attn.status() == (tp.TPMLP_ERR_BAD_PAGE, 0x10000)
        spans = [(b, b, max(0, n - window) if window else 0, n) for b, n in enumerate(lens)]
        check_without(c, q, got, lse, spans, Hq, D, scale, there)
        got, lse = attn.prompt(q.cuda(), cu, cache, window=window, return_lse=True)
        torch.cuda.synchronize()
        assert attn.status() == (tp.TPMLP_ERR_BAD_PAGE, 0x10000)
        spans = prompt_spans(lens, new, window)
        check_without(c, q, got, lse, spans[:17:4] + spans[17::29] + spans[-3:], Hq, D, scale, there)
        # the context is as good as before
        cache.page_table.copy_(c["table"])
        want, lse = attn.prompt(q.cuda(), cu, cache, window=window, return_lse=True)
        ok(attn)
        check_rows(c, q, want, lse, spans[::53], Hq, D, scale)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 64), (4, 4, 64, 16), (40, 2, 64, 128), (12, 1, 128, 256),
                                           (24, 2, 64, 32)])
def test_strides_of_pools_tables_and_rows(lib, kv, Hq, Hkv, D, page):
    """K and V in one tensor with something between the pages, a table that is a part of a wider one,
    rows of wider tensors: the same bits as with dense ones, and what lies between stays."""
    lens, new = [700, 33, 0, 2500], [90, 33, 0, 5]
    c = ref.make(Hkv, D, page, kv, lens, seed=92)
    n, T, dtype = c["K"].shape[0], sum(new), c["K"].dtype
    both = torch.full((n, 2 * Hkv + 1, page, D), math.nan).to(dtype).cuda()
    both.view(torch.uint8 if kv == "e4m3" else torch.int16)[:, :Hkv] = c["K"].cuda().view(
        torch.uint8 if kv == "e4m3" else torch.int16)
    both.view(torch.uint8 if kv == "e4m3" else torch.int16)[:, Hkv:2 * Hkv] = c["V"].cuda().view(
        torch.uint8 if kv == "e4m3" else torch.int16)
    wide = torch.full((len(lens), c["table"].shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, 3:-2] = c["table"].cuda()
    q = queries(T, Hq, D, 92).cuda()
    pitched = torch.full((T, Hq * D + 40), math.nan, dtype=torch.bfloat16, device="cuda")
    pitched[:, 8:8 + Hq * D] = q
    cu = torch.tensor([0, 90, 123, 123, 128], dtype=torch.int32).cuda()
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        dense = on_device(c, attn)
        part = tp.PagedCache(attn, both[:, :Hkv], both[:, Hkv:2 * Hkv], wide[:, 3:-2], dense.lens)
        for window in (0, 100):
            want, lse = attn.prompt(q, cu, dense, window=window, return_lse=True)
            room = torch.full((T, Hq * D + 24), 7.0, dtype=torch.bfloat16, device="cuda")
            got, lse2 = attn.prompt(pitched[:, 8:8 + Hq * D], cu, part, window=window, out=room[:, 16:16 + Hq * D],
                                    return_lse=True)
            ok(attn)
            assert torch.equal(got, want) and torch.equal(lse, lse2)
            assert bool((room[:, :16] == 7.0).all()) and bool((room[:, 16 + Hq * D:] == 7.0).all())
            check_rows(c, q.cpu(), got, lse, prompt_spans(lens, new, window)[::13], Hq, D, 1.0 / math.sqrt(D))
            want, lse = attn.decode(q[:4], dense, window=window, return_lse=True)
            got, lse2 = attn.decode(pitched[:4, 8:8 + Hq * D], part, window=window, out=room[:4, 16:16 + Hq * D],
                                    return_lse=True)
            ok(attn)
            assert torch.equal(got, want) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,new,window", [
    (80, 1, 128, 64, [300, 37], [61, 37], 0),
    (128, 1, 64, 16, [70, 0, 9], [70, 0, 2], 0),
    (130, 2, 128, 128, [4100], [9], 0),           # 65: one token to a tile, split
    (200, 2, 64, 32, [150], [150], 33),
])
def test_prompt_of_groups_of_more_than_64(lib, kv, Hq, Hkv, D, page, lens, new, window):
    c = ref.make(Hkv, D, page, kv, lens, seed=93)
    q = queries(sum(new), Hq, D, 93)
    cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32).cuda()
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        got, lse = attn.prompt(q.cuda(), cu, on_device(c, attn), window=window, return_lse=True)
        ok(attn)
    check_rows(c, q, got, lse, prompt_spans(lens, new, window)[::3], Hq, D, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("Hq,Hkv", [(17, 1), (72, 3), (64, 2)])
def test_decode_in_two_passes_over_the_heads(lib, Hq, Hkv):
    """Groups of 17 to 32 heads of 64 over an e4m3 cache, sequences of no, few and many keys."""
    lens = [9000, 0, 1, 130, 4097] + [(11 * b) % 90 for b in range(40)]
    c = ref.make(Hkv, 64, 32, "e4m3", lens, seed=94)
    q = queries(len(lens), Hq, 64, 94)
    with tp.Attention(Hq, Hkv, 64, 32, kv_dtype="e4m3") as attn:
        cache = on_device(c, attn)
        for window in (0, 77):
            got, lse = attn.decode(q.cuda(), cache, window=window, return_lse=True)
            ok(attn)
            spans = [(b, b, max(0, n - window) if window else 0, n) for b, n in enumerate(lens)]
            check_rows(c, q, got, lse, spans, Hq, 64, 0.125)
