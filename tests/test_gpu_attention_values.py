"""Attention over values (V) that are not finite."""
import math

import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from test_gpu_attention import ok, on_device, prompt_spans, queries

pytestmark = pytest.mark.gpu


def plant(c, b, key, heads, dims, value):
    """Values of a key of sequence b, on the CPU."""
    page = c["page"]
    at, row = int(c["table"][b, key // page]), key % page
    V = c["V"].float()
    for h in heads:
        V[at, h, row, dims] = value
    c["V"] = V.to(c["V"].dtype)


def check(c, q, got, lse, spans, Hq, D, scale):
    """As by definition, an element that is not finite included: the same infinity, or NaN where
    the definition adds infinities of both signs or has NaN."""
    out, lse = got.cpu().double().view(-1, Hq, D), lse.cpu().double()
    for r, b, lo, hi in spans:
        o, l, spread, big = ref.attend(c, b, q[r].double().view(Hq, D), hi, lo, scale)
        finite = o.isfinite()
        assert bool((out[r].isfinite() == finite).all()), (r, b, lo, hi)
        assert bool(((out[r] == o) | (out[r].isnan() & o.isnan()) | finite).all()), (r, b, lo, hi)
        tol = ref.out_tolerance(o, spread, c["kv"])
        assert bool(((out[r] - o).abs()[finite] <= tol[finite]).all()), (r, b, lo, hi)
        if hi > lo:
            assert bool(((lse[r] - l).abs() <= ref.lse_tolerance(l, big, D)).all()), (r, b, lo, hi)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens", [
    (8, 2, 128, 64, [20001, 3]), (4, 4, 64, 16, [5000, 1, 7000]), (20, 2, 64, 64, [30011]), (12, 1, 128, 32, [9000])])
def test_infinite_values_stay_infinite_in_joins(lib, kv, Hq, Hkv, D, page, lens):
    """Sequences split over many CTAs, with values of the first, a middle and the last key that are
    not finite (decode, and a prompt of one token)."""
    c = ref.make(Hkv, D, page, kv, lens, seed=60)
    kinds = [math.inf, -math.inf, math.inf] if kv == "bf16" else [math.nan] * 3
    for b, n in enumerate(lens):
        for i, key in enumerate((0, n // 2, n - 1)):
            plant(c, b, key, range(Hkv), [3 + 16 * i + b % 16], kinds[i])
    B = len(lens)
    q = queries(B, Hq, D, 60)
    cu = torch.arange(B + 1, dtype=torch.int32).cuda()
    spans = [(b, b, 0, n) for b, n in enumerate(lens)]
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache = on_device(c, attn)
        for got, lse in (attn.decode(q.cuda(), cache, return_lse=True),
                         attn.prompt(q.cuda(), cu, cache, return_lse=True)):
            ok(attn)
            check(c, q, got, lse, spans, Hq, D, D ** -0.5)


CASES = [  # Hq, Hkv, D, page, lens, new, window, keys (sequence, key) with values that are not finite
    (4, 4, 128, 16, [300], [300], 0, [(0, 0), (0, 37), (0, 255), (0, 256), (0, 299)]),
    (2, 2, 64, 64, [700, 90], [411, 90], 0, [(0, 288), (0, 289), (0, 290), (0, 545), (1, 89)]),
    (12, 1, 128, 32, [90, 65], [50, 65], 0, [(0, 41), (0, 88), (1, 3), (1, 64)]),
    (8, 2, 64, 128, [600], [301], 100, [(0, 200), (0, 201), (0, 299), (0, 300), (0, 450), (0, 598)]),
    (3, 3, 128, 256, [900, 40], [500, 40], 33, [(0, 368), (0, 400), (0, 777), (1, 20)]),
    (128, 1, 64, 16, [70], [5], 0, [(0, 66), (0, 67), (0, 69)]),
    (2, 1, 128, 64, [130], [130], 1, [(0, 0), (0, 64), (0, 129)]),
    (8, 2, 128, 64, [9001], [7], 0, [(0, 1234), (0, 8995), (0, 8998)]),       # split and joined
    (4, 4, 64, 32, [7000, 7000], [300, 17], 3000, [(0, 3701), (0, 5000), (0, 6800), (1, 6990)]),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,lens,new,window,keys", CASES)
def test_values_reach_only_queries_that_see_them(lib, kv, Hq, Hkv, D, page, lens, new, window, keys):
    """In a causal chunk, under a window, and in split items."""
    c = ref.make(Hkv, D, page, kv, lens, seed=61)
    kinds = [math.inf, -math.inf, math.nan] if kv == "bf16" else [math.nan]
    for i, (b, key) in enumerate(keys):
        # one dimension for each key (some of them shared), in one head or all
        dims = [(5 * i) % D, (D - 1 - i // 2) % D]
        plant(c, b, key, [i % Hkv] if i % 2 else range(Hkv), dims, kinds[i % len(kinds)])
    T = sum(new)
    q = queries(T, Hq, D, 61)
    cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32).cuda()
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache = on_device(c, attn)
        got, lse = attn.prompt(q.cuda(), cu, cache, window=window, return_lse=True)
        ok(attn)
        for _ in range(2):  # the joins' counters and the deal are back at 0
            again, lse2 = attn.prompt(q.cuda(), cu, cache, window=window, return_lse=True)
            assert torch.equal(again.view(torch.int16), got.view(torch.int16)) and torch.equal(lse, lse2)
        ok(attn)
    check(c, q, got, lse, prompt_spans(lens, new, window)[::3], Hq, D, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_every_value_of_the_last_token_is_nan(lib, kv):
    """Many items in rounds, each with a chunk whose last token's values are all NaN: no other token
    is touched."""
    Hq, Hkv, D, page = 24, 24, 64, 64
    lens = [40 + 9 * b for b in range(48)]
    c = ref.make(Hkv, D, page, kv, lens, seed=62)
    for b, n in enumerate(lens):
        plant(c, b, n - 1, range(Hkv), slice(None), math.nan)
    q = queries(sum(lens), Hq, D, 62)
    starts = [sum(lens[:b]) for b in range(len(lens) + 1)]
    cu = torch.tensor(starts, dtype=torch.int32).cuda()
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        got, lse = attn.prompt(q.cuda(), cu, on_device(c, attn), return_lse=True)
        ok(attn)
    last = torch.zeros(sum(lens), dtype=torch.bool)
    last[torch.tensor(starts[1:]) - 1] = True
    assert bool(got.cpu()[last].isnan().all()) and bool(got.cpu()[~last].isfinite().all())
    check(c, q, got, lse, prompt_spans(lens, lens, 0)[::61], Hq, D, D ** -0.5)
