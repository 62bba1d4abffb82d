"""Attention over values (V) that are not finite."""
import math

import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from test_gpu_attention import ok, on_device, queries

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
