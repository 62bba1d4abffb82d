"""Attention over an e4m3 cache, whose products take queries in fp16: queries of any size that bf16
holds."""
import math

import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from test_gpu_attention import check_rows, ok, on_device, prompt_spans, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [-110, 0, 101, 113, 120])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 2, 128, 64), (12, 1, 128, 16), (8, 2, 64, 32), (40, 2, 64, 64),
                                           (24, 1, 128, 128)])
def test_queries_of_any_size_over_e4m3(lib, k, Hq, Hkv, D, page):
    """Queries times 2^k over keys with scales times 2^-k: the same scores for every k. One row is
    zero throughout."""
    lens, new = [300, 17, 3000], [70, 17, 3]
    c = ref.make(Hkv, D, page, "e4m3", lens, seed=71)
    c["ks"] = (c["ks"].double() * 2.0 ** -k).float()
    T = sum(new)
    q = (queries(T, Hq, D, 71).double() * 2.0 ** k).bfloat16()
    q[1] = 0.0
    assert bool(q.isfinite().all())
    cu = torch.tensor([0, 70, 87, 90], dtype=torch.int32).cuda()
    with tp.Attention(Hq, Hkv, D, page, kv_dtype="e4m3") as attn:
        cache = on_device(c, attn)
        got, lse = attn.decode(q[:3].cuda(), cache, return_lse=True)
        ok(attn)
        check_rows(c, q, got, lse, [(b, b, 0, n) for b, n in enumerate(lens)], Hq, D, 1.0 / math.sqrt(D))
        got, lse = attn.prompt(q.cuda(), cu, cache, return_lse=True)
        ok(attn)
        check_rows(c, q, got, lse, prompt_spans(lens, new, 0)[::4] + [(1, 0, 0, 232)], Hq, D, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 2, 128, 64), (40, 2, 64, 64)])
def test_scores_too_small_for_fp32(lib, Hq, Hkv, D, page):
    """A softmax scale and scales of the keys whose product is 0 in fp32: all weights are alike, and
    masked keys stay masked."""
    lens, new = [300, 17], [70, 17]
    c = ref.make(Hkv, D, page, "e4m3", lens, seed=72)
    c["ks"] = torch.full((Hkv,), 1e-8)
    q = queries(87, Hq, D, 72)
    cu = torch.tensor([0, 70, 87], dtype=torch.int32).cuda()
    with tp.Attention(Hq, Hkv, D, page, kv_dtype="e4m3") as attn:
        cache = on_device(c, attn)
        got, lse = attn.decode(q[:2].cuda(), cache, scale=1e-38, return_lse=True)
        ok(attn)
        check_rows(c, q, got, lse, [(b, b, 0, n) for b, n in enumerate(lens)], Hq, D, 1e-38)
        got, lse = attn.prompt(q.cuda(), cu, cache, scale=1e-38, return_lse=True)
        ok(attn)
        check_rows(c, q, got, lse, prompt_spans(lens, new, 0)[::4], Hq, D, 1e-38)
