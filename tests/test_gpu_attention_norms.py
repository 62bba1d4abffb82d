"""Append with norms of the query and key heads on the GPU against the formula in fp64."""
import math

import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from test_gpu_attention import ok, on_device

pytestmark = pytest.mark.gpu

EPS = 1e-6


def normed(x, w, eps=EPS):
    """x fp64 [T, heads, D]; w fp64 [D] or [heads, D]."""
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w


def weights(heads, D, per_head, g):
    return (1 + torch.randn((heads, D) if per_head else (D,), generator=g) / 2).bfloat16()


def slack(x):
    """fp32 of the norm and the rotation: a head's sum of squares in 20 steps, halved by the root
    (2^-20.7), its reciprocal root (2^-22), two products and the two of the rotation, sines to 2^-21:
    2^-18.4 of the head's largest value."""
    return x.abs().amax(-1, keepdim=True) * 2.0 ** -18 + 1e-35


def check(got, want, half, more=0.0):
    err = (got - want).abs()
    tol = want.abs() * half + more
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D,page,rot,interleaved,per_head,T", [
    (4, 4, 128, 16, 128, False, False, 1),
    (32, 32, 128, 16, 128, False, True, 3),
    (12, 2, 64, 32, 64, True, True, 37),
    (5, 5, 64, 16, 32, False, False, 130),
    (15, 3, 128, 64, 48, True, True, 65),
    (16, 1, 128, 256, 96, False, False, 9),
    (3, 1, 64, 128, 0, False, True, 7),
    (1, 1, 64, 64, 64, False, True, 9001),       # several tokens to a block
    (2, 1, 128, 64, 64, True, False, 9001),
])
def test_matches_formula(lib, kv, Hq, Hkv, D, page, rot, interleaved, per_head, T):
    g = torch.Generator().manual_seed(T + Hq)
    lens = [T // 2 + 60, 1, T - T // 2 + 77]
    c = ref.make(Hkv, D, page, kv, lens, seed=T)
    width = (Hq + 2 * Hkv) * D
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g) * (torch.rand((T, Hq + 2 * Hkv, 1), generator=g) * 4)
    qkv = torch.cat([qkv.reshape(T, width), torch.zeros(T, 8)], 1).bfloat16()  # wider rows
    places = [(b, p) for b, n in enumerate(lens) for p in range(n)]
    pick = torch.randperm(len(places), generator=g)[:T].tolist()
    seq = torch.tensor([places[i][0] for i in pick], dtype=torch.int32)
    pos = torch.tensor([places[i][1] for i in pick], dtype=torch.int32)
    if T > 5:
        pos[::5] = -1  # skipped tokens
    wq, wk = weights(Hq, D, per_head, g), weights(Hkv, D, per_head, g)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        if rot:
            attn.set_rope(rot, interleaved=interleaved)
        attn.set_norms(wq.cuda(), wk.cuda(), EPS)
        cache = on_device(c, attn)
        d = qkv.cuda()
        q, k, v = d[:, :Hq * D], d[:, Hq * D:(Hq + Hkv) * D], d[:, (Hq + Hkv) * D:width]
        q_out = torch.full((T, Hq * D), 7.0, dtype=torch.bfloat16, device="cuda")
        attn.append(q, k, v, cache, pos.cuda(), seq.cuda(), q_out=q_out)
        ok(attn)
        K, V = cache.K.cpu().float().double(), cache.V.cpu().float().double()
        kept = pos >= 0
        # keys alone give the same keys; in place gives the same queries
        cache.K.view(torch.uint8).zero_()
        assert attn.append(None, k, v, cache, pos.cuda(), seq.cuda()) is None
        inplace = attn.append(q, k, v, cache, pos.cuda(), seq.cuda(), q_out=q)
        ok(attn)
        assert torch.equal(inplace[kept], q_out[kept]) and bool((q_out[~kept] == 7.0).all())
        sl, pg = pos[kept].long() % page, c["table"][seq[kept].long(), pos[kept].long() // page].long()
        again = cache.K.cpu().float().double()[pg, :, sl]
        assert torch.equal(again, K[pg, :, sl])
    x = qkv.double()
    wantq = normed(x[:, :Hq * D].view(T, Hq, D), wq.double())
    wantk = normed(x[:, Hq * D:(Hq + Hkv) * D].reshape(T, Hkv, D), wk.double())
    sq, sk = slack(wantq)[kept], slack(wantk)[kept]
    if rot:
        freq = [1e4 ** (-2 * i / rot) for i in range(rot // 2)]
        wantq, wantk = (ref.rotate(y, pos, rot, interleaved, freq) for y in (wantq, wantk))
    check(q_out.cpu().double().view(T, Hq, D)[kept], wantq[kept], ref.HALF_STEP["bf16"], sq)
    ks, vs = c["ks"].double()[:, None], c["vs"].double()[:, None]
    wantk, wantv = wantk[kept] / ks, x[kept][:, (Hq + Hkv) * D:width].reshape(-1, Hkv, D) / vs
    if kv == "e4m3":  # held to 448; half of the smallest step, 2^-9
        wantk, wantv, low = wantk.clamp(-448, 448), wantv.clamp(-448, 448), 2.0 ** -10
    else:
        low = 0.0
    check(K[pg, :, sl], wantk, ref.HALF_STEP[kv], sk / ks + low)
    check(V[pg, :, sl], wantv, ref.HALF_STEP[kv], wantv.abs() * 2.0 ** -22 + low)


def one_token(x, w, **kw):
    """q_out of one token whose one head is x [D], without a rotation."""
    D = x.numel()
    with tp.Attention(1, 1, D, 16) as attn:
        attn.set_norms(w.cuda(), w.cuda(), **kw)
        K = torch.zeros((1, 1, 16, D), dtype=torch.bfloat16, device="cuda")
        cache = tp.PagedCache(attn, K, K.clone(), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                              torch.ones(1, dtype=torch.int32, device="cuda"))
        x = x.bfloat16().view(1, D).cuda()
        out = attn.append(x, x, x, cache, torch.zeros(1, dtype=torch.int32, device="cuda"))
        ok(attn)
        torch.testing.assert_close(cache.K[0, 0, 0], out[0], rtol=0, atol=0, equal_nan=True)
        torch.testing.assert_close(cache.V[0, 0, 0], x[0], rtol=0, atol=0, equal_nan=True)  # as they are
        return out[0].cpu().double()


@pytest.mark.parametrize("size", [3e38, 1e30, 1e19, 1e-3, 1e-20, 1e-38, 0.0])
@pytest.mark.parametrize("eps", [2.0 ** -40, 1e-6, 1.0])
def test_sizes_of_inputs(lib, size, eps):
    """Squares that leave fp32's range, and heads beside which eps counts."""
    g = torch.Generator().manual_seed(3)
    for D in (64, 128):
        x = (torch.randn(D, generator=g).clamp(-1, 1) * size).bfloat16()
        w = weights(1, D, False, g)
        want = normed(x.double(), w.double(), torch.tensor(eps, dtype=torch.float32).double())
        # (fp32 results below 2^-126 may be flushed)
        check(one_token(x, w, eps=eps), want, 2.0 ** -8, slack(want) + 2.0 ** -126)


def test_values_that_are_not_finite(lib):
    w = torch.ones(64, dtype=torch.bfloat16)
    x = torch.ones(64)
    x[5] = math.inf
    got = one_token(x, w)
    assert bool(got[5].isnan()) and bool((got[torch.arange(64) != 5] == 0).all())
    x[5] = math.nan
    assert bool(one_token(x, w).isnan().all())


def test_a_head_touches_no_other(lib):
    """Heads of NaN beside heads of numbers, in both parts of a block's work."""
    Hq, Hkv, D, T = 9, 3, 64, 5
    g = torch.Generator().manual_seed(8)
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=g)
    bad = torch.rand((T, Hq + Hkv), generator=g) < 0.4
    x[:, :Hq + Hkv][bad] = math.nan
    x = x.bfloat16()
    with tp.Attention(Hq, Hkv, D, 16) as attn:
        w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
        attn.set_norms(w, w)
        K = torch.zeros((5, Hkv, 16, D), dtype=torch.bfloat16, device="cuda")
        cache = tp.PagedCache(attn, K, K.clone(), torch.arange(5, dtype=torch.int32, device="cuda")[:, None],
                              torch.ones(5, dtype=torch.int32, device="cuda"))
        d = x.view(T, -1).cuda()
        out = attn.append(d[:, :Hq * D], d[:, Hq * D:(Hq + Hkv) * D], d[:, (Hq + Hkv) * D:], cache,
                          torch.zeros(5, dtype=torch.int32, device="cuda"))
        ok(attn)
        nan_q, nan_k = out.view(T, Hq, D).isnan().cpu(), cache.K[:, :, 0].isnan().cpu()
    assert torch.equal(nan_q, bad[:, :Hq, None].expand(-1, -1, D))
    assert torch.equal(nan_k, bad[:, Hq:, None].expand(-1, -1, D))


def test_norms_are_set_replaced_and_dropped(lib):
    """Appends follow the last call; without norms they give what they gave before; a captured append
    reads the last weights."""
    Hq, Hkv, D, T = 6, 2, 128, 11
    g = torch.Generator().manual_seed(5)
    x = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g).bfloat16().cuda()
    q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], dim=1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    ones = torch.ones(D, dtype=torch.bfloat16, device="cuda")

    def run(attn, cache):
        out = attn.append(q, k, v, cache, pos, seq)
        ok(attn)
        return out, cache.K.clone()

    with tp.Attention(Hq, Hkv, D, 16) as attn:
        attn.set_rope(D)
        table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
        cache = tp.PagedCache(attn, torch.zeros((1, Hkv, 16, D), dtype=torch.bfloat16, device="cuda"),
                              torch.zeros((1, Hkv, 16, D), dtype=torch.bfloat16, device="cuda"), table,
                              torch.tensor([T], dtype=torch.int32, device="cuda"))
        plain = run(attn, cache)
        attn.set_norms(ones, ones)
        once = run(attn, cache)
        assert not torch.equal(once[0], plain[0])
        graph = torch.cuda.CUDAGraph()
        out = torch.empty_like(once[0])
        with torch.cuda.graph(graph):
            attn.append(q, k, v, cache, pos, seq, q_out=out)
        graph.replay()
        ok(attn)
        assert torch.equal(out, once[0])
        attn.set_norms(2 * ones, 4 * ones)  # powers of two: exact
        twice = run(attn, cache)
        assert torch.equal(twice[0], 2 * once[0]) and torch.equal(twice[1], 4 * once[1])
        graph.replay()
        ok(attn)
        assert torch.equal(out, twice[0])
        per_head = torch.arange(1, Hq + 1, device="cuda").exp2().bfloat16()[:, None] * ones
        attn.set_norms(per_head, 4 * ones.expand(Hkv, D).contiguous())
        each = run(attn, cache)
        assert torch.equal(each[0].view(T, Hq, D), once[0].view(T, Hq, D) * per_head) and torch.equal(each[1], twice[1])
        attn.set_norms(None, None)
        assert all(torch.equal(a, b) for a, b in zip(run(attn, cache), plain))
        for bad in ((ones, None), (None, ones), (ones, per_head), (ones[:64], ones), (ones.float(), ones.float()),
                    (per_head, per_head)):
            with pytest.raises((TypeError, ValueError)):
                attn.set_norms(*bad)


def test_first_set_norms_is_refused_under_capture(lib):
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    with tp.Attention(1, 1, 64, 16) as attn:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(tp.TpmlpError, match="capture"):
                attn.set_norms(w, w)
