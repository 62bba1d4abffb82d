"""Head norms where a head's size and its weights lie far apart, and captured appends when norms of the
other kind are set."""
import pytest
import torch

import tensor_transformer_mlp_tmem_gb300 as tp
from test_gpu_attention import ok
from test_gpu_attention_norms import check, normed, one_token, slack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size,weight,eps", [
    (3e38, -16, 1e-6), (3e38, -20, 1e-6), (1e37, -30, 1e-6), (1e30, -40, 1e-6),  # large heads, small weights
    (1e-20, 120, 2.0 ** -40), (0.0, 120, 2.0 ** -40), (1e-3, 100, 1e-6),         # small heads, large weights
    (1.0, -100, 1.0), (3e38, 100, 1e-6),
])
def test_weights_far_from_the_heads(lib, D, size, weight, eps):
    """x over its root mean square is an ordinary number, whatever x; only then come the weights. The
    root's reciprocal may be subnormal (2^-128, half a step 2^-150: 2^-22 of it, inside the slack)."""
    g = torch.Generator().manual_seed(weight + 200)
    x = (torch.randn(D, generator=g).clamp(-1, 1) * size).bfloat16()
    w = ((1 + torch.rand(D, generator=g)) * 2.0 ** weight).bfloat16()
    want = normed(x.double(), w.double(), torch.tensor(eps, dtype=torch.float32).double())
    check(one_token(x, w, eps=eps), want, 2.0 ** -8, slack(want) + 2.0 ** -126)


@pytest.mark.parametrize("first", [False, True])
def test_captured_appends_keep_their_kind_of_weights(lib, first):
    """A captured append with weights per head (first) or shared reads those that the last call of its kind
    has set; calls of the other kind, and none at all, change nothing of it."""
    Hq, Hkv, D, T = 6, 2, 64, 11
    g = torch.Generator().manual_seed(15)
    x = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g).bfloat16().cuda()
    q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], dim=1)
    pos, seq = torch.arange(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")

    def weights(per_head):
        return tuple(torch.randn((n, D) if per_head else (D,), generator=g).bfloat16().cuda() for n in (Hq, Hkv))

    with tp.Attention(Hq, Hkv, D, 16) as attn:
        attn.set_rope(D)
        pool = torch.zeros((1, Hkv, 16, D), dtype=torch.bfloat16, device="cuda")
        cache = tp.PagedCache(attn, pool, pool.clone(), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                              torch.tensor([T], dtype=torch.int32, device="cuda"))

        def run():
            out = attn.append(q, k, v, cache, pos, seq)
            ok(attn)
            return out, cache.K.clone()

        attn.set_norms(*weights(first))
        want = run()
        graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want[0])
        with torch.cuda.graph(graph):
            attn.append(q, k, v, cache, pos, seq, q_out=out)

        def replay():
            cache.K.zero_()
            out.zero_()
            graph.replay()
            ok(attn)
            return out.clone(), cache.K.clone()

        def same(a, b):
            return all(torch.equal(x, y) for x, y in zip(a, b))

        assert same(replay(), want)
        attn.set_norms(*weights(not first))
        other = run()
        assert not same(other, want)
        assert same(replay(), want)          # the other kind's: nothing of this graph's
        attn.set_norms(None, None)
        assert same(replay(), want)
        attn.set_norms(*weights(first))
        again = run()
        assert not same(again, want)
        assert same(replay(), again)         # the last ones of its own kind
        attn.set_norms(*weights(not first), eps=0.5)
        assert not same(run(), other)
        assert same(replay(), again)
