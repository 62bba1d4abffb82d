"""The attention calls on a stream that is not the current one."""
import pytest
import torch

import tensor_transformer_mlp_tmem_gb300 as tp
from test_gpu_attention import ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("call", ["append", "decode", "prompt"])
def test_results_on_a_side_stream_are_memory_of_their_own(lib, call, raw):
    """The current stream frees tensors of the results' size while work on them is still pending, then
    a call on a side stream makes its results: the pending work does not reach them."""
    Hq, Hkv, D, page, B = 4, 2, 64, 16, 300
    g = torch.Generator(device="cuda").manual_seed(81)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    q, k = normal(B, Hq * D), normal(B, Hkv * D)
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    lens, pos, cu = ints([5] * B), ints([4] * B), ints(list(range(B + 1)))
    with tp.Attention(Hq, Hkv, D, page) as attn:
        cache = tp.PagedCache(attn, normal(B, Hkv, page, D), normal(B, Hkv, page, D), table, lens)
        attn.append(None, k, k, cache, pos)

        def run(stream=None):
            if call == "append":
                return (attn.append(q, k, k, cache, pos, stream=stream),)
            if call == "decode":
                return attn.decode(q, cache, return_lse=True, stream=stream)
            return attn.prompt(q, cu, cache, return_lse=True, stream=stream)

        want = [x.clone() for x in run()]
        ok(attn)
        side = torch.cuda.Stream()
        torch.cuda._sleep(1 << 27)  # tens of milliseconds
        for _ in range(4):
            for x in [torch.empty_like(w) for w in want for _ in range(8)]:
                x.fill_(7.0)
        got = run(side.cuda_stream if raw else side)
        torch.cuda.synchronize()
        ok(attn)
        for x, w in zip(got, want):
            assert torch.equal(x, w)
        assert all(x.device.type == "cuda" for x in got)
