"""The operators as a decoder layer of an encoder-decoder uses them: head norms in every append, decode
behind shared prompts and attention to an encoder's states in one captured step, against decode over
page tables that name the shared pages, and other calls of the two contexts in between."""
import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp

pytestmark = pytest.mark.gpu

PAGE, STEPS = 16, 5
PROMPTS, MEMBERS = [96, 16], [4, 2]          # whole pages, and the sequences behind each
STATES = [70, 1, 0, 33, 129, 16]             # the encoder's, of each sequence
B = sum(MEMBERS)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (12, 12, 64), (40, 1, 64)])
def test_steps_in_a_graph(lib, kv, Hq, Hkv, D):
    g = torch.Generator(device="cuda").manual_seed(Hq)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    wide = (Hq + 2 * Hkv) * D
    cut = [Hq * D, Hkv * D, Hkv * D]
    with tp.Attention(Hq, Hkv, D, PAGE, kv_dtype=kv) as own, tp.Attention(Hq, Hkv, D, PAGE, kv_dtype=kv) as cross:
        own.set_rope(D)
        for attn in (own, cross):
            attn.set_norms(1 + normal(D) / 8, 1 + normal(D) / 8)
            if kv == "e4m3":
                scale = torch.full((Hkv,), 1 / 32, device="cuda")
                attn.set_scales(scale, scale)

        # the encoder's states: keys and values alone
        width = -(-max(STATES) // PAGE)
        at = ints(*[i for n in STATES for i in range(n)])
        seq = ints(*[b for b, n in enumerate(STATES) for _ in range(n)])
        states = cross.new_cache(B * width, torch.arange(B * width, device="cuda").int().view(B, width), ints(*STATES))
        x = normal(len(at), 2 * Hkv * D)
        cross.append(None, x[:, :Hkv * D], x[:, Hkv * D:], states, at, seq)

        # the prompts, and full page tables of the sequences: their prompt's pages, then two of their own
        pages = [n // PAGE for n in PROMPTS]
        most = max(pages) + 2
        table = torch.zeros((B, most), dtype=torch.int32, device="cuda")
        own_table = torch.zeros((B, 2), dtype=torch.int32, device="cuda")
        prefix_table = torch.zeros((2, max(pages)), dtype=torch.int32, device="cuda")
        free, b = 0, 0
        for p, n in enumerate(pages):
            prefix_table[p, :n] = torch.arange(free, free + n)
            free += n
        plens = []
        for p, n in enumerate(MEMBERS):
            for _ in range(n):
                table[b, :pages[p]] = prefix_table[p, :pages[p]]
                own_table[b] = torch.arange(free, free + 2)
                table[b, pages[p]:pages[p] + 2] = own_table[b]
                plens.append(PROMPTS[p])
                free, b = free + 2, b + 1
        pos, own_lens = ints(*plens), torch.zeros(B, dtype=torch.int32, device="cuda")
        full = own.new_cache(free, table, pos.clone())
        for pool in (full.K, full.V):
            pool.view(torch.uint8).fill_(0x7F)  # NaN in both types
        prefix = tp.PagedCache(own, full.K, full.V, prefix_table, ints(*PROMPTS))
        behind = tp.PagedCache(own, full.K, full.V, own_table, own_lens)
        cu, cu_cross = ints(0, MEMBERS[0], B), ints(*range(B + 1))
        T = sum(PROMPTS)
        q, k, v = normal(T, wide).split(cut, dim=1)
        own.append(q, k, v, prefix, ints(*[i for n in PROMPTS for i in range(n)]),
                   ints(*[p for p, n in enumerate(PROMPTS) for _ in range(n)]))

        def step(x, q2):
            q, k, v = x.split(cut, dim=1)
            q = own.append(q, k, v, full, pos)   # at its position, behind the prompt
            own_lens.add_(1)
            pos.add_(1)
            a = own.decode_shared(q, behind, prefix, cu)
            return q, a, cross.cross(q2, cu_cross, states)

        own.reserve(B)
        inputs = [(normal(B, wide), normal(B, Hq * D)) for _ in range(STEPS)]
        x, q2 = (t.clone() for t in inputs[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(x, q2)
        for i in range(STEPS):
            x.copy_(inputs[i][0])
            q2.copy_(inputs[i][1])
            graph.replay()
            q, a, c = (t.clone() for t in got)
            assert own_lens.tolist() == [i + 1] * B
            full.lens.copy_(pos)
            want = own.decode(q, full)                  # the same keys, read once for each sequence
            want_cross = cross.decode(q2, states)
            prompt = own.prompt(q, cu_cross, full)      # the contexts' workspaces, used in between
            for attn in (own, cross):
                torch.cuda.synchronize()
                assert attn.status()[0] == tp.TPMLP_OK
            # every one within its output's and its weights' rounding of the definition
            biggest = max(float(t.V.float().nan_to_num().abs().max()) for t in (full, states))
            tol = 2 * biggest * (ref.P_HALF_STEP[kv] + 2.0 ** -8 + 2.0 ** -12) / (32 if kv == "e4m3" else 1)
            for x1, x2 in ((a, want), (a, prompt), (c, want_cross)):
                assert bool(x1.isfinite().all())
                assert float((x1.float() - x2.float()).abs().max()) <= tol
            assert bool((c[2] == 0).all())              # a sequence without states
