"""Decode steps of several operators against the definition in fp64, each row with its own tolerance, which a
missing key is not within: in a captured graph, and over page tables that name shared pages."""
import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from test_attention_tolerance import rejects_a_missing_key, within
from test_gpu_attention import ok, queries
from test_gpu_attention_cross import starts
from test_gpu_attention_shared import split

pytestmark = pytest.mark.gpu

PAGE, STEPS = 16, 5
PROMPTS, MEMBERS = [96, 16], [4, 2]          # whole pages, and the sequences behind each
STATES = [70, 1, 0, 33, 129, 16]             # an encoder's, of each sequence
B = sum(MEMBERS)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def host(cache, scale):
    """The pools as they are, for attention_ref."""
    Hkv = cache.K.shape[1]
    return dict(K=cache.K.cpu(), V=cache.V.cpu(), table=cache.page_table.cpu(), page=cache.K.shape[2],
                ks=torch.full((Hkv,), scale), vs=torch.full((Hkv,), scale),
                kv="bf16" if cache.K.dtype == torch.bfloat16 else "e4m3")


def check(c, q, got, lens, Hq, D):
    """Row b of got [B, Hq * D] against the definition over the first lens[b] keys of sequence b."""
    for b, n in enumerate(lens):
        x = q[b].cpu().double().view(Hq, D)
        o, _, spread, _ = ref.attend(c, b, x, n, 0, D ** -0.5)
        out = got[b].cpu().double().view(Hq, D)
        assert within(out, o, spread, c["kv"]), (b, n, float(((out - o).abs() / ref.out_tolerance(o, spread, c["kv"])).max()))
        if n > 0:
            assert rejects_a_missing_key(c, b, x, n, D ** -0.5)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (12, 12, 64), (40, 1, 64)])
def test_captured_steps_match_the_definition(lib, kv, Hq, Hkv, D):
    """Head norms in every append, decode behind shared prompts and attention to an encoder's states in one
    captured step, as the own keys grow; NaN wherever nothing has been written."""
    g = torch.Generator(device="cuda").manual_seed(Hq + 1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    def nothing(cache):
        for pool in (cache.K, cache.V):
            if kv == "bf16":
                pool.fill_(float("nan"))
            else:
                pool.view(torch.uint8).fill_(0x7F)
            assert bool(pool.float().isnan().all())
        return cache

    wide, unit = (Hq + 2 * Hkv) * D, 1 / 32 if kv == "e4m3" else 1.0
    cut = [Hq * D, Hkv * D, Hkv * D]
    with tp.Attention(Hq, Hkv, D, PAGE, kv_dtype=kv) as own, tp.Attention(Hq, Hkv, D, PAGE, kv_dtype=kv) as cross:
        own.set_rope(D)
        for attn in (own, cross):
            attn.set_norms(1 + normal(D) / 8, 1 + normal(D) / 8)
            if kv == "e4m3":
                scale = torch.full((Hkv,), unit, device="cuda")
                attn.set_scales(scale, scale)
        width = -(-max(STATES) // PAGE)
        states = nothing(cross.new_cache(B * width, torch.arange(B * width, device="cuda").int().view(B, width),
                                         ints(*STATES)))
        x = normal(sum(STATES), 2 * Hkv * D)
        cross.append(None, x[:, :Hkv * D], x[:, Hkv * D:], states, ints(*[i for n in STATES for i in range(n)]),
                     ints(*[b for b, n in enumerate(STATES) for _ in range(n)]))

        # full page tables of the sequences: their prompt's pages, then two of their own
        pages = [n // PAGE for n in PROMPTS]
        behind_which = [p for p, n in enumerate(MEMBERS) for _ in range(n)]
        prefix_table = torch.zeros((2, max(pages)), dtype=torch.int32)
        prefix_table[0], prefix_table[1, :pages[1]] = torch.arange(pages[0]), torch.arange(pages[1]) + pages[0]
        own_table = (sum(pages) + torch.arange(2 * B, dtype=torch.int32)).view(B, 2)
        table = torch.zeros((B, max(pages) + 2), dtype=torch.int32)
        for b, p in enumerate(behind_which):
            table[b, :pages[p] + 2] = torch.cat([prefix_table[p, :pages[p]], own_table[b]])
        plens = [PROMPTS[p] for p in behind_which]
        pos, own_lens = ints(*plens), torch.zeros(B, dtype=torch.int32, device="cuda")
        full = nothing(own.new_cache(sum(pages) + 2 * B, table.cuda(), pos.clone()))
        prefix = tp.PagedCache(own, full.K, full.V, prefix_table.cuda(), ints(*PROMPTS))
        behind = tp.PagedCache(own, full.K, full.V, own_table.cuda(), own_lens)
        cu, cu_cross = ints(0, MEMBERS[0], B), ints(*range(B + 1))
        q, k, v = normal(sum(PROMPTS), wide).split(cut, dim=1)
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
            for attn in (own, cross):
                ok(attn)
            assert pos.tolist() == [n + i + 1 for n in plens] and own_lens.tolist() == [i + 1] * B
            check(host(full, unit), q, a, pos.tolist(), Hq, D)
            check(host(states, unit), q2, c, STATES, Hq, D)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_decode_behind_a_prefix_and_over_one_table(lib, kv):
    """decode_shared, and decode over tables that name the prefix's pages and then each sequence's own: both
    within each row's tolerance of the definition, which a missing key is not."""
    Hq, Hkv, D, page, prefix, lens = 8, 2, 128, 32, 320, [1, 64, 300]
    c = ref.make(Hkv, D, page, kv, [prefix] + lens, seed=3)
    q = queries(3, Hq, D, 3)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache, shared = split(c, attn, 1)
        a = attn.decode_shared(q.cuda(), cache, shared, starts([3]))
        table = torch.cat([shared.page_table.expand(3, -1)[:, :prefix // page], cache.page_table], 1).contiguous()
        b = attn.decode(q.cuda(), tp.PagedCache(attn, cache.K, cache.V, table, cache.lens + prefix))
        ok(attn)
    one = dict(c, table=table.cpu())
    for got in (a, b):
        check(one, q, got, [prefix + n for n in lens], Hq, D)
