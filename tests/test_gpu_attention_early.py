"""Calls whose lengths, tables, offsets and scales the kernels just before have written, and prefixes in pools
of their own."""
import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from test_gpu_attention import ok, queries
from test_gpu_attention_cross import starts
from test_gpu_attention_shared import split

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("wide", [False, True])
def test_lengths_tables_and_offsets_written_just_before(lib, kv, wide):
    """The call's kernels start before those ahead of them have ended, and read lengths, tables, offsets and
    scales that these have just written: back to back as with a pause after each."""
    Hq, Hkv, D, page = (40, 1, 64, 16) if wide else (8, 2, 64, 16)
    prefix, lens = [200, 70, 33], [48] * 20
    c = ref.make(Hkv, D, page, kv, prefix + lens, seed=23)
    q = queries(20, Hq, D, 23).cuda()
    g = torch.Generator().manual_seed(23)
    rounds = []
    for i in range(16):
        order = torch.randperm(20, generator=g)
        cut = sorted(torch.randint(0, 21, (4,), generator=g).tolist())
        rounds.append((torch.randint(0, 49, (20,), generator=g).int().cuda(), c["table"][3:][order].cuda(),
                       torch.tensor(cut, dtype=torch.int32).cuda(), (1 + torch.rand(Hkv, generator=g)).cuda() / 64))
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache, shared = split(c, attn, 3)
        cache = tp.PagedCache(attn, cache.K, cache.V, cache.page_table.clone(), cache.lens.clone())
        cu = starts([1, 2, 3])

        def step(lens, table, offsets, scale):
            cache.lens.copy_(lens)
            cache.page_table.copy_(table)
            cu.copy_(offsets)
            if kv == "e4m3":
                attn.set_scales(scale, scale)
            return attn.decode_shared(q, cache, shared, cu), attn.cross(q, cu, shared)

        def pick(pair, offsets):  # (rows of no prefix are not written by cross)
            return pair[0], pair[1][int(offsets[0]):int(offsets[-1])]

        slow = []
        for r in rounds:
            slow.append(step(*r))
            torch.cuda.synchronize()
        fast = [step(*r) for r in rounds]
        ok(attn)
    for r, x, y in zip(rounds, slow, fast):
        assert all(torch.equal(a, b) for a, b in zip(pick(x, r[2]), pick(y, r[2])))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("members", [[3, 2], [40, 1]])
def test_prefixes_in_pools_of_their_own(lib, kv, members):
    """The prefixes' pools may be others than the sequences', with pages as far apart as they like."""
    Hq, Hkv, D, page, prefix = 6, 2, 128, 32, [300, 65]
    lens = [(17 * b) % 90 for b in range(sum(members))]
    c = ref.make(Hkv, D, page, kv, prefix + lens, seed=29)
    q = queries(len(lens), Hq, D, 29).cuda()
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        cache, shared = split(c, attn, 2)
        want, lse = attn.decode_shared(q, cache, shared, starts(members), return_lse=True)
        ids = shared.page_table[shared.page_table >= 0].long()
        table = torch.full_like(shared.page_table, -1)
        table[shared.page_table >= 0] = torch.arange(len(ids), dtype=torch.int32, device="cuda")
        pools = []
        for pool in (shared.K, shared.V):
            apart = torch.empty((len(ids), 3, Hkv, page, D), dtype=pool.dtype, device="cuda")
            apart.view(torch.uint8).fill_(0x7F)
            apart[:, 0] = pool[ids]
            pools.append(apart[:, 0])
        other = tp.PagedCache(attn, *pools, table, shared.lens)
        got, lse2 = attn.decode_shared(q, cache, other, starts(members), return_lse=True)
        ok(attn)
        assert torch.equal(got, want) and torch.equal(lse, lse2)
