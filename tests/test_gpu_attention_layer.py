"""The attention operators in a layer (examples/serve_layer.py), and the Python classes' checks."""
import importlib.util
import os

import pytest
import torch

import tensor_transformer_mlp_tmem_gb300 as tp

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "serve_layer", os.path.join(ROOT, "examples", "serve_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_generated_rows_match_one_pass(lib, kv):
    """Decode steps in a captured graph give what one pass over the whole sequences gives. The
    two take the same rounded keys and values (the projections' GEMMs differ in summation order
    with the token count: a bf16 half step, 2^-8, now and then, in each of a few tensors)."""
    got, want = example().generate(kv)
    assert bool(got.isfinite().all())
    off = (got.float() - want.float()).norm(dim=-1) / want.float().norm(dim=-1)
    assert float(off.max()) < 1e-2


def test_classes_refuse_what_the_kernels_cannot_read(lib):
    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    with pytest.raises(ValueError, match="kv_dtype"):
        tp.Attention(4, 2, 64, 16, kv_dtype="int8")
    with pytest.raises(tp.TpmlpError) as e:
        tp.Attention(4, 3, 64, 16)
    assert e.value.status == tp.TPMLP_ERR_UNSUPPORTED_SHAPE
    with tp.Attention(4, 2, 64, 16) as attn, tp.Attention(4, 2, 64, 32) as other:
        table, lens = torch.zeros((2, 3), dtype=torch.int32, device="cuda"), ints(5, 7)
        cache = attn.new_cache(8, table, lens)
        K = cache.K
        bad = [
            (K.cpu(), K, table, lens, TypeError), (K, K.float(), table, lens, ValueError),
            (K[:, :1], K, table, lens, ValueError), (K, K[:4], table, lens, ValueError),
            (K.transpose(2, 3), K, table, lens, ValueError),
            (K[:1].expand(8, -1, -1, -1), K, table, lens, ValueError),
            (K, K, table.cpu(), lens, TypeError), (K, K, table.long(), lens, ValueError),
            (K, K, table[:1].expand(2, -1), lens, ValueError), (K, K, table, lens[:1], ValueError),
            (K, K, table, lens.long(), ValueError),
        ]
        for k, v, t, n, error in bad:
            with pytest.raises(error):
                tp.PagedCache(attn, k, v, t, n)
        q = torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda")
        for x, error in ((q.cpu(), TypeError), (q.float(), ValueError), (q[:1], ValueError),
                         (q[:, :128], ValueError), (q.t().contiguous().t(), ValueError)):
            with pytest.raises(error):
                attn.decode(x, cache)
            with pytest.raises(error):
                attn.decode(q, cache, out=x)
        with pytest.raises(ValueError, match="another head layout"):
            other.decode(q, cache)
        with pytest.raises(ValueError, match="cu_q"):
            attn.prompt(q, ints(0, 2), cache)
        kv = q[:, :128]
        with pytest.raises(ValueError, match="pos"):
            attn.append(q, kv, kv, cache, ints(0))
        with pytest.raises(ValueError, match="seq"):
            attn.append(q, kv, kv, cache, ints(0, 1), ints(0))
        with pytest.raises(ValueError, match="freq"):
            attn.set_rope(64, freq=[1.0])
        with pytest.raises(tp.TpmlpError):
            attn.decode(q, cache, scale=0.0)
        with pytest.raises(tp.TpmlpError):
            attn.set_scales(torch.ones(2, device="cuda"), torch.ones(2, device="cuda"))
        # none of it reached the device
        assert attn.launches == 0 and attn.status()[0] == tp.TPMLP_OK
        # pools that are one tensor, and a table that is a part of a wider one
        both = torch.zeros((8, 2, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
        wide = torch.zeros((2, 7), dtype=torch.int32, device="cuda")
        wide[:, 2:5] = ints(3, 1, 6)
        part = tp.PagedCache(attn, both[:, 0], both[:, 1], wide[:, 2:5], lens)
        g = torch.Generator(device="cuda").manual_seed(1)
        x = torch.randn((5, 512), generator=g, device="cuda").bfloat16()
        pos, seq = ints(0, 1, 2, 3, 4), ints(0, 0, 0, 0, 0)
        dense = tp.PagedCache(attn, torch.zeros_like(K), torch.zeros_like(K), wide[:, 2:5].contiguous(), lens)
        for c in (part, dense):
            attn.append(None, x[:, :128], x[:, 128:256], c, pos, seq)
        lens[1] = 0
        assert torch.equal(attn.decode(q + 1, part), attn.decode(q + 1, dense))
        assert torch.equal(both[:, 0], dense.K) and torch.equal(both[:, 1], dense.V)
        assert attn.status()[0] == tp.TPMLP_OK
