"""A wait of the unmasked attention kernel that runs out (a test build whose TMA producer never fills
one stage): the call ends after about a second, the host reads TPMLP_ERR_DEVICE_TIMEOUT, and the
context stays usable. And a piece that outlasts every step's limit is not taken for one."""
import ctypes
import math

import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from tensor_transformer_mlp_tmem_gb300 import _build

pytestmark = pytest.mark.gpu

OPEN_SITES = 0x4000  # the kernel records this | the role that gave up


def load(path):
    dbg = ctypes.CDLL(path)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    kv = ctypes.POINTER(tp.KvCache)
    dbg.tpmlp_attn_create.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i32, ctypes.c_uint32]
    dbg.tpmlp_attn_set_scales.argtypes = [vp, vp, vp, vp]
    dbg.tpmlp_attn_cross.argtypes = [vp, vp, i64, i64, vp, kv, f32, vp, i64, vp, vp]
    dbg.tpmlp_attn_decode_shared.argtypes = [vp, vp, i64, kv, vp, kv, f32, vp, i64, vp, vp]
    dbg.tpmlp_get_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
    dbg.tpmlp_destroy.argtypes = [vp]
    return dbg


def view(K, V, table, lens):
    return tp.KvCache(K=K.data_ptr(), V=V.data_ptr(), num_pages=K.shape[0], page_stride=0,
                      page_table=table.data_ptr(), table_stride=table.stride(0), table_pages=table.shape[1],
                      B=table.shape[0], lens=lens.data_ptr())


@pytest.fixture(scope="module")
def stall_lib(tmp_path_factory):
    return load(_build.build(out=str(tmp_path_factory.mktemp("stall") / "libtpmlp_stall.so"),
                             extra_flags=["-DTPMLP_TEST_SKIP_STAGE=5"]))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("call", ["cross", "shared"])
def test_wait_runs_out_and_is_reported(lib, stall_lib, kv, call):
    """One item over all CTAs: 500 blocks of keys give most of them three or four (the stage is met), 150
    one (it is not). The second call, with fewer keys, is right."""
    Hq, Hkv, D, page, rows = 4, 1, 128, 64, 20  # (more rows than the row kernel takes)
    longest, shorter = 64000, 19200
    c = ref.make(Hkv, D, page, kv, [longest] + [(40, 7, 300)[b % 3] for b in range(rows)], seed=41)
    q = torch.randn((rows, Hq * D), generator=torch.Generator().manual_seed(41)).bfloat16().cuda()
    K, V, table, lens = c["K"].cuda(), c["V"].cuda(), c["table"].cuda(), c["lens"].cuda()
    cu = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    out, scale = torch.zeros_like(q), 1.0 / math.sqrt(D)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        if kv == "e4m3":
            attn.set_scales(c["ks"].cuda(), c["vs"].cuda())
        lens[0] = shorter
        first = tp.PagedCache(attn, K, V, table[:1], lens[:1])
        want = (attn.cross(q, cu, first) if call == "cross" else
                attn.decode_shared(q, tp.PagedCache(attn, K, V, table[1:], lens[1:].clone()), first, cu))
        torch.cuda.synchronize()
        assert attn.status()[0] == tp.TPMLP_OK

    prefix, own_lens = view(K, V, table[:1], lens), lens[1:].clone()
    own = view(K, V, table[1:], own_lens)
    ctx, detail = ctypes.c_void_p(), ctypes.c_int32(0)
    flags = tp.TPMLP_FLAG_KV_E4M3 if kv == "e4m3" else 0
    assert stall_lib.tpmlp_attn_create(ctypes.byref(ctx), Hq, Hkv, D, page, flags) == 0

    def run():
        if call == "cross":
            rc = stall_lib.tpmlp_attn_cross(ctx, q.data_ptr(), Hq * D, rows, cu.data_ptr(), ctypes.byref(prefix), scale,
                                            out.data_ptr(), Hq * D, None, None)
        else:
            rc = stall_lib.tpmlp_attn_decode_shared(ctx, q.data_ptr(), Hq * D, ctypes.byref(prefix), cu.data_ptr(),
                                                    ctypes.byref(own), scale, out.data_ptr(), Hq * D, None, None)
        assert rc == 0
        return stall_lib.tpmlp_get_status(ctx, None, ctypes.byref(detail))

    try:
        if kv == "e4m3":
            ks, vs = c["ks"].cuda(), c["vs"].cuda()
            assert stall_lib.tpmlp_attn_set_scales(ctx, ks.data_ptr(), vs.data_ptr(), None) == 0
        lens[0] = longest
        torch.cuda.synchronize()
        assert run() == tp.TPMLP_ERR_DEVICE_TIMEOUT
        assert detail.value & ~0xFF == OPEN_SITES, hex(detail.value)
        lens[0] = shorter
        torch.cuda.synchronize()
        assert run() == tp.TPMLP_OK, hex(detail.value)
        assert torch.equal(out, want)
    finally:
        stall_lib.tpmlp_destroy(ctx)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_long_piece_is_not_taken_for_a_wait_that_ran_out(lib, tmp_path_factory, kv):
    """Roles that have nothing to do wait for the others' whole piece, however long its keys. Here each
    step's limit is 2 ms and a piece (409600 keys, all on one page) takes longer, two of them to a CTA:
    the second sequence has rows for both tiles, the first for one."""
    dbg = load(_build.build(out=str(tmp_path_factory.mktemp("short") / "libtpmlp_short.so"),
                            extra_flags=["-DTPMLP_TEST_WAIT_NS=2000000ull"]))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    H, D, page, B, keys, rows = sms, 64, 256, 2, 1600 * 256, (1, 200)
    c = ref.make(H, D, page, kv, [page], seed=43, extra_pages=0)
    q = torch.randn((sum(rows), H * D), generator=torch.Generator().manual_seed(43)).bfloat16()
    K, V, qd = c["K"].cuda(), c["V"].cuda(), q.cuda()
    table = torch.zeros((B, 1600), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), keys, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1, 201], dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(qd), torch.zeros((sum(rows), H), device="cuda")
    cache = view(K, V, table, lens)
    c["ks"] = c["vs"] = torch.ones(H)  # as a new context has them
    scale = 0.02 / 60.0 if kv == "e4m3" else 0.02
    ctx, detail = ctypes.c_void_p(), ctypes.c_int32(0)
    assert dbg.tpmlp_attn_create(ctypes.byref(ctx), H, H, D, page, tp.TPMLP_FLAG_KV_E4M3 if kv == "e4m3" else 0) == 0
    try:
        torch.cuda.synchronize()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        stream = torch.cuda.current_stream().cuda_stream
        start.record()
        assert dbg.tpmlp_attn_cross(ctx, qd.data_ptr(), H * D, sum(rows), cu.data_ptr(), ctypes.byref(cache), scale,
                                    out.data_ptr(), H * D, lse.data_ptr(), stream) == 0
        end.record()
        rc = dbg.tpmlp_get_status(ctx, stream, ctypes.byref(detail))
        assert rc == tp.TPMLP_OK, f"{rc} ({detail.value:#x}) after {start.elapsed_time(end):.1f} ms"
        assert start.elapsed_time(end) > 2 * 2.0  # the pieces outlasted the limit
    finally:
        dbg.tpmlp_destroy(ctx)
    # the same weights over one page's keys. O is summed in 4 products a step, 25600 in all, each of
    # which may drop 2^-23 of the sum, all one way at worst; the weights' sum in 6400 steps (2^-24)
    for r in (0, 1, 130, 200):
        o, l, spread, _ = ref.attend(c, 0, q[r].double().view(H, D), page, 0, scale)
        tol = ref.out_tolerance(o, spread, kv) + (25600 * 2.0 ** -23 + 6400 * 2.0 ** -24) * spread
        assert bool(((out[r].cpu().double().view(H, D) - o).abs() <= tol).all())
        assert bool(((lse[r].cpu().double() - l - math.log(1600)).abs() <= 6400 * 2.0 ** -24 + 2.0 ** -14).all())
