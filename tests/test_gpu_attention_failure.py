"""A wait of the prompt attention that runs out: a test build of the library whose TMA producer
never fills one stage. The waits for it end after about a second each, the kernel records where,
drains the copies and products it has in flight, frees its tensor memory and returns; the host
reads TPMLP_ERR_DEVICE_TIMEOUT. The context stays usable: arrivals that the call left behind at
its split items are cleared with the status, and the next call is right."""
import ctypes
import math

import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from tensor_transformer_mlp_tmem_gb300 import _build

pytestmark = pytest.mark.gpu

PROMPT_SITES = 0x2000  # the kernel records this | the role that gave up


@pytest.fixture(scope="module")
def stall_lib(tmp_path_factory):
    path = _build.build(out=str(tmp_path_factory.mktemp("stall") / "libtpmlp_stall.so"),
                        extra_flags=["-DTPMLP_TEST_SKIP_STAGE=5"])
    dbg = ctypes.CDLL(path)
    vp, i64, i32, u32, f32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32,
                              ctypes.c_float)
    dbg.tpmlp_attn_create.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i32, u32]
    dbg.tpmlp_attn_set_scales.argtypes = [vp, vp, vp, vp]
    dbg.tpmlp_attn_prompt.argtypes = [vp, vp, i64, i64, vp, ctypes.POINTER(tp.KvCache), f32, i32, vp, i64, vp, vp]
    dbg.tpmlp_get_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
    dbg.tpmlp_destroy.argtypes = [vp]
    return dbg


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_prompt_wait_runs_out_and_is_reported(lib, stall_lib, kv):
    Hq, Hkv, D, page, new = 4, 1, 128, 64, 3
    # one item over all CTAs: 500 blocks of keys give most of them four (the stage is met), 150 one
    # or two (it is not)
    longest, shorter = 64000, 19200
    c = ref.make(Hkv, D, page, kv, [longest], seed=41)
    g = torch.Generator().manual_seed(41)
    q = torch.randn((new, Hq * D), generator=g).bfloat16().cuda()
    K, V, table = c["K"].cuda(), c["V"].cuda(), c["table"].cuda()
    lens = torch.tensor([longest], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    scale = 1.0 / math.sqrt(D)
    with tp.Attention(Hq, Hkv, D, page, kv_dtype=kv) as attn:
        if kv == "e4m3":
            attn.set_scales(c["ks"].cuda(), c["vs"].cuda())
        lens[0] = shorter
        want = attn.prompt(q, cu, tp.PagedCache(attn, K, V, table, lens))
        torch.cuda.synchronize()
        assert attn.status()[0] == tp.TPMLP_OK

    view = tp.KvCache(K=K.data_ptr(), V=V.data_ptr(), num_pages=K.shape[0], page_stride=0,
                      page_table=table.data_ptr(), table_stride=0, table_pages=table.shape[1], B=1,
                      lens=lens.data_ptr())
    ctx, detail = ctypes.c_void_p(), ctypes.c_int32(0)
    flags = tp.TPMLP_FLAG_KV_E4M3 if kv == "e4m3" else 0
    assert stall_lib.tpmlp_attn_create(ctypes.byref(ctx), Hq, Hkv, D, page, flags) == 0

    def call():
        assert stall_lib.tpmlp_attn_prompt(ctx, q.data_ptr(), Hq * D, new, cu.data_ptr(), ctypes.byref(view),
                                           scale, 0, out.data_ptr(), Hq * D, None, None) == 0
        return stall_lib.tpmlp_get_status(ctx, None, ctypes.byref(detail))

    try:
        if kv == "e4m3":
            ks, vs = c["ks"].cuda(), c["vs"].cuda()
            assert stall_lib.tpmlp_attn_set_scales(ctx, ks.data_ptr(), vs.data_ptr(), None) == 0
        lens[0] = longest
        torch.cuda.synchronize()
        assert call() == tp.TPMLP_ERR_DEVICE_TIMEOUT
        assert detail.value & ~0xFF == PROMPT_SITES, hex(detail.value)
        lens[0] = shorter
        torch.cuda.synchronize()
        assert call() == tp.TPMLP_OK, hex(detail.value)
        assert torch.equal(out, want)
    finally:
        stall_lib.tpmlp_destroy(ctx)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_bad_page_does_not_hide_a_wait_that_ran_out(lib, stall_lib, kv):
    """The call meets a page outside the pool in its first block of keys, then a wait runs out: the
    caller is told that the call did not end, and of the page beside it."""
    Hq, Hkv, D, page, new, longest = 4, 1, 128, 64, 3, 64000
    c = ref.make(Hkv, D, page, kv, [longest], seed=42)
    q = torch.zeros((new, Hq * D), dtype=torch.bfloat16, device="cuda")
    K, V, table = c["K"].cuda(), c["V"].cuda(), c["table"].cuda()
    table[0, 0] = -1
    lens = torch.tensor([longest], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    view = tp.KvCache(K=K.data_ptr(), V=V.data_ptr(), num_pages=K.shape[0], page_stride=0,
                      page_table=table.data_ptr(), table_stride=0, table_pages=table.shape[1], B=1,
                      lens=lens.data_ptr())
    ctx, detail = ctypes.c_void_p(), ctypes.c_int32(0)
    flags = tp.TPMLP_FLAG_KV_E4M3 if kv == "e4m3" else 0
    assert stall_lib.tpmlp_attn_create(ctypes.byref(ctx), Hq, Hkv, D, page, flags) == 0
    try:
        torch.cuda.synchronize()
        assert stall_lib.tpmlp_attn_prompt(ctx, q.data_ptr(), Hq * D, new, cu.data_ptr(), ctypes.byref(view),
                                           0.1, 0, out.data_ptr(), Hq * D, None, None) == 0
        assert stall_lib.tpmlp_get_status(ctx, None, ctypes.byref(detail)) == tp.TPMLP_ERR_DEVICE_TIMEOUT
        assert detail.value & 0x10000 and detail.value & 0xFF00 == PROMPT_SITES, hex(detail.value)
        assert stall_lib.tpmlp_get_status(ctx, None, ctypes.byref(detail)) == tp.TPMLP_OK
    finally:
        stall_lib.tpmlp_destroy(ctx)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_long_piece_is_not_taken_for_a_wait_that_ran_out(lib, tmp_path_factory, kv):
    """Roles of the prompt kernel that have nothing to do wait for the others' whole piece, however
    long its keys. Here each step's limit is 2 ms and a piece (409600 keys, all on one page) takes
    longer, two of them to a CTA."""
    path = _build.build(out=str(tmp_path_factory.mktemp("short") / "libtpmlp_short.so"),
                        extra_flags=["-DTPMLP_TEST_WAIT_NS=2000000ull"])
    dbg = ctypes.CDLL(path)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    dbg.tpmlp_attn_create.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i32, ctypes.c_uint32]
    dbg.tpmlp_attn_prompt.argtypes = [vp, vp, i64, i64, vp, ctypes.POINTER(tp.KvCache), f32, i32, vp, i64, vp, vp]
    dbg.tpmlp_get_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
    dbg.tpmlp_destroy.argtypes = [vp]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    H, D, page, B, keys = sms, 64, 256, 2, 1600 * 256
    c = ref.make(H, D, page, kv, [page], seed=43, extra_pages=0)
    q = torch.randn((B, H * D), generator=torch.Generator().manual_seed(43)).bfloat16()
    K, V, qd = c["K"].cuda(), c["V"].cuda(), q.cuda()
    table = torch.zeros((B, 1600), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), keys, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(qd), torch.zeros((B, H), device="cuda")
    view = tp.KvCache(K=K.data_ptr(), V=V.data_ptr(), num_pages=K.shape[0], page_stride=0,
                      page_table=table.data_ptr(), table_stride=0, table_pages=1600, B=B, lens=lens.data_ptr())
    c["ks"] = c["vs"] = torch.ones(H)  # as a new context has them
    scale = 0.02 / 60.0 if kv == "e4m3" else 0.02
    ctx, detail = ctypes.c_void_p(), ctypes.c_int32(0)
    assert dbg.tpmlp_attn_create(ctypes.byref(ctx), H, H, D, page, tp.TPMLP_FLAG_KV_E4M3 if kv == "e4m3" else 0) == 0
    try:
        torch.cuda.synchronize()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        assert dbg.tpmlp_attn_prompt(ctx, qd.data_ptr(), H * D, B, cu.data_ptr(), ctypes.byref(view), scale, 0,
                                     out.data_ptr(), H * D, lse.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream) == 0
        end.record()
        rc = dbg.tpmlp_get_status(ctx, torch.cuda.current_stream().cuda_stream, ctypes.byref(detail))
        assert rc == tp.TPMLP_OK, f"{rc} ({detail.value:#x}) after {start.elapsed_time(end):.1f} ms"
        assert start.elapsed_time(end) > 2 * 2.0  # the pieces outlasted the limit
    finally:
        dbg.tpmlp_destroy(ctx)
    # the same weights over one page's keys. O is summed in 4 products a step, 25600 in all, each of
    # which may drop 2^-23 of the sum, all one way at worst; the weights' sum in 6400 steps (2^-24)
    for b in range(B):
        o, l, spread, _ = ref.attend(c, 0, q[b].double().view(H, D), page, 0, scale)
        tol = ref.out_tolerance(o, spread, kv) + (25600 * 2.0 ** -23 + 6400 * 2.0 ** -24) * spread
        assert bool(((out[b].cpu().double().view(H, D) - o).abs() <= tol).all())
        assert bool(((lse[b].cpu().double() - l - math.log(1600)).abs() <= 6400 * 2.0 ** -24 + 2.0 ** -14).all())
