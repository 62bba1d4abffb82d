"""Waits of a tile without rows, behind a piece that outlasts every step's limit (a test build whose limit
is 2 ms): its softmax warps are at the next piece while the other tile goes through this one."""
import ctypes
import math

import pytest
import torch

import attention_ref as ref
import tensor_transformer_mlp_tmem_gb300 as tp
from tensor_transformer_mlp_tmem_gb300 import _build

pytestmark = pytest.mark.gpu

LIMIT_MS, PAGES, PAGE = 2.0, 1600, 256


@pytest.fixture(scope="module")
def short_lib(tmp_path_factory):
    dbg = ctypes.CDLL(_build.build(out=str(tmp_path_factory.mktemp("short") / "libtpmlp_short.so"),
                                   extra_flags=["-DTPMLP_TEST_WAIT_NS=2000000ull"]))
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    kv = ctypes.POINTER(tp.KvCache)
    dbg.tpmlp_attn_create.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i32, ctypes.c_uint32]
    dbg.tpmlp_attn_cross.argtypes = [vp, vp, i64, i64, vp, kv, f32, vp, i64, vp, vp]
    dbg.tpmlp_attn_prompt.argtypes = [vp, vp, i64, i64, vp, kv, f32, i32, vp, i64, vp, vp]
    dbg.tpmlp_get_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
    dbg.tpmlp_destroy.argtypes = [vp]
    return dbg


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("call", ["cross", "prompt"])
def test_a_tile_without_rows_waits_for_the_others_piece(lib, short_lib, kv, call):
    """Two items to a CTA, in turn of 1 and of 200 rows, each on 409600 keys (all on one page): 304 items of
    3201 units on 152 SMs, split in runs of 6402, so that every CTA has one item of one tile and then
    one of two."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    D, keys, B = 64, PAGES * PAGE, 2 * sms
    c = ref.make(1, D, PAGE, kv, [PAGE], seed=47, extra_pages=0)
    c["ks"] = c["vs"] = torch.ones(1)  # as a new context has them
    T = 201 * sms
    q = torch.randn((T, D), generator=torch.Generator().manual_seed(47)).bfloat16()
    K, V, qd = c["K"].cuda(), c["V"].cuda(), q.cuda()
    table = torch.zeros((B, PAGES), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), keys, dtype=torch.int32, device="cuda")
    cu = torch.tensor([201 * (b // 2) + b % 2 for b in range(B + 1)], dtype=torch.int32).cuda()
    out, lse = torch.zeros_like(qd), torch.zeros((T, 1), device="cuda")
    cache = tp.KvCache(K=K.data_ptr(), V=V.data_ptr(), num_pages=1, page_stride=0, page_table=table.data_ptr(),
                       table_stride=0, table_pages=PAGES, B=B, lens=lens.data_ptr())
    scale = 0.02 / 60.0 if kv == "e4m3" else 0.02
    ctx, detail = ctypes.c_void_p(), ctypes.c_int32(0)
    flags = tp.TPMLP_FLAG_KV_E4M3 if kv == "e4m3" else 0
    assert short_lib.tpmlp_attn_create(ctypes.byref(ctx), 1, 1, D, PAGE, flags) == 0
    try:
        torch.cuda.synchronize()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        stream = torch.cuda.current_stream().cuda_stream
        start.record()
        if call == "cross":
            rc = short_lib.tpmlp_attn_cross(ctx, qd.data_ptr(), D, T, cu.data_ptr(), ctypes.byref(cache), scale,
                                            out.data_ptr(), D, lse.data_ptr(), stream)
        else:
            rc = short_lib.tpmlp_attn_prompt(ctx, qd.data_ptr(), D, T, cu.data_ptr(), ctypes.byref(cache), scale, 0,
                                             out.data_ptr(), D, lse.data_ptr(), stream)
        assert rc == 0
        end.record()
        rc = short_lib.tpmlp_get_status(ctx, stream, ctypes.byref(detail))
        assert rc == tp.TPMLP_OK, f"{rc} ({detail.value:#x}) after {start.elapsed_time(end):.1f} ms"
        assert start.elapsed_time(end) > 2 * LIMIT_MS  # the pieces outlasted the limit
    finally:
        short_lib.tpmlp_destroy(ctx)
    # The weights of one page's keys, 1600 times over (a prompt's earlier tokens see the last ones once less). O
    # is summed in 4 products a step, 25600 in all, each of which may drop 2^-23 of the sum, all one way at
    # worst; the weights' sum in 6400 steps (2^-24).
    k, v = (ref.rows_of(c, which, 0, PAGE)[:, 0] for which in ("K", "V"))
    for r in (0, 1, 128, 130, 200, 201, 202, T - 200, T - 1):
        i = r % 201 - 1  # of 200 rows, or -1: a sequence's only one
        seen = keys if call == "cross" or i < 0 else keys - 199 + i
        times = torch.where(torch.arange(PAGE) < seen - (PAGES - 1) * PAGE, PAGES, PAGES - 1).double()
        s = k @ q[r].double() * scale
        w = times * s.exp()
        o, spread, l = w @ v / w.sum(), w @ v.abs() / w.sum(), w.sum().log()
        tol = ref.out_tolerance(o, spread, kv) + (25600 * 2.0 ** -23 + 6400 * 2.0 ** -24) * spread
        err = (out[r].cpu().double() - o).abs()
        assert bool((err <= tol).all()), (r, float((err / tol).max()))
        assert abs(float(lse[r, 0]) - float(l)) <= 6400 * 2.0 ** -24 + 2.0 ** -14, r
