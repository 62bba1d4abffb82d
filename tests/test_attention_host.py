"""Argument checks of the paged-cache attention entry points (no GPU needed)."""
import ctypes
import math

import pytest

import tensor_transformer_mlp_tmem_gb300 as tp
from tensor_transformer_mlp_tmem_gb300 import _build

INV, SHAPE, MIS, OK = (tp.TPMLP_ERR_INVALID_ARG, tp.TPMLP_ERR_UNSUPPORTED_SHAPE,
                       tp.TPMLP_ERR_MISALIGNED, tp.TPMLP_OK)


@pytest.fixture(scope="module")
def hooks(tmp_path_factory):
    """A test build whose attention contexts hold no device memory (see test_abi_host.py)."""
    path = _build.build(out=str(tmp_path_factory.mktemp("hooks") / "libtpmlp_hooks.so"),
                        extra_flags=["-DTPMLP_TEST_HOOKS"])
    h = ctypes.CDLL(path)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    h.tpmlp_test_attn_context.argtypes = [i32, i32, i32, i32, i32, ctypes.c_uint32]
    h.tpmlp_test_attn_context.restype = vp
    h.tpmlp_test_set_current_device.argtypes = [i32]
    h.tpmlp_last_error.argtypes = [vp]
    h.tpmlp_last_error.restype = ctypes.c_char_p
    h.tpmlp_destroy.argtypes = [vp]
    h.tpmlp_launch_count.argtypes = [vp]
    h.tpmlp_launch_count.restype = i64
    h.tpmlp_attn_create.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i32, ctypes.c_uint32]
    h.tpmlp_attn_set_rope.argtypes = [vp, i32, i32, ctypes.POINTER(ctypes.c_double)]
    h.tpmlp_attn_set_scales.argtypes = [vp, vp, vp, vp]
    h.tpmlp_attn_append.argtypes = [vp, vp, i64, vp, i64, vp, i64, i64, vp, vp, vp, vp, i64, vp]
    h.tpmlp_attn_decode.argtypes = [vp, vp, i64, vp, ctypes.c_float, i32, vp, i64, vp, vp]
    h.tpmlp_attn_prompt.argtypes = [vp, vp, i64, i64, vp, vp, ctypes.c_float, i32, vp, i64, vp, vp]
    yield h
    h.tpmlp_test_set_current_device(-1)


@pytest.fixture
def ctx(hooks):
    hooks.tpmlp_test_set_current_device(3)
    c = hooks.tpmlp_test_attn_context(8, 2, 128, 64, 3, 0)
    yield c
    assert hooks.tpmlp_launch_count(c) == 0
    hooks.tpmlp_test_set_current_device(-1)
    hooks.tpmlp_destroy(c)


def kv(**over):
    f = dict(K=4096, V=8192, num_pages=10, page_stride=0, page_table=256, table_stride=0,
             table_pages=4, B=3, lens=512)
    f.update(over)
    return tp.KvCache(*[f[n] for n, _ in tp.KvCache._fields_])


def decode(h, c, q=64, ldq=1024, cache=None, scale=0.1, window=0, out=128, ldo=1024, lse=None):
    cache = kv() if cache is None else cache
    return h.tpmlp_attn_decode(c, q, ldq, ctypes.byref(cache) if cache else None, scale, window,
                               out, ldo, lse, None)


def prompt(h, c, q=64, ldq=1024, T=5, cu=256, cache=None, scale=0.1, out=128, ldo=1024, lse=None):
    cache = kv() if cache is None else cache
    return h.tpmlp_attn_prompt(c, q, ldq, T, cu, ctypes.byref(cache) if cache else None, scale, 0,
                               out, ldo, lse, None)


def append(h, c, q=64, ldq=1536, k=64, ldk=1536, v=64, ldv=1536, T=3, pos=256, seq=None,
           cache=None, qo=128, ldqo=1024):
    cache = kv() if cache is None else cache
    return h.tpmlp_attn_append(c, q, ldq, k, ldk, v, ldv, T, pos, seq,
                               ctypes.byref(cache) if cache else None, qo, ldqo, None)


def test_create_refuses(hooks):
    out = ctypes.c_void_p()
    make = lambda *a: hooks.tpmlp_attn_create(ctypes.byref(out), *a)  # noqa: E731
    assert hooks.tpmlp_attn_create(None, 8, 2, 128, 64, 0) == INV
    for bad in ((0, 2, 128, 64, 0), (8, 0, 128, 64, 0), (8, 2, 0, 64, 0), (8, 2, 128, 0, 0),
                (8, 2, 128, 64, 0x1), (8, 2, 128, 64, 0x20)):
        assert make(*bad) == INV, bad
    for bad in ((8, 3, 128, 64, 0), (129, 1, 128, 64, 0), (8, 2, 96, 64, 0), (8, 2, 256, 64, 0),
                (8, 2, 128, 8, 0), (8, 2, 128, 48, 0), (8, 2, 128, 512, 0), (1 << 17, 1 << 17, 64, 16, 0)):
        assert make(*bad) == SHAPE, bad
    assert out.value is None


def test_null_context_and_other_kinds(hooks, ctx):
    for f in (decode, prompt, append):
        assert f(hooks, None) == INV
    assert hooks.tpmlp_attn_set_rope(None, 0, 0, None) == INV
    assert hooks.tpmlp_attn_set_scales(None, 16, 16, None) == INV
    # a block context is no attention context, and the other way round
    hooks.tpmlp_test_host_context.restype = ctypes.c_void_p
    block = hooks.tpmlp_test_host_context(ctypes.c_int64(256), ctypes.c_int64(1024), 4, 3, 0, 1, 0)
    try:
        for f in (decode, prompt, append):
            assert f(hooks, ctypes.c_void_p(block)) == INV
    finally:
        hooks.tpmlp_destroy(ctypes.c_void_p(block))
    c = ctypes.c_void_p(ctx)
    i64 = ctypes.c_int64
    for name, args in (("tpmlp_forward", (16, i64(1), i64(64), 16, None)),
                       ("tpmlp_gemm1", (16, i64(64), 16, None)),
                       ("tpmlp_linear_pack", (16, 16, None)),
                       ("tpmlp_linear_forward", (16, i64(64), 16, None)),
                       ("tpmlp_pack_shards", (16, 16, 16, 16, None)),
                       ("tpmlp_reserve", (i64(64),)),
                       ("tpmlp_set_layernorm", (16, 16, ctypes.c_float(1e-5), None))):
        assert getattr(hooks, name)(c, *[ctypes.c_void_p(a) if isinstance(a, int) else a for a in args]) == INV, name


def test_every_call_checks_the_device(hooks, ctx):
    hooks.tpmlp_test_set_current_device(0)
    for f in (decode, prompt, append):
        assert f(hooks, ctx) == INV
        msg = hooks.tpmlp_last_error(ctx).decode()
        assert "device 3" in msg and "device 0" in msg


def test_empty_calls_are_no_ops(hooks, ctx):
    assert decode(hooks, ctx, cache=kv(B=0), q=None, out=None) == OK
    assert prompt(hooks, ctx, T=0, q=None, out=None, cu=None) == OK
    assert prompt(hooks, ctx, cache=kv(B=0)) == OK
    assert append(hooks, ctx, T=0, q=None, k=None, v=None, pos=None, qo=None) == OK


@pytest.mark.parametrize("over,want", [
    (dict(K=None), INV), (dict(V=None), INV), (dict(page_table=None), INV),
    (dict(num_pages=0), INV), (dict(table_pages=0), INV), (dict(table_stride=3), INV),
    (dict(page_stride=2 * 64 * 128 - 8), INV), (dict(K=4104), MIS), (dict(V=8200), MIS),
    (dict(page_stride=2 * 64 * 128 + 4), MIS), (dict(page_table=258), MIS),
    (dict(table_pages=1 << 26), SHAPE), (dict(B=-1), INV),
])
def test_caches_are_checked(hooks, ctx, over, want):
    for f in (decode, prompt, append):
        assert f(hooks, ctx, cache=kv(**over)) == want, f.__name__


def test_lengths_are_checked(hooks, ctx):
    assert decode(hooks, ctx, cache=kv(lens=None)) == INV
    assert prompt(hooks, ctx, cache=kv(lens=None)) == INV
    assert decode(hooks, ctx, cache=kv(lens=514)) == MIS


@pytest.mark.parametrize("f", [decode, prompt])
def test_attend_arguments(hooks, ctx, f):
    assert f(hooks, ctx, cache=False) == INV
    assert f(hooks, ctx, q=None) == INV and f(hooks, ctx, out=None) == INV
    assert f(hooks, ctx, q=72) == MIS and f(hooks, ctx, out=136) == MIS
    assert f(hooks, ctx, ldq=1023) == INV and f(hooks, ctx, ldo=1016) == INV
    assert f(hooks, ctx, ldq=1028) == MIS and f(hooks, ctx, ldo=1028) == MIS
    assert f(hooks, ctx, lse=18) == MIS
    for s in (0.0, -1.0, math.nan, math.inf):
        assert f(hooks, ctx, scale=s) == INV, s


def test_prompt_arguments(hooks, ctx):
    assert prompt(hooks, ctx, T=-1) == INV
    assert prompt(hooks, ctx, cu=None) == INV and prompt(hooks, ctx, cu=257) == MIS
    assert prompt(hooks, ctx, T=1 << 31) == SHAPE


def test_append_arguments(hooks, ctx):
    assert append(hooks, ctx, cache=False) == INV
    assert append(hooks, ctx, T=-1) == INV and append(hooks, ctx, T=1 << 31) == SHAPE
    assert append(hooks, ctx, pos=None) == INV and append(hooks, ctx, pos=257) == MIS
    assert append(hooks, ctx, seq=257) == MIS
    assert append(hooks, ctx, q=None) == INV and append(hooks, ctx, qo=None) == INV
    assert append(hooks, ctx, k=None) == INV and append(hooks, ctx, v=None) == INV
    assert append(hooks, ctx, ldq=1016) == INV and append(hooks, ctx, ldqo=1016) == INV
    assert append(hooks, ctx, ldk=248) == INV and append(hooks, ctx, ldv=248) == INV
    assert append(hooks, ctx, ldk=258) == MIS and append(hooks, ctx, v=72) == MIS


def test_rope_and_scales_arguments(hooks, ctx):
    f = (ctypes.c_double * 64)(*([0.5] * 64))
    rope = hooks.tpmlp_attn_set_rope
    assert rope(ctx, -16, 0, f) == INV and rope(ctx, 64, 0, None) == INV and rope(ctx, 64, 2, f) == INV
    assert rope(ctx, 24, 0, f) == SHAPE and rope(ctx, 144, 0, f) == SHAPE
    assert rope(ctx, 0, 0, None) == OK and rope(ctx, 128, 1, f) == OK and rope(ctx, 48, 0, f) == OK
    f[3] = math.nan
    assert rope(ctx, 64, 0, f) == INV
    assert hooks.tpmlp_attn_set_scales(ctx, 16, 16, None) == INV  # a bf16 cache has no scales
    e4m3 = hooks.tpmlp_test_attn_context(8, 2, 128, 64, 3, 0x10)
    try:
        assert hooks.tpmlp_attn_set_scales(e4m3, None, 16, None) == INV
        assert hooks.tpmlp_attn_set_scales(e4m3, 16, None, None) == INV
    finally:
        hooks.tpmlp_destroy(e4m3)


def test_packed_calls_check_alike(hooks, ctx):
    """The one-structure forms take the fields in the header's order and give the same answers."""
    import struct
    append_args, attend_args = struct.Struct("@PPqPqPqqPPPPqP"), struct.Struct("@PPqqPPdqPqPP")
    cache = kv()
    at = ctypes.addressof(cache)

    def packed(name, layout, *fields):
        buf = ctypes.create_string_buffer(layout.pack(*fields))
        fn = getattr(hooks, name)
        fn.argtypes = [ctypes.c_void_p]
        return fn(ctypes.addressof(buf))

    for name in ("append", "decode", "prompt"):
        fn = getattr(hooks, f"tpmlp_attn_{name}_packed")
        fn.argtypes = [ctypes.c_void_p]
        assert fn(None) == INV

    def app(T=0, ldq=1536, pos=256, c=ctx, q=64):
        return packed("tpmlp_attn_append_packed", append_args, c, q, ldq, 64, 1536, 64, 1536, T,
                      pos, 0, at, 128, 1024, 0)

    assert app() == OK and app(T=-1) == INV and app(T=1, pos=257) == MIS and app(c=0) == INV
    assert app(T=3, ldq=1016) == INV and app(T=3, q=72) == MIS

    def dec(window=0, scale=0.1, ldo=1024, kv_at=at, name="decode", T=5, cu=256):
        return packed(f"tpmlp_attn_{name}_packed", attend_args, ctx, 64, 1024, T, cu, kv_at, scale,
                      window, 128, ldo, 18, 0)  # the Lse address is misaligned: the last check

    for name in ("decode", "prompt"):
        assert dec(name=name) == MIS
        assert dec(name=name, scale=0.0) == INV and dec(name=name, ldo=1016) == INV
        assert dec(name=name, kv_at=0) == INV and dec(name=name, window=1 << 40) == INV
    assert dec(name="prompt", T=0) == OK and dec(name="prompt", T=-1) == INV
