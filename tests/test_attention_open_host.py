"""Argument checks of head norms, cross attention and decode behind shared prefixes (no GPU needed)."""
import ctypes
import math
import struct

import pytest

import tensor_transformer_mlp_tmem_gb300 as tp
from test_attention_host import INV, MIS, OK, SHAPE, ctx, hooks as plain_hooks, kv  # noqa: F401


@pytest.fixture(scope="module")
def hooks(plain_hooks):  # noqa: F811
    h = plain_hooks
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    h.tpmlp_attn_set_norms.argtypes = [vp, vp, vp, i32, f32, vp]
    h.tpmlp_attn_cross.argtypes = [vp, vp, i64, i64, vp, vp, f32, vp, i64, vp, vp]
    h.tpmlp_attn_decode_shared.argtypes = [vp, vp, i64, vp, vp, vp, f32, vp, i64, vp, vp]
    h.tpmlp_attn_reserve.argtypes = [vp, i64]
    return h


def at(cache):
    return ctypes.byref(cache) if cache else None


def cross(h, c, q=64, ldq=1024, T=5, cu=256, cache=None, scale=0.1, out=128, ldo=1024, lse=None):
    return h.tpmlp_attn_cross(c, q, ldq, T, cu, at(kv() if cache is None else cache), scale, out, ldo, lse, None)


def shared(h, c, q=64, ldq=1024, prefix=None, cu=256, cache=None, scale=0.1, out=128, ldo=1024, lse=None):
    prefix = kv(B=2) if prefix is None else prefix
    return h.tpmlp_attn_decode_shared(c, q, ldq, at(prefix), cu, at(kv() if cache is None else cache), scale, out,
                                      ldo, lse, None)


CALLS = [cross, shared]


def test_contexts(hooks, ctx):  # noqa: F811
    hooks.tpmlp_test_host_context.restype = ctypes.c_void_p
    block = ctypes.c_void_p(hooks.tpmlp_test_host_context(ctypes.c_int64(256), ctypes.c_int64(1024), 4, 3, 0, 1, 0))
    try:
        for c in (None, block):
            for f in CALLS:
                assert f(hooks, c) == INV
            assert hooks.tpmlp_attn_set_norms(c, 16, 16, 0, 1e-6, None) == INV
            assert hooks.tpmlp_attn_reserve(c, 4) == INV
    finally:
        hooks.tpmlp_destroy(block)
    hooks.tpmlp_test_set_current_device(0)
    for f in CALLS + [lambda h, c: h.tpmlp_attn_set_norms(c, 16, 16, 0, 1e-6, None),
                      lambda h, c: h.tpmlp_attn_reserve(c, 4)]:
        assert f(hooks, ctx) == INV
        msg = hooks.tpmlp_last_error(ctx).decode()
        assert "device 3" in msg and "device 0" in msg


def test_empty_calls_are_no_ops(hooks, ctx):  # noqa: F811
    assert cross(hooks, ctx, T=0, q=None, out=None, cu=None) == OK
    assert cross(hooks, ctx, cache=kv(B=0)) == OK
    assert shared(hooks, ctx, cache=kv(B=0), q=None, out=None, cu=None) == OK
    assert hooks.tpmlp_attn_reserve(ctx, 0) == OK
    assert hooks.tpmlp_attn_set_norms(ctx, None, None, 0, 0.0, None) == OK


@pytest.mark.parametrize("f", CALLS)
def test_attend_arguments(hooks, ctx, f):  # noqa: F811
    assert f(hooks, ctx, cache=False) == INV
    assert f(hooks, ctx, q=None) == INV and f(hooks, ctx, out=None) == INV
    assert f(hooks, ctx, q=72) == MIS and f(hooks, ctx, out=136) == MIS
    assert f(hooks, ctx, ldq=1023) == INV and f(hooks, ctx, ldo=1016) == INV
    assert f(hooks, ctx, ldq=1028) == MIS and f(hooks, ctx, ldo=1028) == MIS
    assert f(hooks, ctx, lse=18) == MIS
    assert f(hooks, ctx, cu=None) == INV and f(hooks, ctx, cu=257) == MIS
    for s in (0.0, -1.0, math.nan, math.inf):
        assert f(hooks, ctx, scale=s) == INV, s


@pytest.mark.parametrize("over,want", [
    (dict(K=None), INV), (dict(V=None), INV), (dict(page_table=None), INV), (dict(lens=None), INV),
    (dict(num_pages=0), INV), (dict(table_pages=0), INV), (dict(table_stride=3), INV),
    (dict(page_stride=2 * 64 * 128 - 8), INV), (dict(K=4104), MIS), (dict(V=8200), MIS),
    (dict(page_stride=2 * 64 * 128 + 4), MIS), (dict(page_table=258), MIS), (dict(lens=514), MIS),
    (dict(table_pages=1 << 26), SHAPE), (dict(B=-1), INV),
])
def test_caches_are_checked(hooks, ctx, over, want):  # noqa: F811
    for f in CALLS:
        assert f(hooks, ctx, cache=kv(**over)) == want, f.__name__
    assert shared(hooks, ctx, prefix=kv(**over)) == want


def test_sizes(hooks, ctx):  # noqa: F811
    assert cross(hooks, ctx, T=-1) == INV and cross(hooks, ctx, T=1 << 31) == SHAPE
    assert shared(hooks, ctx, prefix=False) == INV
    assert shared(hooks, ctx, cache=kv(B=(1 << 31) - 1)) == SHAPE
    assert hooks.tpmlp_attn_reserve(ctx, -1) == INV
    assert hooks.tpmlp_attn_reserve(ctx, 1 << 31) == SHAPE
    # without prefixes it is a decode, with its checks
    assert shared(hooks, ctx, prefix=kv(B=0), cu=None, q=72) == MIS


def test_norm_arguments(hooks, ctx):  # noqa: F811
    norms = hooks.tpmlp_attn_set_norms
    assert norms(ctx, 16, None, 0, 1e-6, None) == INV and norms(ctx, None, 16, 0, 1e-6, None) == INV
    assert norms(ctx, 16, 16, 2, 1e-6, None) == INV
    for eps in (0.0, -1e-6, 1e-13, 1.5, math.nan, math.inf):
        assert norms(ctx, 16, 16, 0, eps, None) == INV, eps
    assert norms(ctx, 24, 16, 0, 1e-6, None) == MIS and norms(ctx, 16, 24, 1, 1e-6, None) == MIS


def test_packed_calls_check_alike(hooks, ctx):  # noqa: F811
    attend, shared_args = struct.Struct("@PPqqPPdqPqPP"), struct.Struct("@PPqPPPdPqPP")
    own, prefix = kv(), kv(B=2)
    a, p = ctypes.addressof(own), ctypes.addressof(prefix)

    def packed(name, layout, *fields):
        buf = ctypes.create_string_buffer(layout.pack(*fields))
        fn = getattr(hooks, name)
        fn.argtypes = [ctypes.c_void_p]
        return fn(ctypes.addressof(buf))

    for name in ("tpmlp_attn_cross_packed", "tpmlp_attn_decode_shared_packed"):
        fn = getattr(hooks, name)
        fn.argtypes = [ctypes.c_void_p]
        assert fn(None) == INV

    def crossed(T=5, window=0, scale=0.1, ldo=1024, cu=256, lse=18):
        return packed("tpmlp_attn_cross_packed", attend, ctx, 64, 1024, T, cu, a, scale, window, 128, ldo, lse, 0)

    assert crossed() == MIS and crossed(T=0) == OK and crossed(T=-1) == INV
    assert crossed(window=4) == INV and crossed(scale=0.0) == INV and crossed(ldo=1016) == INV
    assert crossed(lse=16, cu=0) == INV and crossed(lse=16, cu=257) == MIS

    def behind(cu=256, scale=0.1, ldo=1024, lse=18, prefix_at=p, kv_at=a):
        return packed("tpmlp_attn_decode_shared_packed", shared_args, ctx, 64, 1024, prefix_at, cu, kv_at, scale,
                      128, ldo, lse, 0)

    assert behind() == MIS and behind(prefix_at=0) == INV and behind(kv_at=0) == INV
    assert behind(scale=0.0) == INV and behind(ldo=1016) == INV
    assert behind(lse=16, cu=0) == INV and behind(lse=16, cu=257) == MIS


def test_structure_layouts():
    """The binding packs tpmlp_shared_args in the header's order and size."""
    assert tp._SHARED.size == 11 * 8
