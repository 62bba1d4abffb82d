"""Workspaces of decode behind shared prefixes, on a fake of the CUDA runtime (fake_cuda.h): cleared
before the call returns, whatever streams do; kept when they grow; refused without memory."""
import ctypes

import pytest

import tensor_transformer_mlp_tmem_gb300 as tp
from test_attention_memory_order import D, Hq, Context, context, lib  # noqa: F401


@pytest.fixture(autouse=True)
def signatures(lib):  # noqa: F811
    lib.tpmlp_attn_reserve.argtypes = [ctypes.c_void_p, ctypes.c_int64]


def values(lib, i):  # noqa: F811
    return (ctypes.c_uint32 * (lib.fake_block_bytes(i) // 4)).from_address(lib.fake_block(i))


def test_cleared_before_the_call_returns(lib, context):  # noqa: F811
    """Two blocks: partial sums with their counters at the end, and the results over both kinds of keys
    (fp32 [sequences][Hq][D], and 16 bytes a head)."""
    first = lib.fake_blocks()
    assert lib.tpmlp_attn_reserve(context.ctx, 3) == tp.TPMLP_OK
    assert lib.fake_blocks() == first + 2
    assert lib.fake_block_bytes(first + 1) == 2 * 3 * Hq * (D * 4 + 16)
    counters, results = values(lib, first), values(lib, first + 1)
    assert not any(counters[-600:]) and not any(results)
    counters[-1], results[0] = 7, 9  # a call on a side stream
    lib.fake_catch_up()
    assert counters[-1] == 7 and results[0] == 9


def test_doubles_and_keeps_what_it_had(lib, context):  # noqa: F811
    assert lib.tpmlp_attn_reserve(context.ctx, 3) == tp.TPMLP_OK
    first = lib.fake_blocks()
    values(lib, first - 1)[5] = 11  # a captured graph's call reads here
    assert lib.tpmlp_attn_reserve(context.ctx, 2) == tp.TPMLP_OK
    assert lib.tpmlp_attn_reserve(context.ctx, 3) == tp.TPMLP_OK
    assert lib.fake_blocks() == first  # room enough
    assert lib.tpmlp_attn_reserve(context.ctx, 4) == tp.TPMLP_OK
    assert lib.fake_blocks() == first + 1 and lib.fake_block_bytes(first) == 2 * 6 * Hq * (D * 4 + 16)
    lib.fake_catch_up()
    assert values(lib, first - 1)[5] == 11
    assert lib.tpmlp_attn_reserve(context.ctx, 6) == tp.TPMLP_OK and lib.fake_blocks() == first + 1


@pytest.mark.parametrize("which", range(2))
def test_without_memory(lib, context, which):  # noqa: F811
    """The call says so, and works once there is some."""
    lib.fake_fail_allocation(lib.fake_blocks() + which)
    assert lib.tpmlp_attn_reserve(context.ctx, 3) == tp.TPMLP_ERR_OOM
    assert lib.tpmlp_attn_reserve(context.ctx, 3) == tp.TPMLP_OK
