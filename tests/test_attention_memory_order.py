"""Order of an attention context's own memory operations against the caller's streams, on a fake of
the CUDA runtime (fake_cuda.h): what the library clears or fills on its own account is done before
the call returns, so it can neither meet the work of a stream that does not wait for the default
stream nor overwrite what that work has written."""
import ctypes
import os

import pytest

import tensor_transformer_mlp_tmem_gb300 as tp
from tensor_transformer_mlp_tmem_gb300 import _build

FAKE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "fake_cuda.h")
Hq, Hkv, D, PAGE = 8, 2, 128, 64
SIDE = 4096  # a stream that does not block on the default one
BAD_PAGE_BIT = 0x10000


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    path = _build.build(out=str(tmp_path_factory.mktemp("fake") / "libtpmlp_fake.so"),
                        extra_flags=["-include", FAKE, "-DTPMLP_TEST_HOOKS"])
    h = ctypes.CDLL(path)
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    h.tpmlp_attn_create.argtypes = [ctypes.POINTER(vp), i32, i32, i32, i32, ctypes.c_uint32]
    h.tpmlp_get_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
    h.tpmlp_destroy.argtypes = [vp]
    h.fake_block.restype = vp
    h.fake_block_bytes.restype = ctypes.c_int64
    return h


class Context:
    """An attention context whose blocks the test reads and writes as a kernel would."""

    def __init__(self, lib, flags=0):
        first = lib.fake_blocks()
        self.ctx = ctypes.c_void_p()
        assert lib.tpmlp_attn_create(ctypes.byref(self.ctx), Hq, Hkv, D, PAGE, flags) == tp.TPMLP_OK
        at = [(lib.fake_block(i), lib.fake_block_bytes(i)) for i in range(first, lib.fake_blocks())]
        (scales, _), (_, _), (count, bytes_), (status, words) = at
        self.scales = (ctypes.c_float * (2 * Hkv)).from_address(scales)
        self.count = (ctypes.c_uint32 * (bytes_ // 4)).from_address(count)
        self.word = (ctypes.c_int32 * (words // 4)).from_address(status)


@pytest.fixture
def context(lib):
    c = Context(lib)
    lib.fake_catch_up()
    yield c
    lib.tpmlp_destroy(c.ctx)


def status(lib, c, stream=SIDE):
    detail = ctypes.c_int32(-1)
    return lib.tpmlp_get_status(c.ctx, stream, ctypes.byref(detail)), detail.value


def test_a_bad_page_does_not_hide_a_wait_that_ran_out(lib, context):
    """Both kinds of report stand beside each other, and the one that leaves outputs unwritten is
    answered first."""
    assert status(lib, context) == (tp.TPMLP_OK, 0)
    lib.fake_catch_up()
    context.word[1] = 1
    assert status(lib, context) == (tp.TPMLP_ERR_BAD_PAGE, BAD_PAGE_BIT)
    lib.fake_catch_up()
    context.word[0], context.word[1] = 0x2005, 1
    assert status(lib, context) == (tp.TPMLP_ERR_DEVICE_TIMEOUT, BAD_PAGE_BIT | 0x2005)
    lib.fake_catch_up()
    context.word[0] = 0x2005
    assert status(lib, context) == (tp.TPMLP_ERR_DEVICE_TIMEOUT, 0x2005)
    lib.fake_catch_up()
    assert status(lib, context) == (tp.TPMLP_OK, 0)


def test_status_is_cleared_before_the_next_call(lib, context):
    """What a call enqueued on a side stream right after reports and counts stays; what the call that
    gave up left at its joins is gone."""
    context.word[0], context.count[7] = 0x2005, 3
    assert status(lib, context) == (tp.TPMLP_ERR_DEVICE_TIMEOUT, 0x2005)
    assert context.word[0] == 0 and context.count[7] == 0
    context.word[0], context.count[9] = 0x2003, 2  # the next call's kernel
    lib.fake_catch_up()
    assert context.word[0] == 0x2003 and context.count[9] == 2


@pytest.mark.parametrize("bad_page", [0, 1])
def test_arrivals_of_a_call_that_runs_are_left_alone(lib, context, bad_page):
    """Without a wait that ran out nothing is left behind, and the arrivals may be those of a call on
    another stream."""
    context.word[1], context.count[5] = bad_page, 2
    assert status(lib, context)[0] == (tp.TPMLP_ERR_BAD_PAGE if bad_page else tp.TPMLP_OK)
    lib.fake_catch_up()
    assert context.count[5] == 2 and context.word[1] == 0


@pytest.mark.parametrize("flags", [0, tp.TPMLP_FLAG_KV_E4M3])
def test_a_new_context_is_ready_for_every_stream(lib, flags):
    """What the first calls on a side stream set and count stays: nothing of the context's own set-up
    is still to run."""
    c = Context(lib, flags)
    assert list(c.scales) == [1.0] * (2 * Hkv) and not any(c.count) and not any(c.word)
    c.scales[1], c.count[3], c.word[0], c.word[1] = 0.5, 1, 0x2001, 1
    lib.fake_catch_up()
    assert (c.scales[1], c.count[3], c.word[0], c.word[1]) == (0.5, 1, 0x2001, 1)
    lib.tpmlp_destroy(c.ctx)


@pytest.mark.parametrize("which", range(4))
def test_a_context_that_finds_no_memory_is_refused(lib, which):
    lib.fake_fail_allocation(lib.fake_blocks() + which)
    out = ctypes.c_void_p()
    assert lib.tpmlp_attn_create(ctypes.byref(out), Hq, Hkv, D, PAGE, 0) == tp.TPMLP_ERR_OOM
    assert out.value is None
    lib.fake_catch_up()


def test_a_new_block_context_is_ready_for_every_stream(lib):
    """The same of a block's context: its status and the counters of its split tiles."""
    lib.tpmlp_create.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                 ctypes.c_uint32]
    first, ctx = lib.fake_blocks(), ctypes.c_void_p()
    assert lib.tpmlp_create(ctypes.byref(ctx), 256, 1024, 2, 0) == tp.TPMLP_OK
    blocks = range(first, lib.fake_blocks())
    status_words, counters = [  # 8 bytes, and 152 tiles x 2 CTAs x a counter per epilogue warp
        next((ctypes.c_int32 * (n // 4)).from_address(lib.fake_block(i))
             for i in blocks for n in [lib.fake_block_bytes(i)] if wanted(n))
        for wanted in (lambda n: n == 8, lambda n: n % (152 * 2 * 4) == 0 and 1 <= n // (152 * 2 * 4) <= 16)]
    assert not any(status_words) and not any(counters)
    status_words[0], counters[5] = 0x101, 7
    lib.fake_catch_up()
    assert status_words[0] == 0x101 and counters[5] == 7
    lib.tpmlp_destroy(ctx)


def test_the_backward_pass_has_its_zeros_on_every_stream(lib):
    """The zeros that a backward pass makes on its first call hold before anything is enqueued (the
    call itself ends at its first tensor map: there is no driver here)."""
    lib.tpmlp_test_host_context.restype = ctypes.c_void_p
    lib.tpmlp_test_set_current_device(0)
    ctx = ctypes.c_void_p(lib.tpmlp_test_host_context(ctypes.c_int64(256), ctypes.c_int64(1024), 2, 0, 0, 1, 0))
    first, at = lib.fake_blocks(), ctypes.c_void_p(1 << 20)
    i64 = ctypes.c_int64
    assert lib.tpmlp_backward(ctx, at, at, at, at, at, at, i64(1), i64(64), at, at, at, at, at,
                              ctypes.c_void_p(SIDE)) != tp.TPMLP_OK
    zeros = [i for i in range(first, lib.fake_blocks()) if lib.fake_block_bytes(i) == 4 * 1024]
    assert len(zeros) == 1 and not any((ctypes.c_uint32 * 1024).from_address(lib.fake_block(zeros[0])))
    lib.tpmlp_test_set_current_device(-1)
    lib.tpmlp_destroy(ctx)
