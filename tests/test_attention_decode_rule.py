"""Which kernel decode takes, by the head group's width, the head size and the cache's type."""
import ctypes

import tensor_transformer_mlp_tmem_gb300 as tp
from test_attention_host import hooks  # noqa: F401


def test_decode_takes_the_faster_kernel(hooks):  # noqa: F811
    """The widest group of the row kernel (its comment has both kernels' times)."""
    rule = hooks.tpmlp_test_decode_on_rows
    rule.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_uint32]
    for D, flags, widest in ((128, 0, 8), (128, tp.TPMLP_FLAG_KV_E4M3, 16), (64, 0, 16),
                             (64, tp.TPMLP_FLAG_KV_E4M3, 32)):
        assert [rule(G, D, flags) for G in (1, widest, widest + 1, 128)] == [1, 1, 0, 0], (D, flags)
