"""What the attention tests' tolerance tells apart (no GPU needed): a result that leaves a key out is not
within it."""
import pytest
import torch

import attention_ref as ref


def within(got, o, spread, kv):
    return bool(((got - o).abs() <= ref.out_tolerance(o, spread, kv)).all())


def rejects_a_missing_key(c, b, q, n, scale):
    """Whether the definition over n keys of sequence b turns away the one over n - 1 of them."""
    o, _, spread, _ = ref.attend(c, b, q, n, 0, scale)
    less = ref.attend(c, b, q, n - 1, 0, scale)[0]
    return within(o, o, spread, c["kv"]) and not within(less, o, spread, c["kv"])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 17, 100, 384, 640])
def test_a_missing_key_is_noticed(kv, D, n):
    c = ref.make(2, D, 32, kv, [n], seed=n + D)
    q = torch.randn((8, D), generator=torch.Generator().manual_seed(n)).bfloat16().double()
    assert rejects_a_missing_key(c, 0, q, n, D ** -0.5)
