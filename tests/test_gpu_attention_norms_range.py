"""Head norms where a head's size and its weights lie far apart."""
import pytest
import torch

from test_gpu_attention_norms import check, normed, one_token, slack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size,weight,eps", [
    (3e38, -16, 1e-6), (3e38, -20, 1e-6), (1e37, -30, 1e-6), (1e30, -40, 1e-6),  # large heads, small weights
    (1e-20, 120, 2.0 ** -40), (0.0, 120, 2.0 ** -40), (1e-3, 100, 1e-6),         # small heads, large weights
    (1.0, -100, 1.0), (3e38, 100, 1e-6),
])
def test_weights_far_from_the_heads(lib, D, size, weight, eps):
    """x over its root mean square is an ordinary number, whatever x; only then come the weights. The
    root's reciprocal may be subnormal (2^-128, half a step 2^-150: 2^-22 of it, inside the slack)."""
    g = torch.Generator().manual_seed(weight + 200)
    x = (torch.randn(D, generator=g).clamp(-1, 1) * size).bfloat16()
    w = ((1 + torch.rand(D, generator=g)) * 2.0 ** weight).bfloat16()
    want = normed(x.double(), w.double(), torch.tensor(eps, dtype=torch.float32).double())
    check(one_token(x, w, eps=eps), want, 2.0 ** -8, slack(want) + 2.0 ** -126)
