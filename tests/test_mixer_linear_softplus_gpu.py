"""The projection's softplus element by element, down to pre-activations where it is about e^x.

The inputs are 0, so the pre-activation is the bias, exactly.  The result is rounded to bf16 once (half a step, 2^-8
relative); the fp32 evaluation before it is held to 2^-16: the fast exponential (2^-22, and 2^-24 times an exponent below
2^5) and ten fp32 steps."""
import pytest
import torch

import mixer_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 100])  # the few-row kernel and the tiles
def test_softplus_is_relatively_exact(kda, M):
    N = 40000
    bias = torch.cat([torch.linspace(-12, -4, N // 2), torch.linspace(-30, 10, N // 2)])
    x, W = torch.zeros((M, 8), dtype=torch.bfloat16), torch.zeros((N, 8), dtype=torch.bfloat16)
    y = kda.linear_act(x.cuda(), W.cuda(), bias.cuda(), act="softplus").double().cpu()
    want = ref.softplus(bias.double())
    rel = ((y - want).abs() / want).max()
    assert rel <= 2.0 ** -8 + 2.0 ** -16, float(rel)
