"""Log probabilities over logits at the edges of their kernels. Bounds count roundings as in
head_ops_testlib, u = 2^-24."""
import math

import numpy as np
import pytest

from head_ops_testlib import U, check_logprobs, sum_eps
from oracle import head_ops as ho

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _rng(seed):
    return np.random.Generator(np.random.Philox(np.random.SeedSequence([seed, 67])))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
def test_gradient_at_a_token_with_the_types_lowest_logit(dtype, T):
    """p is 0 there and 1 - p is 1, whether its log probability still is a number or, at
    temperatures below 1, -inf. At a logit of -inf there is no gradient."""
    lowest = torch.finfo(TYPES[dtype]).min
    z = torch.zeros(3, 40, dtype=TYPES[dtype], device=DEV)
    z[0, 7] = lowest
    z[1, 7] = -math.inf
    z[2, 7] = -1000.0
    y = torch.full((3,), 7, dtype=torch.int32, device=DEV)
    r = flce.token_logprobs(z, y, temperature=T)
    a = torch.tensor([0.75, 0.75, 0.75], device=DEV)
    g = flce.token_logprobs_backward(z, y, r, dlogprob=a, dentropy=a, dlse=a, temperature=T)
    want = torch.tensor([0.75 / T, 0.0, 0.75 / T], device=DEV)
    assert float((g[:, 7].float() - want).abs().max()) <= 4 * U   # 0.75 / T is a number of each type
