"""How the log probabilities add up long rows, on the GPU against the definition."""
import math

import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests.reference64 import close, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,V", [(1, 131072), (100, 65536), (641, 65536), (700, 50001)])
def test_many_small_terms_beside_a_large_one(T, V, dtype):
    """A logit of 0 among others of -16.75, whose exponentials, 0.89 * 2^-24, are each lost beside a sum of 1.

    A lane adds at most 32 logits before their sum joins its others, one for each of V / 4096 + 1 turns at most; then
    come 6 sums over lanes, 3 over waves and 63 over parts, 73 in all.  Each is off by half a step, 2^-24, of at most
    S; the terms e^d by (|d| + 2) 2^-23 relatively, ln S by 2^-22 relatively, and a step for each of the last three
    operations."""
    small = -16.75
    x = torch.full((T, V), small, dtype=dtype, device=DEV)
    at = (torch.arange(T, device=DEV) * 4999) % V                     # the first turn, later ones, the last
    x.scatter_(1, at.unsqueeze(1), 0.0)
    logprob, entropy, lse, _, _ = q.token_logprobs(x, at)
    e = math.exp(small)
    S, W = 1.0 + (V - 1) * e, (V - 1) * e * small
    want = math.log1p((V - 1) * e)
    n = 32 + V // 4096 + 1 + 73
    tol = 2.0 ** -24 * n + (S - 1) * (abs(small) + 2) * 2.0 ** -23 + 2.0 ** -22 * want + 3 * 2.0 ** -24 * want
    one = np.ones(T)
    close(f64(lse), want * one, tol * one, "lse")
    close(f64(logprob), -want * one, tol * one, "logprob")
    # W is summed as S is, of terms that are off by one product more; then W / S and a difference
    D = -W / S
    more = D * (2 * 2.0 ** -24 * n + (2 * abs(small) + 5) * 2.0 ** -23 + 2 * 2.0 ** -24) + 2.0 ** -24 * (want + D)
    close(f64(entropy), (want + D) * one, (tol + more) * one, "entropy")
