"""How exact the log probabilities are, on the GPU against the definition: sums of long rows, rows far from zero."""
import math

import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests import reference_ops as ref
from tests.reference64 import HALF, close, f64

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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0.0, -800.0, 1e4, -3e4])
def test_gradient_of_rows_far_from_zero(shift, dtype):
    """Against lse and entropy of 64 bits.  The kernels' lse is off by its own bound and half a step, |lse| 2^-24; p by
    as much relatively, and ln p + H by that and the entropy's error beside it."""
    T, V = 20, 3001
    g = torch.Generator().manual_seed(int(abs(shift)) + 1)
    x = (2.5 * torch.randn((T, V), generator=g) + shift).to(dtype)
    target = torch.randint(-1, V, (T,), generator=g)
    dl, dh = torch.randn(T, generator=g), 0.3 * torch.randn(T, generator=g)
    dev = x.to(DEV), target.to(DEV)
    _, entropy, lse, _, _ = q.token_logprobs(*dev)
    got = q.token_logprobs_backward(dl.to(DEV), *dev, lse, entropy=entropy, dentropy=dh.to(DEV))
    _, entropy, lse, _, top = ref.logprobs(f64(x), target.numpy(), 1)
    want, tol = ref.logprobs_backward(f64(dl), f64(x), target.numpy(), lse, entropy, f64(dh))
    _, de, dlse, _ = (b[:, None] if b.ndim == 1 else b for b in ref.logprobs_bounds(f64(x), target.numpy(), top))
    dlse = dlse + 2.0 ** -24 * np.abs(lse[:, None])
    z = f64(x) - lse[:, None]
    p = np.exp(z)
    h = np.abs(f64(dh))[:, None]
    there = ((target.numpy() >= 0) * np.abs(f64(dl)))[:, None]
    # p (g + h (z + H)): p's error times the bracket, and p times the bracket's (1.01: products of errors)
    tol = tol + 1.01 * p * (dlse * (there + h * np.abs(z + entropy[:, None])) + h * (dlse + de))
    close(f64(got), want, ref.rounded(want, tol, HALF[dtype]), f"{shift}")
