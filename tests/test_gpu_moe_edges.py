"""Expert routing on the GPU at the edges of what the header allows."""
import sys

import pytest
import torch

import int8_gemm_linear_amd as q

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-moe-edges]", *a, flush=True)
    sys.stdout.flush()


@pytest.mark.parametrize("tokens,gradients", [((1 << 26) + 5, True), ((1 << 28) + 5, False)])
def test_tokens_past_one_launch(tokens, gradients):
    # 256 threads serve four tokens of the gradient and sixteen of the others: past
    # 2^26 and 2^28 tokens that is more threads than a launch may have.  A row of one
    # value for each token, in reverse order; every eleventh token has none
    say("tokens", tokens, gradients)
    row = torch.arange(tokens - 1, -1, -1, dtype=torch.int32, device="cuda").view(-1, 1)
    absent = (row % 11 == 3)
    row[absent] = -1
    x = (torch.arange(tokens, dtype=torch.int32, device="cuda") % 251).to(torch.bfloat16).view(-1, 1)
    w = torch.full((tokens, 1), 2.0, device="cuda")
    back = x.flip(0)                                     # the row of token t holds x[tokens - 1 - t] of it
    if gradients:
        dy, dw = q.moe_combine_backward(x, x, row, w, dy=torch.zeros_like(x))
        torch.cuda.synchronize()
        assert torch.equal(dy, torch.where(absent, 0, 2 * x).flip(0))
        assert torch.equal(dw, torch.where(absent, 0.0, x.float() * back.float()))
        return
    scale = x.float().view(-1)
    out, out_scale = q.moe_permute(x, row, scale, out=torch.zeros_like(x), out_scale=torch.zeros_like(scale))
    torch.cuda.synchronize()
    want = torch.where(absent, 0, x).flip(0)
    assert torch.equal(out, want) and torch.equal(out_scale, want.float().view(-1))
    del out, out_scale, want, scale
    assert torch.equal(q.moe_combine(x, row, w), torch.where(absent, 0, 2 * back))
    assert torch.equal(q.moe_permute_backward(x, row), torch.where(absent, 0, back))
