"""Outputs beside inputs in one buffer are taken, outputs over inputs refused before anything is written."""
import pytest
import torch

import int8_gemm_linear_amd as q
from tests.test_gpu_lora import DEV, backward, forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [30, 300])
def test_columns_of_one_buffer(T):
    d = make(T, 72, 40, 16, 3, T)
    want, back = forward(d), backward(d)
    wide = torch.full((T, 300), 5.0, dtype=torch.bfloat16, device=DEV)
    x, base, y, dx = wide[:, :72], wide[:, 72:112], wide[:, 112:152], wide[:, 152:224]
    x.copy_(d["x"])
    base.copy_(d["base"])
    q.lora_mm(x, d["a"], d["b"], d["ids"], scale=d["scale"], base=base, out=y)
    assert torch.equal(y, want) and torch.equal(x, d["x"]) and torch.equal(base, d["base"])
    y.copy_(d["dy"])
    got = q.lora_mm_backward(y, x, d["a"], d["b"], d["ids"], scale=d["scale"], base=d["dbase"], out=dx)
    assert all(torch.equal(g, w) for g, w in zip(got, back))
    assert (wide[:, 224:] == 5).all()
    with pytest.raises(q.QlinError):
        q.lora_mm(x, d["a"], d["b"], d["ids"], base=base, out=wide[:, 71:111])
    with pytest.raises(q.QlinError):
        q.lora_mm_backward(y, x, d["a"], d["b"], d["ids"], out=wide[:, 100:172])
    assert torch.equal(x, d["x"]) and torch.equal(base, d["base"]) and torch.equal(y, d["dy"])


def test_one_tokens_row():
    """A single row's stride says nothing: base and out are the same row."""
    d = make(1, 64, 48, 8, 2, 5)
    want = forward(d)
    wide = torch.zeros((2, 100), dtype=torch.bfloat16, device=DEV)
    wide[:1, :48] = d["base"]
    assert torch.equal(forward({**d, "base": wide[:1, :48]}, out=wide[0, :48].view(1, 48)), want)


def test_log_probabilities_and_embedding():
    logits = torch.randn((6, 90), device=DEV)
    target = torch.arange(6, device=DEV)
    one = torch.ones(6, device=DEV)
    lse = q.token_logprobs(logits, target)[2]
    want = q.token_logprobs_backward(one, logits, target, lse)
    wide = torch.zeros((6, 200), device=DEV)
    wide[:, :90] = logits
    got = q.token_logprobs_backward(one, wide[:, :90], target, lse, out=wide[:, 90:180])
    assert torch.equal(got, want) and torch.equal(wide[:, :90], logits)
    with pytest.raises(q.QlinError):
        q.token_logprobs_backward(one, wide[:, :90], target, lse, out=wide[:, 1:91])
    flat = torch.zeros(6 * 91, device=DEV)
    with pytest.raises(q.QlinError):
        q.token_logprobs_backward(one, flat[:540].view(6, 90), target, lse, out=flat[1:541].view(6, 90))
    table = torch.randn((8, 60), device=DEV)
    both = torch.zeros((8, 120), device=DEV)
    both[:, :60] = table
    ids = torch.arange(7, -1, -1, device=DEV)
    assert torch.equal(q.embedding(ids, both[:, :60], out=both[:, 60:]), table.flip(0))
    with pytest.raises(q.QlinError):
        q.embedding(ids, both[:, :60], out=both[:, 59:119])
    d = both[:, 60:]
    assert torch.equal(q.embedding_backward(d, ids, 8, out=both[:, :60]), table)
    with pytest.raises(q.QlinError):
        q.embedding_backward(d, ids, 8, out=both[:, 1:61])
