"""The adapters' plan on the GPU: the offsets that the gradients of A and B sum by, the order of tokens, and that no
result depends on it; with up to 64 tokens, up to 8192, and more, which are planned in three ways."""
import pytest
import torch

from tests.test_gpu_lora import DEV, backward, check_backward, check_forward, forward, make

pytestmark = pytest.mark.gpu


# a workgroup of 512 threads writes adapters + 1 offsets: less than a wave, whole turns, ends inside a wave
@pytest.mark.parametrize("L", [1, 62, 63, 64, 510, 511, 512, 700, 1023, 2047])
@pytest.mark.parametrize("T", [1, 33, 64])
def test_offsets_of_many_adapters(T, L):
    d = make(T, 72, 40, 8, L, T + L, bits=64)
    d["ids"][T - 1] = L - 1
    check_backward(d, backward(d), what=str((T, L)))


def shuffled(d, p):
    """The same tokens in another order."""
    return {k: v[p] if k in ("x", "ids", "base", "dy", "dbase") else v for k, v in d.items()}


# each way of planning, with few and with many tokens an adapter, and K in parts and whole
@pytest.mark.parametrize("T,K,N,R,L", [(40, 384, 320, 16, 7), (64, 2048, 200, 32, 3), (64, 1100, 130, 64, 2),
                                       (500, 384, 320, 16, 7), (300, 1100, 264, 24, 40), (3000, 136, 200, 64, 3),
                                       (8193, 72, 136, 16, 9), (9000, 200, 72, 40, 700), (20000, 64, 130, 8, 2)])
def test_the_order_of_tokens_does_not_matter(T, K, N, R, L):
    """y and dx of a token are the same bits wherever it stands; dA and dB sum in the tokens' order."""
    d = make(T, K, N, R, L, T + K)
    y, back = forward(d), backward(d)
    check_forward(d, y)
    check_backward(d, back)
    g = torch.Generator().manual_seed(T)
    for _ in range(2):
        p = torch.randperm(T, generator=g).to(DEV)
        s = shuffled(d, p)
        assert torch.equal(forward(s), y[p])
        got = backward(s)
        assert torch.equal(got[0], back[0][p])
        check_backward(s, got)
    for _ in range(2):                                # and a call gives the same bits again
        assert torch.equal(forward(d), y)
        for a, b in zip(backward(d), back):
            assert torch.equal(a, b)
