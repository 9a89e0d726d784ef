"""The adapters' plan on the GPU: the offsets that the gradients of A and B sum by, the order of tokens, and that no
result depends on it; with up to 64 tokens, up to 8192, and more, which are planned in three ways."""
import pytest

from tests.test_gpu_lora import backward, check_backward, make

pytestmark = pytest.mark.gpu


# a workgroup of 512 threads writes adapters + 1 offsets: less than a wave, whole turns, ends inside a wave
@pytest.mark.parametrize("L", [1, 62, 63, 64, 510, 511, 512, 700, 1023, 2047])
@pytest.mark.parametrize("T", [1, 33, 64])
def test_offsets_of_many_adapters(T, L):
    d = make(T, 72, 40, 8, L, T + L, bits=64)
    d["ids"][T - 1] = L - 1
    check_backward(d, backward(d), what=str((T, L)))
