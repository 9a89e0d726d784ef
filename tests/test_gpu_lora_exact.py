"""Low-rank adapters on values whose sums are exact in fp32, bit for bit: what X A^T
and dY B hold reaches every output whole.

v takes values a0 + a1 2^-8 + a2 2^-16 with three runs of eight bits, which no fewer
than three bf16 numbers hold; ranks that cancel leave the last run alone."""
import pytest
import torch

import int8_gemm_linear_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def digits(shape, g):
    """Numbers 1 + i / 128: eight bits with the first one set."""
    return 1.0 + torch.randint(0, 128, shape, generator=g) / 128.0


# tokens, width, rank, adapters: one launch, few and many tokens an adapter, the first product's sums in parts and whole
FORMS = [(1, 64, 8, 1), (3, 300, 16, 2), (40, 130, 32, 3), (20, 200, 40, 1), (64, 5000, 16, 2), (90, 640, 24, 4),
         (100, 700, 128, 2), (300, 600, 8, 2), (300, 1100, 16, 1), (520, 130, 64, 2), (2000, 136, 48, 3),
         (9000, 72, 16, 3), (2200, 4104, 32, 30)]


def chain(T, K, R, L, seed):
    """x [T,K] and a [L,R,K] whose product, exact in fp32, is v [T,L,R]: whole numbers of 2^-23 below 2."""
    g = torch.Generator().manual_seed(seed)
    x = torch.zeros((T, K))
    a = torch.zeros((L, R, K))
    at = torch.randperm(K, generator=g)[:3]
    x[:, at] = torch.tensor([1.0, 2.0 ** -8, 2.0 ** -16])
    x[torch.rand(T, generator=g) < 0.5] *= -1.0
    a[:, :, at] = digits((L, R, 3), g)
    a[:, 1::2] = a[:, 0::2]                          # ranks in pairs, equal but for the last run of bits
    a[:, 1::2, at[2]] = 0.0
    v = torch.einsum("tk,lrk->tlr", x.double(), a.double())
    return x, a, v


def inputs(T, K, R, L, seed):
    x, a, v = chain(T, K, R, L, seed)
    g = torch.Generator().manual_seed(seed + 1)
    ids = torch.randint(-1, L, (T,), generator=g)
    N = K + 3
    # a column takes a pair's difference, times a power of two
    pair = torch.randint(0, R // 2, (L, N), generator=g)
    f = torch.tensor([0.5, 1.0, -2.0])[torch.randint(0, 3, (L, N), generator=g)]
    b = torch.zeros((L, N, R))
    b.scatter_(2, 2 * pair.unsqueeze(2), f.unsqueeze(2))
    b.scatter_(2, 2 * pair.unsqueeze(2) + 1, -f.unsqueeze(2))
    scale = torch.tensor([0.5, 2.0, 1.0])[torch.randint(0, 3, (L,), generator=g)]
    return x, a, b, ids, scale, v


def dev(t):
    return t.to(torch.bfloat16).contiguous().to(DEV)


@pytest.mark.parametrize("T,K,R,L", FORMS)
def test_forward_takes_the_first_product_whole(T, K, R, L):
    x, a, b, ids, scale, v = inputs(T, K, R, L, T + K + R)
    y = q.lora_mm(dev(x), dev(a), dev(b), ids.to(DEV), scale=scale.to(DEV))
    at = ids.clamp(min=0)
    own = v[torch.arange(T), at] * scale[at].unsqueeze(1) * (ids >= 0).unsqueeze(1)
    want = torch.zeros((T, b.shape[1]), dtype=torch.float64)
    for i in range(L):
        want[ids == i] = own[ids == i] @ b[i].double().t()
    assert torch.equal(y.cpu().double(), want)


@pytest.mark.parametrize("T,K,R,L", FORMS)
def test_gradients_take_both_products_whole(T, K, R, L):
    # dy takes x's part: u = dy b with b the first product's factor, and dx = u a
    dy, bt, u = chain(T, K, R, L, T + K + R + 5)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, L, (T,), generator=g)
    W = K + 5
    pair = torch.randint(0, R // 2, (L, W), generator=g)
    a = torch.zeros((L, W, R))
    a.scatter_(2, 2 * pair.unsqueeze(2), 1.0)
    a.scatter_(2, 2 * pair.unsqueeze(2) + 1, -1.0)
    a = a.transpose(1, 2)
    # one token of each adapter has an x, so that dA is its u times powers of two
    x = torch.zeros((T, W))
    some = {}
    for i in range(L):
        t = torch.nonzero(ids == i).flatten()
        if t.numel():
            some[i] = int(t[int(torch.randint(0, t.numel(), (1,), generator=g))])
            x[some[i]] = torch.tensor([0.5, 1.0, -4.0])[torch.randint(0, 3, (W,), generator=g)]
    dx, da, _ = q.lora_mm_backward(dev(dy), dev(x), dev(a), dev(bt.transpose(1, 2)), ids.to(DEV))
    own = u[torch.arange(T), ids.clamp(min=0)] * (ids >= 0).unsqueeze(1)
    want, wa = torch.zeros((T, W), dtype=torch.float64), torch.zeros((L, R, W), dtype=torch.float64)
    for i in range(L):
        want[ids == i] = own[ids == i] @ a[i].double()
        if i in some:
            wa[i] = own[some[i]].unsqueeze(1) * x[some[i]].double()
    assert torch.equal(dx.cpu().double(), want)
    assert torch.equal(da.cpu().double(), wa)


@pytest.mark.parametrize("T,K,R,L", FORMS)
def test_gradient_of_b_takes_the_first_product_whole(T, K, R, L):
    x, a, b, ids, scale, v = inputs(T, K, R, L, T + K + R + 9)
    g = torch.Generator().manual_seed(T)
    dy = torch.zeros((T, b.shape[1]))
    want = torch.zeros(b.shape, dtype=torch.float64)
    for i in range(L):
        t = torch.nonzero(ids == i).flatten()
        if t.numel():
            t = int(t[int(torch.randint(0, t.numel(), (1,), generator=g))])
            dy[t] = torch.tensor([0.5, 1.0, -4.0])[torch.randint(0, 3, (b.shape[1],), generator=g)]
            want[i] = dy[t].double().unsqueeze(1) * v[t, i] * scale[i]
    _, _, db = q.lora_mm_backward(dev(dy), dev(x), dev(a), dev(b), ids.to(DEV), scale=scale.to(DEV))
    assert torch.equal(db.cpu().double(), want)
