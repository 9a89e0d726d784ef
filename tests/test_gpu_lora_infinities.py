"""Infinities and NaNs beside the adapters' tokens where an adapter has many: the second product that shares weights
between 64 tokens, and the gradients' sums by several waves and in parts."""
import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests.reference64 import f64
from tests.test_gpu_lora import DEV, backward, forward, make

pytestmark = pytest.mark.gpu
SIZES = [(300, 4), (200, 1), (1100, 2), (9000, 3)]


@pytest.mark.parametrize("R", [8, 24, 64])
@pytest.mark.parametrize("T,L", SIZES)
def test_infinities_and_nans_stay_with_their_tokens(T, L, R):
    d = make(T, 160, 130, R, L, T + R)
    ids = d["ids"]
    ids[:7] = torch.tensor([0, 0, 1 % L, 1 % L, 2 % L, L - 1, -1], dtype=torch.int32)
    clean, cleaned = forward(d), backward(d)
    d["x"][0, 5], d["x"][2, 7] = float("nan"), float("inf")
    d["x"][6] = float("nan")                         # no adapter: never read
    y = forward(d)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[[0, 2]] = False
    assert torch.equal(y[keep], clean[keep]) and y[0].isnan().all() and not y[2].isfinite().any()
    d["dy"][1, 3] = float("nan")
    d["dy"][6] = float("nan")
    dx, da, db = backward(d)
    assert dx[1].isnan().all()
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[1] = False
    assert torch.equal(dx[keep], cleaned[0][keep])
    assert da[0].isnan().any() and db[0].isnan().any()
    for i in range(2, L):
        assert torch.equal(da[i], cleaned[1][i]) and torch.equal(db[i], cleaned[2][i])


@pytest.mark.parametrize("R", [8, 24, 64])
@pytest.mark.parametrize("T", [200, 700, 9000])
def test_an_adapter_that_no_token_has_is_not_read(T, R):
    d = make(T, 160, 130, R, 3, T + R + 1, [0, 2, -1])
    y, back = forward(d), backward(d)
    d["a"][1], d["b"][1], d["scale"][1] = float("nan"), float("inf"), float("nan")
    assert torch.equal(forward(d), y)
    for g, w in zip(backward(d), back):
        assert torch.equal(g, w)


@pytest.mark.parametrize("R", [8, 24, 64])
@pytest.mark.parametrize("T", [90, 200, 9000])
def test_infinity_of_one_row_of_b(T, R):
    """An infinity in b reaches its output column with its sign, and no other."""
    d = make(T, 64, 70, R, 1, T + R + 2, [0])
    y = forward(d)
    d["b"][0, 33, 2] = float("inf")
    got = forward(d)
    keep = torch.ones(70, dtype=torch.bool, device=DEV)
    keep[33] = False
    assert torch.equal(got[:, keep], y[:, keep])
    v = f64(d["x"]) @ f64(d["a"])[0, 2]
    assert np.array_equal(f64(got[:, 33]), np.sign(v) * np.inf)


@pytest.mark.parametrize("R", [8, 16, 40, 128])
@pytest.mark.parametrize("T", [90, 300, 1100, 9000])
def test_infinities_beside_short_values(T, R):
    """v and u of few bits leave nothing for their lower pieces: an infinity that meets them stays one."""
    K, N = 24, 40
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1.0
    a = torch.zeros((1, R, K), dtype=torch.bfloat16, device=DEV)
    a[0, 0, 0] = 0.5
    b = torch.zeros((1, N, R), dtype=torch.bfloat16, device=DEV)
    b[0, :, 0] = 1.0
    ids = torch.zeros(T, dtype=torch.int64, device=DEV)
    b[0, 7, 0] = float("inf")
    y = q.lora_mm(x, a, b, ids)
    assert (y[:, 7] == float("inf")).all() and (y[:, :7] == 0.5).all() and (y[:, 8:] == 0.5).all()
    b[0, 7, 0] = 1.0
    dy = torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
    dy[:, 3] = 2.0
    dy[4, 9] = float("-inf")
    x[5, 11] = float("inf")
    a[0, 0, 11] = 1.0
    dx, da, db = q.lora_mm_backward(dy, x, a, b, ids)
    # token 4: u = -inf at rank 0, and NaN (-inf times b's 0) at the others; token 5: v = inf, u = 2
    assert da[0, 0, 0] == float("-inf") and da[0, 0, 11].isnan() and dx[0, 0] == 1.0 and dx[4, 0].isnan()
    assert db[0, 3, 0] == float("inf") and db[0, 9, 0].isnan() and db[0, 20, 0].isnan()
    x[5, 11], dy[4, 9], x[6, 1] = 0.0, 0.0, float("inf")
    a[0, 0, 11] = float("inf")
    dx, da, db = q.lora_mm_backward(dy, x, a, b, ids)
    assert da[0, 0, 1] == float("inf") and da[0, 0, 0] == 2.0 * T
    assert (dx[:, 11] == float("inf")).all() and (dx[:, 0] == 1.0).all() and not dx[:, 1:11].any()


@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("low", [-85, -60, -30, 0])
def test_infinities_beside_small_values(T, low):
    """Down to 2^-86 the stand-in for an empty piece is a bf16 number."""
    x = torch.zeros((T, 16), dtype=torch.bfloat16, device=DEV)
    x[:, 3] = 2.0 ** low
    a = torch.zeros((1, 8, 16), dtype=torch.bfloat16, device=DEV)
    a[0, 1, 3] = 1.0
    b = torch.zeros((1, 40, 8), dtype=torch.bfloat16, device=DEV)
    b[0, :, 1] = 1.0
    b[0, 5, 1], b[0, 6, 1] = float("inf"), float("-inf")
    y = q.lora_mm(x, a, b, torch.zeros(T, dtype=torch.int32, device=DEV))
    assert (y[:, 5] == float("inf")).all() and (y[:, 6] == float("-inf")).all()
    keep = torch.ones(40, dtype=torch.bool, device=DEV)
    keep[[5, 6]] = False
    assert (y[:, keep] == 2.0 ** low).all()
