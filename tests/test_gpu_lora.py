"""Low-rank adapters on the GPU against the 64-bit reference: shapes that no tile
divides, ranks of every kind, ids in any order, empty adapters, strides, infinities
and NaNs beside the tokens they belong to, streams and graphs."""
import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests import reference_ops as ref
from tests.reference64 import close, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(T, K, N, R, L, seed, spread=None, bits=32):
    """Inputs; `spread`: None, every adapter alike; "runs", in order; a list, the adapters in use (-1: none)."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)
    x, dy = n(T, K).to(torch.bfloat16), n(T, N).to(torch.bfloat16)
    a, b = (n(L, R, K) / K ** 0.5).to(torch.bfloat16), (n(L, N, R) * 0.2).to(torch.bfloat16)
    if isinstance(spread, list):
        ids = torch.tensor(spread)[torch.randint(0, len(spread), (T,), generator=g)]
    else:
        ids = torch.randint(-1, L, (T,), generator=g)
        if spread == "runs":
            ids = ids.sort().values
    scale = 0.5 + torch.rand(L, generator=g)
    d = dict(x=x, a=a, b=b, ids=ids.to(torch.int64 if bits == 64 else torch.int32), scale=scale,
             base=n(T, N).to(torch.bfloat16), dy=dy, dbase=n(T, K).to(torch.bfloat16))
    return {k: v.to(DEV) for k, v in d.items()}


def check_forward(d, y, scale=True, base=True, what=""):
    want, tol = ref.lora(f64(d["x"]), f64(d["a"]), f64(d["b"]), d["ids"].cpu().numpy(),
                         f64(d["scale"]) if scale else None, f64(d["base"]) if base else np.zeros(d["base"].shape))
    assert y.dtype == torch.bfloat16
    close(f64(y), want, ref.rounded(want, tol), what)


def check_backward(d, got, scale=True, base=True, what=""):
    want, tol = ref.lora_backward(f64(d["dy"]), f64(d["x"]), f64(d["a"]), f64(d["b"]), d["ids"].cpu().numpy(),
                                  f64(d["scale"]) if scale else None,
                                  f64(d["dbase"]) if base else np.zeros(d["dbase"].shape))
    assert [g.dtype for g in got] == [torch.bfloat16, torch.float32, torch.float32]
    close(f64(got[0]), want[0], ref.rounded(want[0], tol[0]), what + " dx")
    close(f64(got[1]), want[1], tol[1] + ref.F32_MIN, what + " da")
    close(f64(got[2]), want[2], tol[2] + ref.F32_MIN, what + " db")


def forward(d, **kw):
    return q.lora_mm(d["x"], d["a"], d["b"], d["ids"], scale=d["scale"], base=d["base"], **kw)


def backward(d, **kw):
    return q.lora_mm_backward(d["dy"], d["x"], d["a"], d["b"], d["ids"], scale=d["scale"], base=d["dbase"], **kw)


# tokens, K, N, rank, adapters, ids' order, bits
SHAPES = [
    (1, 64, 64, 8, 1, [0], 32), (1, 2048, 2048, 16, 8, None, 32), (1, 1, 1, 8, 1, [0], 64), (2, 3, 5, 16, 2, None, 32),
    (5, 127, 63, 24, 3, None, 64), (7, 128, 64, 32, 5, None, 32), (16, 129, 65, 40, 2, None, 32),
    (17, 511, 257, 64, 4, None, 32), (33, 513, 130, 72, 3, "runs", 32), (31, 640, 1001, 96, 2, None, 64),
    (64, 1032, 77, 128, 3, "runs", 32), (65, 136, 4104, 8, 40, None, 32), (100, 5120, 48, 16, 2047, None, 64),
    (333, 1032, 1001, 8, 3, None, 32), (257, 255, 300, 16, 1, [0], 32), (300, 256, 511, 32, 2, "runs", 64),
    (130, 384, 640, 64, 1, [0], 32), (1100, 200, 136, 16, 5, "runs", 32), (1500, 72, 264, 32, 300, None, 32),
    (2100, 520, 130, 8, 2, [0, -1], 32), (4001, 96, 120, 48, 6, "runs", 64), (600, 64, 200, 128, 3, None, 32),
    (7700, 72, 40, 16, 2, "runs", 32), (8193, 40, 72, 40, 9, None, 64), (16000, 40, 72, 24, 3, None, 32),
    (15500, 66, 48, 64, 1, [0], 32), (20000, 24, 16, 8, 2000, None, 32), (9001, 24, 16, 8, 2047, None, 64),
    # few tokens and small adapters, and just beyond what one launch takes
    (1, 4096, 512, 16, 3, [2], 32), (1, 4104, 513, 16, 3, [-1], 64), (3, 2048, 1001, 32, 2, [1, -1, 0], 32),
    (64, 300, 700, 8, 70, None, 32), (63, 520, 1500, 24, 3, None, 64), (16, 65, 9000, 16, 12, None, 32),
    (20, 1000, 40, 40, 5, None, 32), (64, 200, 2600, 32, 60, None, 64),
    # many tokens an adapter: both sides of the rules on their number, K whole and in parts
    (63, 600, 72, 16, 1, [0], 32), (64, 600, 72, 16, 1, [0], 64), (65, 600, 72, 16, 2, None, 64), (95, 600, 136, 40, 3, None, 32),
    (200, 1100, 130, 96, 2, None, 32),
    (300, 2000, 264, 32, 1, [0, -1], 32), (511, 4100, 1001, 64, 4, "runs", 32), (1000, 2056, 72, 128, 7, None, 32),
    (520, 70, 200, 40, 8, None, 32), (8000, 40, 136, 16, 100, None, 32), (8192, 40, 72, 8, 128, "runs", 64),
    (12000, 24, 264, 8, 150, None, 32), (9000, 40, 130, 24, 70, "runs", 32), (7700, 264, 136, 128, 2, "runs", 32),
    (2100, 1100, 600, 24, 2, None, 32), (3000, 2600, 520, 72, 40, None, 64), (9000, 640, 1300, 16, 3, "runs", 32),
    (2049, 520, 4100, 40, 1, [0, -1], 32),
]


@pytest.mark.parametrize("T,K,N,R,L,spread,bits", SHAPES)
def test_forward(T, K, N, R, L, spread, bits):
    d = make(T, K, N, R, L, T + K + N + R, spread, bits)
    check_forward(d, forward(d), what=str((T, K, N, R, L)))


@pytest.mark.parametrize("T,K,N,R,L,spread,bits", SHAPES)
def test_backward(T, K, N, R, L, spread, bits):
    d = make(T, K, N, R, L, T + K + N + R + 1, spread, bits)
    check_backward(d, backward(d), what=str((T, K, N, R, L)))


@pytest.mark.parametrize("R", [8, 16, 24, 64])
def test_without_scale_and_base(R):
    d = make(40, 200, 136, R, 3, R)
    y = q.lora_mm(d["x"], d["a"], d["b"], d["ids"])
    check_forward(d, y, scale=False, base=False)
    assert not y[d["ids"] < 0].any()
    got = q.lora_mm_backward(d["dy"], d["x"], d["a"], d["b"], d["ids"])
    check_backward(d, got, scale=False, base=False)


def test_tokens_without_an_adapter_and_adapters_without_tokens():
    d = make(50, 128, 96, 16, 4, 11, [1, -1, 7])
    y, (dx, da, db) = forward(d), backward(d)
    check_forward(d, y)
    check_backward(d, (dx, da, db))
    none = d["ids"] != 1
    assert torch.equal(y[none], d["base"][none]) and torch.equal(dx[none], d["dbase"][none])
    for i in (0, 2, 3):
        assert not da[i].any() and not db[i].any()
    d["ids"].fill_(-1)
    y, (dx, da, db) = forward(d), backward(d)
    assert torch.equal(y, d["base"]) and torch.equal(dx, d["dbase"]) and not da.any() and not db.any()


@pytest.mark.parametrize("T", [30, 70, 700])       # one launch, and both forms of the second product
def test_in_place_and_strides(T):
    d = make(T, 200, 150, 16, 3, 12)
    want, back = forward(d), backward(d)
    wide = {k: torch.full((v.shape[0], v.shape[1] + 13), 7.0, dtype=v.dtype, device=DEV) for k, v in d.items()
            if v.dim() == 2}
    for k, w in wide.items():
        w[:, :d[k].shape[1]] = d[k]
    s = {**d, **{k: w[:, :d[k].shape[1]] for k, w in wide.items()}}
    out = torch.full((T, 200), 3.0, dtype=torch.bfloat16, device=DEV)
    forward(s, out=out[:, 17:167])
    assert torch.equal(out[:, 17:167], want) and (out[:, :17] == 3).all() and (out[:, 167:] == 3).all()
    assert torch.equal(forward(s, out=s["base"]), want) and torch.equal(s["base"], want)
    assert (wide["base"][:, 150:] == 7).all()
    for g, w in zip(backward(s, out=s["dbase"]), back):
        assert torch.equal(g, w)
    assert torch.equal(s["dbase"], back[0]) and (wide["dbase"][:, 200:] == 7).all()


@pytest.mark.parametrize("T", [40, 500])
def test_order_of_tokens_and_calls_do_not_matter(T):
    d = make(T, 384, 320, 16, 7, 13)
    y, back = forward(d), backward(d)
    for _ in range(3):
        assert torch.equal(forward(d), y)
        for g, w in zip(backward(d), back):
            assert torch.equal(g, w)


def test_infinities_and_nans_stay_with_their_tokens():
    d = make(90, 160, 130, 24, 4, 14)
    ids = d["ids"]
    ids[:8] = torch.tensor([0, 0, 1, 1, 2, 3, -1, 2], dtype=torch.int32)
    clean = forward(d)
    cleaned = backward(d)
    d["x"][0, 5], d["x"][2, 7] = float("nan"), float("inf")
    d["x"][6] = float("nan")                       # no adapter: never read
    y = forward(d)
    keep = torch.ones(90, dtype=torch.bool, device=DEV)
    keep[[0, 2]] = False
    assert torch.equal(y[keep], clean[keep]) and y[0].isnan().all()
    # +-inf by the sign of a's element, times b: nothing finite where no product is 0
    assert not y[2].isfinite().any()
    d["dy"][1, 3] = float("nan")
    d["dy"][6] = float("nan")
    dx, da, db = backward(d)
    assert dx[1].isnan().all()
    keep = torch.ones(90, dtype=torch.bool, device=DEV)
    keep[1] = False
    assert torch.equal(dx[keep], cleaned[0][keep])
    for i in (2, 3):
        assert torch.equal(da[i], cleaned[1][i]) and torch.equal(db[i], cleaned[2][i])
    assert da[0].isnan().any() and db[0].isnan().any()
    # an adapter that no token has is not read
    d = make(60, 160, 130, 16, 3, 15, [0, 2, -1])
    y, back = forward(d), backward(d)
    d["a"][1], d["b"][1], d["scale"][1] = float("nan"), float("inf"), float("nan")
    assert torch.equal(forward(d), y)
    for g, w in zip(backward(d), back):
        assert torch.equal(g, w)


def test_infinity_of_one_row_of_b():
    """An infinity in b reaches its output column with its sign, and no other."""
    d = make(20, 64, 70, 24, 1, 16, [0])
    y = forward(d)
    d["b"][0, 33, 2] = float("inf")
    got = forward(d)
    keep = torch.ones(70, dtype=torch.bool, device=DEV)
    keep[33] = False
    assert torch.equal(got[:, keep], y[:, keep])
    v = f64(d["x"]) @ f64(d["a"])[0, 2]
    assert np.array_equal(f64(got[:, 33]), np.sign(v) * np.inf)


@pytest.mark.parametrize("R", [8, 16, 40])
def test_infinities_beside_short_values(R):
    """v and u of few bits leave nothing for their lower pieces: an infinity that meets them stays one."""
    L, T, K, N = 1, 20, 24, 40
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1.0
    a = torch.zeros((L, R, K), dtype=torch.bfloat16, device=DEV)
    a[0, 0, 0] = 0.5
    b = torch.zeros((L, N, R), dtype=torch.bfloat16, device=DEV)
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
    dx, da, db = q.lora_mm_backward(dy, x, a, b, ids)
    assert da[0, 0, 1] == float("inf") and da[0, 0, 0] == 2.0 * T


def test_no_tokens():
    d = make(1, 64, 48, 16, 3, 17)
    e = {k: v[:0] if k in ("x", "ids", "base", "dy", "dbase") else v for k, v in d.items()}
    assert forward(e).shape == (0, 48)
    dx, da, db = backward(e)
    assert dx.shape == (0, 64) and not da.any() and not db.any()


def test_refusals():
    d = make(6, 64, 48, 16, 3, 18)
    with pytest.raises(q.QlinError):
        q.lora_mm(d["x"], d["a"][:, :12].contiguous(), d["b"][:, :, :12].contiguous(), d["ids"])
    with pytest.raises(ValueError):
        q.lora_mm(d["x"], d["a"], d["b"][:2], d["ids"])
    with pytest.raises(ValueError):
        q.lora_mm(d["x"], d["a"], d["b"], d["ids"][:5])
    with pytest.raises(TypeError):
        q.lora_mm(d["x"], d["a"], d["b"], d["ids"].float())
    with pytest.raises(ValueError):
        q.lora_mm(d["x"], d["a"], d["b"], d["ids"], scale=d["scale"][:2])
    with pytest.raises(ValueError):
        q.lora_mm(d["x"], d["a"], d["b"], d["ids"], base=d["base"][:, :47])
    with pytest.raises(ValueError):
        q.lora_mm(d["x"], d["a"][:, :, ::2], d["b"], d["ids"])
    with pytest.raises(ValueError):
        q.lora_mm_backward(d["dy"][:, :47], d["x"], d["a"], d["b"], d["ids"])
    with pytest.raises(ValueError):
        q.lora_mm(d["x"], d["a"], d["b"], d["ids"].cpu())


@pytest.mark.parametrize("T", [20, 200])
def test_own_stream(T):
    d = make(T, 256, 320, 32, 4, 19)
    want, back = forward(d), backward(d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y, got = forward(d), backward(d)
    s.synchronize()
    assert torch.equal(y, want) and all(torch.equal(g, w) for g, w in zip(got, back))


def test_captured_and_replayed():
    """Two graphs and eager calls between their replays; the ids change from replay to replay."""
    graphs = []
    for T, seed in ((40, 20), (300, 21)):
        d = make(T, 192, 136, 16, 5, seed)
        forward(d), backward(d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, back = forward(d), backward(d)
        graphs.append((d, g, y, back))
    for turn in range(3):
        for d, g, y, back in graphs:
            d["ids"].copy_(d["ids"].roll(turn + 1))
            d["x"].mul_(-1.0)
            g.replay()
        torch.cuda.synchronize()
        for d, g, y, back in graphs:
            assert torch.equal(forward(d), y)
            for a, b in zip(backward(d), back):
                assert torch.equal(a, b)


def test_offsets_past_4_gib():
    """Rows of base and out that start behind 2^32 bytes."""
    T, N = 34000, 65536
    d = make(8, 64, N, 8, 2, 22, [0, 1])
    x = d["x"].repeat(T // 8, 1)
    ids = d["ids"].repeat(T // 8)
    base = torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
    y = q.lora_mm(x, d["a"], d["b"], ids, scale=d["scale"], base=base, out=base)
    d["base"].zero_()
    want = forward(d)
    assert torch.equal(y[-8:], want) and torch.equal(y[:8], want) and torch.equal(y[T // 2 // 8 * 8:][:8], want)
