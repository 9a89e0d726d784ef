"""Log probabilities, entropies, alternatives and their gradient on the GPU against
the 64-bit reference: one row to many, vocabularies of one to many, banned tokens,
rows of nothing else, ties, NaNs, strides, graphs."""
import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests import reference_ops as ref
from tests.reference64 import HALF, close, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LEAST = {torch.float32: ref.F32_MIN, torch.bfloat16: ref.F32_MIN, torch.float16: 2.0 ** -25}
INF, NAN = float("inf"), float("nan")


def make(T, V, dtype, seed, sigma=2.5, banned=0.0, bits=64, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, V), generator=g) * sigma + shift
    target = torch.randint(-1, V, (T,), generator=g)
    if T > 2:
        target[1] = V
    if banned:
        x[torch.rand((T, V), generator=g) < banned] = -INF
    d = dict(x=x.to(dtype), target=target.to(torch.int64 if bits == 64 else torch.int32),
             g=torch.randn(T, generator=g), h=torch.randn(T, generator=g) * 0.3)
    return {k: v.to(DEV) for k, v in d.items()}


def check(d, got, top, what=""):
    x, target = f64(d["x"]), d["target"].cpu().numpy()
    want = ref.logprobs(x, target, top)
    tol = ref.logprobs_bounds(x, target, want[4])
    for name, g, w, b in zip(("logprob", "entropy", "lse", "top_logprob"), got, want, tol):
        assert g.dtype == torch.float32
        g = f64(g)
        odd = ~np.isfinite(w)
        assert np.array_equal(g[odd], w[odd], equal_nan=True), (what, name)
        close(np.where(odd, 0, g), np.where(odd, 0, w), b, f"{what} {name}")
    assert got[4].dtype == torch.int32 and np.array_equal(got[4].cpu().numpy(), want[4]), what
    return want


def check_gradient(d, out, lse, entropy, h, what=""):
    want, tol = ref.logprobs_backward(f64(d["g"]), f64(d["x"]), d["target"].cpu().numpy(), f64(lse),
                                      None if entropy is None else f64(entropy), None if h is None else f64(h))
    dt = d["x"].dtype
    assert out.dtype == dt
    close(f64(out), want, ref.rounded(want, tol, HALF[dt], LEAST[dt]), what)


SHAPES = [(1, 1, 0), (1, 1, 1), (1, 7, 7), (3, 64, 64), (2, 100, 5), (5, 511, 20), (1, 4096, 1), (1, 4097, 64),
          (4, 2049, 3), (7, 8191, 32), (1, 50257, 20), (48, 10007, 5), (3, 131072, 64), (70, 4099, 2), (1100, 300, 4),
          (1030, 4111, 1), (1500, 65, 0)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,V,top", SHAPES)
def test_forward_and_gradient(T, V, top, dtype):
    d = make(T, V, dtype, T + V, bits=32 if V % 2 else 64)
    got = q.token_logprobs(d["x"], d["target"], top=top)
    check(d, got, top, str((T, V, top, dtype)))
    lse, entropy = got[2], got[1]
    out = q.token_logprobs_backward(d["g"], d["x"], d["target"], lse, entropy=entropy, dentropy=d["h"])
    check_gradient(d, out, lse, entropy, d["h"], str((T, V, dtype)))
    out = q.token_logprobs_backward(d["g"], d["x"], d["target"], lse)
    check_gradient(d, out, lse, None, None, str((T, V, dtype)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("banned", [0.5, 0.999])
def test_banned_tokens(dtype, banned):
    d = make(40, 9001, dtype, 3, banned=banned)
    d["x"][5] = -INF
    d["x"][6, :] = -INF
    d["x"][6, 4500] = 1.5
    d["x"][7] = torch.finfo(dtype).min
    d["x"][8, 100:] = torch.finfo(dtype).min
    got = q.token_logprobs(d["x"], d["target"], top=20)
    check(d, got, 20)
    out = q.token_logprobs_backward(d["g"], d["x"], d["target"], got[2], entropy=got[1], dentropy=d["h"])
    check_gradient(d, out, got[2], got[1], d["h"])
    assert not out[5].any() and torch.isfinite(out.float()).all()


@pytest.mark.parametrize("T", [1, 1200])
def test_ties_and_one_value(T):
    d = make(T, 5000, torch.bfloat16, 4)
    d["x"].round_()
    check(d, q.token_logprobs(d["x"], d["target"], top=64), 64)
    d["x"].zero_()
    d["x"][:, ::2] = -0.0                            # equal to 0: the order is the index's
    got = q.token_logprobs(d["x"], d["target"], top=64)
    check(d, got, 64)
    assert torch.equal(got[4], torch.arange(64, device=DEV, dtype=torch.int32).expand(T, 64))


@pytest.mark.parametrize("rising", [True, False])
def test_sorted_rows(rising):
    """Every logit enters the alternatives, or none after the first."""
    d = make(3, 20011, torch.float32, 5)
    d["x"] = torch.linspace(-20, 20, 20011, device=DEV).repeat(3, 1)
    if not rising:
        d["x"] = d["x"].flip(1).contiguous()
    check(d, q.token_logprobs(d["x"], d["target"], top=33), 33)


@pytest.mark.parametrize("shift", [1e4, -3e4])
def test_rows_far_from_zero(shift):
    d = make(20, 3001, torch.float32, 6, shift=shift)
    got = q.token_logprobs(d["x"], d["target"], top=3)
    check(d, got, 3)
    out = q.token_logprobs_backward(d["g"], d["x"], d["target"], got[2], entropy=got[1], dentropy=d["h"])
    check_gradient(d, out, got[2], got[1], d["h"])


@pytest.mark.parametrize("T", [6, 1100])
def test_nans_and_infinities_stay_in_their_row(T):
    d = make(T, 5003, torch.bfloat16, 7)
    clean = q.token_logprobs(d["x"], d["target"], top=8)
    dx = q.token_logprobs_backward(d["g"], d["x"], d["target"], clean[2], entropy=clean[1], dentropy=d["h"])
    d["x"][0, 4000] = NAN
    d["x"][3, 17] = INF
    d["x"][4, 5:] = NAN                              # five alternatives are left
    got = q.token_logprobs(d["x"], d["target"], top=8)
    check(d, got, 8)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[[0, 3, 4]] = False
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, clean))
    assert got[4][4].tolist()[5:] == [-1] * 3
    out = q.token_logprobs_backward(d["g"], d["x"], d["target"], got[2], entropy=got[1], dentropy=d["h"])
    assert torch.equal(out[keep], dx[keep]) and out[0].isnan().all() and out[4].isnan().all()
    # rows whose gradients are 0 are not read
    d["g"][[0, 3, 4]] = 0.0
    d["h"][[0, 3, 4]] = 0.0
    out = q.token_logprobs_backward(d["g"], d["x"], d["target"], got[2], entropy=got[1], dentropy=d["h"])
    assert not out[[0, 3, 4]].any() and torch.equal(out[keep], dx[keep])


def test_strides_and_in_place():
    d = make(30, 777, torch.bfloat16, 8)
    want = q.token_logprobs(d["x"], d["target"], top=4)
    dx = q.token_logprobs_backward(d["g"], d["x"], d["target"], want[2], entropy=want[1], dentropy=d["h"])
    wide = torch.full((30, 1001), 50.0, dtype=torch.bfloat16, device=DEV)
    wide[:, 3:780] = d["x"]
    got = q.token_logprobs(wide[:, 3:780], d["target"], top=4)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = q.token_logprobs_backward(d["g"], wide[:, 3:780], d["target"], want[2], entropy=want[1], dentropy=d["h"],
                                    out=wide[:, 3:780])
    assert torch.equal(out, dx) and torch.equal(wide[:, 3:780], dx)
    assert (wide[:, :3] == 50).all() and (wide[:, 780:] == 50).all()


def test_no_rows_and_refusals():
    d = make(4, 100, torch.float32, 9)
    got = q.token_logprobs(d["x"][:0], d["target"][:0], top=3)
    assert [tuple(g.shape) for g in got] == [(0,), (0,), (0,), (0, 3), (0, 3)]
    one = torch.zeros(4, device=DEV)
    assert q.token_logprobs_backward(one[:0], d["x"][:0], d["target"][:0], one[:0]).shape == (0, 100)
    for bad in (lambda: q.token_logprobs(d["x"], d["target"], top=65),
                lambda: q.token_logprobs(d["x"], d["target"][:3]),
                lambda: q.token_logprobs(d["x"].t(), d["target"]),
                lambda: q.token_logprobs_backward(one, d["x"], d["target"], one, dentropy=one),
                lambda: q.token_logprobs_backward(one[:3], d["x"], d["target"], one),
                lambda: q.token_logprobs_backward(one, d["x"], d["target"], one, out=d["x"].half())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        q.token_logprobs(d["x"], d["target"].float())
    with pytest.raises(q.QlinError):
        q.token_logprobs(d["x"][:, :10], d["target"], top=11)


def test_captured_and_replayed():
    graphs = []
    for T, V, seed in ((2, 30011, 10), (1040, 513, 11)):
        d = make(T, V, torch.bfloat16, seed)

        def call(d=d):
            got = q.token_logprobs(d["x"], d["target"], top=6)
            return (*got, q.token_logprobs_backward(d["g"], d["x"], d["target"], got[2], entropy=got[1],
                                                    dentropy=d["h"]))

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((d, call, g, out))
    for turn in range(3):
        for d, call, g, out in graphs:
            d["x"].copy_(d["x"].roll(turn + 1, dims=1))
            g.replay()
        torch.cuda.synchronize()
        for d, call, g, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(call(), out))
    s = torch.cuda.Stream()
    d, call, _, out = graphs[0]
    with torch.cuda.stream(s):
        got = call()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, out))


def test_offsets_past_4_gib():
    T, V = 20000, 131072
    x = torch.zeros((T, V), dtype=torch.bfloat16, device=DEV)
    d = make(3, V, torch.bfloat16, 12)
    at = [0, T // 2, T - 1]
    x[at] = d["x"]
    target = torch.zeros(T, dtype=torch.int64, device=DEV)
    target[at] = d["target"]
    got = q.token_logprobs(x, target, top=2)
    check(d, [g[at] for g in got], 2)
    g = torch.zeros(T, device=DEV)
    g[at] = d["g"]
    out = q.token_logprobs_backward(g, x, target, got[2], out=x)
    check_gradient(d, out[at], got[2][at], None, None)
    assert not out[1:T // 2].any() and not out[T // 2 + 1:T - 1].any()
