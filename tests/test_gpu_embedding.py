"""Embedding lookup and its gradient on the GPU against the 64-bit reference: plain
tables and codes, padding, tokens that fill many chunks, widths that no piece
divides, both digits of the sort, accumulation, graphs."""
import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests import reference_ops as ref
from tests.reference64 import HALF, close, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LEAST = {torch.float32: ref.F32_MIN, torch.bfloat16: ref.F32_MIN, torch.float16: 2.0 ** -25}
TABLES = [torch.float32, torch.bfloat16, torch.float16, torch.int8, torch.float8_e4m3fn]


def codes(V, H, dtype, g):
    x = torch.randn((V, H), generator=g)
    if dtype == torch.int8:
        return (x * 40).round().clamp(-127, 127).to(dtype)
    return (x * 60).clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)


def table64(t):
    return f64(t.float())


@pytest.mark.parametrize("dtype", TABLES)
@pytest.mark.parametrize("T,V,H,cols", [(1, 1, 1, 0), (1, 100, 128, 1), (5, 7, 3, 1), (33, 300, 257, 0), (16, 1000, 5120, 40),
                                        (300, 64, 384, 3), (2000, 513, 130, 1), (7, 20, 12, 0), (64, 33, 2048, 16)])
def test_lookup(T, V, H, cols, dtype):
    g = torch.Generator().manual_seed(T + V + H)
    table = codes(V, H, dtype, g)
    ids = torch.randint(-1, V + 1, (T,), generator=g)
    scale = None if cols == 0 else torch.rand((V,) if cols == 1 else (V, cols), generator=g) + 0.1
    if scale is not None and H == 128:
        scale = scale.view(V, 1)                     # one group of 128
    for out in (None, torch.float32, torch.bfloat16, torch.float16):
        got = q.embedding(ids.to(torch.int32 if T % 2 else torch.int64).to(DEV), table.to(DEV),
                          None if scale is None else scale.to(DEV), scale=0.75, dtype=out)
        if out is None:
            out = table.dtype if table.dtype in HALF else torch.bfloat16
        assert got.dtype == out
        want = ref.embedding(ids.numpy(), table64(table), None if scale is None else f64(scale), 0.75)
        # two fp32 products, then one rounding
        close(f64(got), want, ref.rounded(want, 2.0 ** -23 * np.abs(want), HALF[out], LEAST[out]), str((T, V, H, dtype)))


def test_codes_of_the_quantizers():
    x = torch.randn((200, 256), device=DEV).to(torch.bfloat16)
    ids = torch.arange(199, -1, -1, device=DEV)
    for c, s in (q.quant_per_token(x), q.quant_per_token(x, torch.int8), q.quant_per_group128(x)):
        got = q.embedding(ids, c, s)
        want = ref.embedding(ids.cpu().numpy(), f64(c.float()), f64(s), 1.0)
        close(f64(got), want, ref.rounded(want, 2.0 ** -23 * np.abs(want)))


def test_every_e4m3_code():
    c = torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).view(256, 1)
    got = q.embedding(torch.arange(256, device=DEV), c, dtype=torch.float32)
    want = c.float()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0))


def test_lookup_strides():
    wide = torch.randn((50, 300), device=DEV)
    ids = torch.randint(0, 50, (20,), device=DEV)
    out = torch.full((20, 300), 5.0, device=DEV)
    q.embedding(ids, wide[:, 7:207], out=out[:, 50:250])
    assert torch.equal(out[:, 50:250], wide[ids, 7:207]) and (out[:, :50] == 5).all() and (out[:, 250:] == 5).all()


def check_gradient(dout, ids, V, scale, got, table=None, what=""):
    want, tol = ref.embedding_backward(f64(dout), ids.cpu().numpy(), V, scale, table)
    close(f64(got), want, ref.rounded(want, tol, HALF[got.dtype], LEAST[got.dtype]), what)
    return want


# tokens, vocabulary, width, the number of different tokens
GRADIENTS = [(1, 1, 1, 1), (1, 100, 64, 1), (15, 100, 5, 100), (16, 2047, 64, 3), (17, 2048, 33, 17), (40, 50, 130, 1),
             (500, 2100, 1025, 40), (4096, 131072, 64, 2000), (4097, 131072, 70, 500), (9000, 1 << 20, 8, 9000),
             (20000, 3000, 16, 2), (70000, (1 << 22) - 1, 4, 1000), (3000, 300, 4100, 300)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,V,H,kinds", GRADIENTS)
def test_gradient(T, V, H, kinds, dtype):
    g = torch.Generator().manual_seed(T + V + H)
    some = torch.randint(-1, V + 1, (kinds,), generator=g)
    ids = some[torch.randint(0, kinds, (T,), generator=g)].to(torch.int32 if T % 2 else torch.int64).to(DEV)
    dout = torch.randn((T, H), generator=g).to(dtype).to(DEV)
    got = q.embedding_backward(dout, ids, V, scale=1.5)
    assert got.dtype == dtype and got.shape == (V, H)
    if V * H > 1 << 23:                              # the rows of any token, and that the others are 0
        used = torch.unique(ids[(ids >= 0) & (ids < V)].long())
        assert int((got != 0).any(dim=1).sum()) <= used.numel()
        place = torch.full((V + 2,), -1, dtype=torch.int64, device=DEV)
        place[used] = torch.arange(used.numel(), device=DEV)
        small = torch.where((ids >= 0) & (ids < V), place[ids.clamp(min=0).long()], -1)
        check_gradient(dout, small, max(used.numel(), 1), 1.5, got[used] if used.numel() else got[:1] * 0)
        return
    check_gradient(dout, ids, V, 1.5, got)
    if dtype != torch.float32:
        got = q.embedding_backward(dout, ids, V, scale=1.5, dtype=torch.float32)
        assert got.dtype == torch.float32
        check_gradient(dout, ids, V, 1.5, got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_accumulated_gradient(dtype):
    V, H, T = 90, 200, 1000
    held = torch.randn((V, H), device=DEV).to(dtype)
    ids = torch.randint(-3, 60, (T,), device=DEV)
    dout = torch.randn((T, H), device=DEV).to(torch.bfloat16)
    out = held.clone()
    if dtype == torch.bfloat16:
        held[60:, 0] = float("nan")                  # rows of no token are not read
        out[60:, 0] = float("nan")
    assert q.embedding_backward(dout, ids, V, scale=0.5, out=out, accumulate=True) is out
    check_gradient(dout, ids, 60, 0.5, out[:60], f64(held[:60]))
    assert torch.equal(out[60:].nan_to_num(3.0), held[60:].nan_to_num(3.0))


def test_gradient_strides():
    V, H, T = 40, 90, 300
    ids = torch.randint(0, V, (T,), device=DEV)
    wide = torch.randn((T, 120), device=DEV)
    want = q.embedding_backward(wide[:, 11:101].contiguous(), ids, V)
    out = torch.full((V, 150), 8.0, device=DEV)
    q.embedding_backward(wide[:, 11:101], ids, V, out=out[:, 30:120])
    assert torch.equal(out[:, 30:120], want) and (out[:, :30] == 8).all() and (out[:, 120:] == 8).all()


def test_nans_stay_in_their_rows():
    V, H, T = 50, 64, 400
    ids = torch.randint(1, V, (T,), device=DEV)
    ids[7], ids[9] = 0, -1
    dout = torch.randn((T, H), device=DEV)
    want = q.embedding_backward(dout, ids, V)
    dout[7, 3] = float("nan")
    dout[9] = float("nan")                           # padding: not read
    got = q.embedding_backward(dout, ids, V)
    assert got[0, 3].isnan() and torch.equal(got[1:], want[1:]) and int(got.isnan().sum()) == 1


def test_no_tokens_and_refusals():
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    table = torch.ones((10, 8), device=DEV)
    assert q.embedding(none, table).shape == (0, 8)
    got = q.embedding_backward(torch.zeros((0, 8), device=DEV), none, 10)
    assert got.shape == (10, 8) and not got.any()
    assert torch.equal(q.embedding_backward(torch.zeros((0, 8), device=DEV), none, 10, out=table, accumulate=True), table)
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    d = torch.zeros((4, 8), device=DEV)
    for bad in (lambda: q.embedding(ids.view(2, 2), table), lambda: q.embedding(ids[::2], table),
                lambda: q.embedding(ids, table, torch.ones((10, 2), device=DEV)),
                lambda: q.embedding(ids, table, torch.ones(9, device=DEV)),
                lambda: q.embedding(ids, table, out=torch.zeros((4, 9), device=DEV)),
                lambda: q.embedding_backward(d, ids[:3], 10), lambda: q.embedding_backward(d, ids, 10, accumulate=True),
                lambda: q.embedding_backward(d, ids, 10, out=torch.zeros((9, 8), device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q.embedding(ids.float(), table), lambda: q.embedding(ids, table.double()),
                lambda: q.embedding(ids, table, dtype=torch.int8),
                lambda: q.embedding_backward(d, ids, 10, dtype=torch.bfloat16)):
        with pytest.raises(TypeError):
            bad()
    for vocab in (0, -1, 1 << 22):
        with pytest.raises(q.QlinError):
            q.embedding_backward(d[:, :1], ids, vocab)


def test_captured_and_replayed():
    graphs = []
    for T, V, H in ((60, 500, 130), (6000, 20000, 64)):
        ids = torch.randint(-1, V, (T,), device=DEV)
        ids[: T // 2] = 3
        d = torch.randn((T, H), device=DEV).to(torch.bfloat16)
        table = torch.randn((V, H), device=DEV).to(torch.bfloat16)
        call = lambda ids=ids, d=d, table=table, V=V: (q.embedding(ids, table), q.embedding_backward(d, ids, V))
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((ids, call, g, out))
    for turn in range(3):
        for ids, call, g, out in graphs:
            ids.copy_(ids.roll(turn + 5))
            g.replay()
        torch.cuda.synchronize()
        for ids, call, g, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(call(), out))


def test_offsets_past_4_gib():
    V, H = 300000, 8192
    table = torch.zeros((V, H), dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, V // 2, V - 1], device=DEV)
    table[at] = torch.randn((3, H), device=DEV).to(torch.bfloat16)
    assert torch.equal(q.embedding(at.flip(0), table), table[at.flip(0)])
    d = torch.randn((3, H), device=DEV).to(torch.bfloat16)
    got = q.embedding_backward(d, at, V, out=table)
    assert torch.equal(got[at], d) and not got[1:V // 2].any() and not got[V // 2 + 1:V - 1].any()
