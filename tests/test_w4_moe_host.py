"""Refusals of the 4-bit products and the expert routing, without a GPU:
every call here fails a check (or has nothing to do), so nothing is
launched.  The 64-bit references the GPU tests use are pinned at the end."""
import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests import reference64 as ref

OK, NULL, SHAPE, STRIDE, ALIGN, WS, ARG = 0, 1, 2, 3, 4, 5, 9
A, B, S, Z, Y, I, O, R, W = (0x10000 * k for k in range(1, 10))       # never dereferenced


def w4(M=4, N=64, K=256, group=128, x=A, ldx=None, b=B, ldb=None, st=0, s=S, z=None, y=Y, ldy=None, ws=None, n=0):
    return q.lib().qlin_w4_mm(M, N, K, group, x, K if ldx is None else ldx, b, K // 2 if ldb is None else ldb,
                              st, s, z, y, N if ldy is None else ldy, ws, n, None)


def test_w4_refusals():
    assert w4(M=-1) == SHAPE and w4(N=-1) == SHAPE and w4(K=0) == SHAPE and w4(K=-128) == SHAPE
    assert w4(K=192, group=128) == SHAPE and w4(K=(1 << 20) + 128) == SHAPE
    assert w4(group=16) == ARG and w4(group=0) == ARG and w4(group=256) == ARG and w4(st=3) == ARG
    assert w4(x=None) == NULL and w4(b=None) == NULL and w4(s=None) == NULL and w4(y=None) == NULL
    assert w4(ldx=248) == STRIDE and w4(ldx=260) == STRIDE and w4(ldb=112) == STRIDE and w4(ldb=136) == STRIDE
    assert w4(ldy=63) == STRIDE
    assert w4(x=A + 8) == ALIGN and w4(b=B + 4) == ALIGN and w4(y=Y + 2) == ALIGN and w4(s=S + 2) == ALIGN
    need = q.lib().qlin_w4_workspace_size(32, 512, 8192)
    assert need > 0 and need % (32 * 512 * 4) == 0 and q.lib().qlin_w4_workspace_size(1, 512, 8192) == 0
    assert q.lib().qlin_w4_workspace_size(-1, 512, 8192) == 0
    assert w4(M=32, N=512, K=8192) == WS and w4(M=32, N=512, K=8192, ws=W, n=need - 1) == WS
    assert w4(M=32, N=512, K=8192, ws=W + 8, n=need) == ALIGN
    assert w4(M=0, x=None, y=None) == OK and w4(N=0, b=None, s=None, y=None) == OK


def grouped(groups=4, off=O, max_rows=8, rows=16, N=64, K=256, group=64, x=A, b=B, stride=64 * 128, st=1, s=S,
            z=Z, y=Y):
    return q.lib().qlin_grouped_w4_mm(groups, off, max_rows, rows, N, K, group, x, K, b, K // 2, stride, st, s, z,
                                      y, N, None)


def test_grouped_w4_refusals():
    assert grouped(groups=-1) == SHAPE and grouped(groups=65536) == SHAPE and grouped(rows=-1) == SHAPE
    assert grouped(max_rows=-1) == SHAPE and grouped(N=-1) == SHAPE
    assert grouped(off=None) == NULL and grouped(off=O + 2) == ALIGN
    assert grouped(stride=-16) == STRIDE and grouped(stride=8) == STRIDE
    assert grouped(group=48) == ARG and grouped(x=None) == NULL and grouped(b=B + 8) == ALIGN
    assert grouped(groups=0, off=None) == OK and grouped(rows=0, x=None, y=None) == OK
    assert grouped(max_rows=0) == OK


def sort(bits=32, T=8, topk=2, E=4, ids=I, off=O, row=R, ws=None, n=0):
    return q.lib().qlin_moe_sort(bits, T, topk, E, ids, off, row, ws, n, None)


def test_sort_refusals():
    assert sort(bits=16) == ARG and sort(bits=0) == ARG
    assert sort(T=-1) == SHAPE and sort(topk=0) == SHAPE and sort(topk=1025) == SHAPE
    assert sort(E=0) == SHAPE and sort(E=2049) == SHAPE and sort(T=1 << 30, topk=1) == SHAPE
    assert sort(ids=None) == NULL and sort(off=None) == NULL and sort(row=None) == NULL
    assert sort(ids=I + 2) == ALIGN and sort(bits=64, ids=I + 4) == ALIGN and sort(off=O + 1) == ALIGN
    need = q.lib().qlin_moe_sort_workspace_size(100000, 8, 64)
    assert need > 0 and q.lib().qlin_moe_sort_workspace_size(16, 8, 64) == 0
    assert q.lib().qlin_moe_sort_workspace_size(-1, 8, 64) == 0
    assert sort(T=100000, topk=8, E=64) == WS and sort(T=100000, topk=8, E=64, ws=W, n=need - 1) == WS
    assert sort(T=100000, topk=8, E=64, ws=W + 2, n=need) == ALIGN


def permute(T=8, topk=2, rows=16, nbytes=64, x=A, ldx=64, row=R, out=Y, ldo=64, s=None, cols=0, so=None):
    return q.lib().qlin_moe_permute(T, topk, rows, nbytes, x, ldx, row, out, ldo, s, cols, so, None)


def test_permute_refusals():
    assert permute(T=-1) == SHAPE and permute(topk=0) == SHAPE and permute(rows=-1) == SHAPE
    assert permute(nbytes=0) == SHAPE and permute(nbytes=(1 << 22) + 1, ldx=1 << 23, ldo=1 << 23) == SHAPE
    assert permute(x=None) == NULL and permute(out=None) == NULL and permute(row=None) == NULL
    assert permute(s=S, cols=1) == NULL and permute(cols=1, so=S) == NULL and permute(cols=-1) == SHAPE
    assert permute(ldx=63) == STRIDE and permute(ldo=63) == STRIDE
    assert permute(row=R + 1) == ALIGN and permute(s=S + 2, cols=1, so=Z) == ALIGN
    assert permute(T=0, x=None, out=None, row=None) == OK and permute(rows=0, out=None) == OK
    assert permute(T=0, nbytes=0) == SHAPE


def dispatch(T=8, topk=2, E=4, rows=16, nbytes=64, x=A, out=Y, ldo=64, off=O, row=R):
    return q.lib().qlin_moe_dispatch(32, T, topk, E, I, rows, nbytes, x, 64, out, ldo, None, 0, None, off, row,
                                     None, 0, None)


def test_dispatch_refusals():
    assert dispatch(rows=15) == SHAPE and dispatch(nbytes=0) == SHAPE and dispatch(E=0) == SHAPE
    assert dispatch(x=None) == NULL and dispatch(out=None) == NULL and dispatch(off=None) == NULL
    assert dispatch(ldo=32) == STRIDE and dispatch(T=4096, topk=2, rows=8192) == WS


def combine(rt=1, T=8, topk=2, rows=16, K=64, y=A, ldy=64, row=R, w=W, out=Y, ldo=64):
    return q.lib().qlin_moe_combine(rt, T, topk, rows, K, y, ldy, row, w, out, ldo, None)


def backward(rt=1, T=8, topk=2, rows=16, K=64, d=A, ldo=64, y=B, ldy=64, row=R, w=W, dy=Y, lddy=64, dw=S):
    return q.lib().qlin_moe_combine_backward(rt, T, topk, rows, K, d, ldo, y, ldy, row, w, dy, lddy, dw, None)


def test_combine_refusals():
    assert combine(rt=3) == ARG and combine(T=-1) == SHAPE and combine(K=0) == SHAPE and combine(rows=-1) == SHAPE
    assert combine(y=None) == NULL and combine(row=None) == NULL and combine(w=None) == NULL
    assert combine(out=None) == NULL and combine(ldy=63) == STRIDE and combine(ldo=63) == STRIDE
    assert combine(y=A + 1) == ALIGN and combine(rt=0, out=Y + 2) == ALIGN and combine(w=W + 1) == ALIGN
    assert combine(T=0, y=None, row=None, w=None, out=None) == OK
    assert backward(rt=7) == ARG and backward(topk=0) == SHAPE and backward(K=(1 << 20) + 1) == SHAPE
    for name in ("d", "y", "row", "w", "dy", "dw"):
        assert backward(**{name: None}) == NULL, name
    assert backward(ldo=1) == STRIDE and backward(ldy=1) == STRIDE and backward(lddy=1) == STRIDE
    assert backward(dy=Y + 1) == ALIGN and backward(dw=S + 2) == ALIGN and backward(T=0, d=None) == OK
    pb = q.lib().qlin_moe_permute_backward
    assert pb(1, 8, 2, 16, 64, None, 64, R, Y, 64, None) == NULL
    assert pb(5, 8, 2, 16, 64, A, 64, R, Y, 64, None) == ARG
    assert pb(1, 0, 2, 16, 64, None, 64, None, None, 64, None) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    b = torch.zeros((64, 128), dtype=torch.uint8)
    s = torch.ones((64, 2))
    with pytest.raises(ValueError):
        q.w4_mm(x, b, s)
    with pytest.raises(TypeError):
        q.w4_mm(x.float(), b, s)
    with pytest.raises(TypeError):
        q.w4_mm(x, b.to(torch.int32), s)
    off = torch.zeros((2,), dtype=torch.int32)
    with pytest.raises(ValueError):
        q.grouped_w4_mm(x, b[None], s[None], off, 4)
    ids = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        q.moe_sort(ids, 4)
    with pytest.raises(TypeError):
        q.moe_sort(ids.float(), 4)
    with pytest.raises(ValueError):
        q.moe_dispatch(x, ids, 4)
    with pytest.raises(ValueError):
        q.moe_permute(x, ids)
    with pytest.raises(ValueError):
        q.moe_combine(x, ids, torch.ones((4, 2)))
    with pytest.raises(TypeError):
        q.moe_combine(ids, ids, torch.ones((4, 2)))
    with pytest.raises(TypeError):
        q.moe_combine_backward(x.float(), x, ids, torch.ones((4, 2)))
    with pytest.raises(ValueError):
        q.moe_permute_backward(x, ids)


def test_references():
    # the sort against an explicit small table; the product against a loop
    off, row = ref.sort_reference(np.array([[2, 0], [-1, 2], [0, 3]]), 3)
    assert off.tolist() == [0, 2, 2, 4] and row.tolist() == [[2, 0], [-1, 3], [1, -1]]
    g = np.random.default_rng(1)
    codes = g.integers(0, 16, (3, 64))
    packed = ref.pack4(codes)
    assert packed.shape == (3, 32) and packed[1, 5] == codes[1, 10] + 16 * codes[1, 11]
    s, z = g.random((3, 2)), g.integers(0, 16, (3, 2))
    w = ref.w4_weights(codes, s, z, 32)
    for n in range(3):
        for k in range(64):
            assert w[n, k] == s[n, k // 32] * (float(codes[n, k]) - float(z[n, k // 32]))
    y = g.standard_normal((4, 5))
    out, mag = ref.combine_reference(y, row, np.ones((3, 2)) * 2.0)
    assert np.allclose(out[0], 2 * (y[2] + y[0])) and np.allclose(out[1], 2 * y[3]) and np.all(mag >= np.abs(out))
    dy, dw, _ = ref.combine_backward_reference(out, y, row, np.full((3, 2), 2.0), np.zeros((4, 5)))
    assert np.allclose(dy[3], 2 * out[1]) and np.allclose(dw[1], [0, out[1] @ y[3]])
