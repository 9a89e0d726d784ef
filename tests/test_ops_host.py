"""Refusals of the low-rank adapters, the log probabilities and the embedding,
without a GPU: every call here fails a check (or has nothing to do), so nothing is
launched.  At the end the 64-bit references the GPU tests use are pinned: against
worked examples, and the gradients against differences."""
import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests import reference_ops as ref

OK, NULL, SHAPE, STRIDE, ALIGN, WS, ARG = 0, 1, 2, 3, 4, 5, 9
X, A, B, I, S, Z, Y, W, G = (0x10000 * k for k in range(1, 10))       # never dereferenced
BIG = 1 << 40


def lora(bits=32, T=4, K=64, N=48, R=16, L=3, x=X, ldx=None, a=A, b=B, ids=I, s=S, base=Z, ldb=None, y=Y, ldy=None,
         ws=W, n=BIG):
    return q.lib().qlin_lora_mm(bits, T, K, N, R, L, x, K if ldx is None else ldx, a, b, ids, s, base,
                                N if ldb is None else ldb, y, N if ldy is None else ldy, ws, n, None)


def lora_backward(bits=32, T=4, K=64, N=48, R=16, L=3, dy=G, lddy=None, x=X, ldx=None, a=A, b=B, ids=I, s=S, base=Z,
                  ldb=None, dx=Y, lddx=None, da=A, db=B, ws=W, n=BIG):
    return q.lib().qlin_lora_mm_backward(bits, T, K, N, R, L, dy, N if lddy is None else lddy, x,
                                         K if ldx is None else ldx, a, b, ids, s, base, K if ldb is None else ldb, dx,
                                         K if lddx is None else lddx, da, db, ws, n, None)


@pytest.mark.parametrize("call", [lora, lora_backward])
def test_lora_refusals(call):
    assert call(bits=16) == ARG and call(bits=0) == ARG
    assert call(T=-1) == SHAPE and call(T=(1 << 24) + 1) == SHAPE
    assert call(K=0) == SHAPE and call(K=-8) == SHAPE and call(K=(1 << 20) + 1) == SHAPE
    assert call(N=-1) == SHAPE and call(N=(1 << 20) + 1) == SHAPE
    assert call(R=0) == SHAPE and call(R=4) == SHAPE and call(R=12) == SHAPE and call(R=136) == SHAPE
    assert call(L=0) == SHAPE and call(L=2048) == SHAPE
    assert call(L=2047, K=1 << 20) == SHAPE and call(L=512, R=128, N=1 << 19) == SHAPE
    assert call(x=None) == NULL and call(a=None) == NULL and call(b=None) == NULL and call(ids=None) == NULL
    assert call(ldx=63) == STRIDE and call(ldx=(1 << 31) + 1) == STRIDE
    assert call(ldb=0) == STRIDE and call(ldb=(1 << 31) + 1) == STRIDE
    assert call(x=X + 1) == ALIGN and call(a=A + 1) == ALIGN and call(b=B + 1) == ALIGN and call(base=Z + 1) == ALIGN
    assert call(ids=I + 2) == ALIGN and call(bits=64, ids=I + 4) == ALIGN and call(s=S + 2) == ALIGN
    assert call(ws=W + 8) == ALIGN
    assert call(ws=None) == WS and call(n=0) == WS


def test_lora_in_place():
    """Only `base` may be written over: X and dY are still read when the first outputs are stored."""
    assert lora(y=X, N=64) == ARG and lora(y=X, base=X, N=64) == ARG
    assert lora_backward(dx=X) == ARG and lora_backward(dx=G, N=64) == ARG


def test_lora_forward_only():
    assert lora(y=None) == NULL and lora(y=Y + 1) == ALIGN and lora(ldy=47) == STRIDE
    assert lora(T=0, x=None, ids=None, y=None, ws=None, n=0) == OK and lora(N=0, b=None, y=None, ws=None, n=0) == OK
    need = q.lib().qlin_lora_workspace_size(4, 64, 48, 16, 3)
    assert need > 0 and lora(n=need - 1) == WS
    assert q.lib().qlin_lora_workspace_size(0, 64, 48, 16, 3) == 0
    assert q.lib().qlin_lora_workspace_size(4, 64, 48, 12, 3) == 0


def test_lora_backward_only():
    assert lora_backward(N=0) == SHAPE
    assert lora_backward(dy=None) == NULL and lora_backward(dx=None) == NULL
    assert lora_backward(da=None) == NULL and lora_backward(db=None) == NULL
    assert lora_backward(dy=G + 1) == ALIGN and lora_backward(dx=Y + 1) == ALIGN
    assert lora_backward(da=A + 2) == ALIGN and lora_backward(db=B + 2) == ALIGN
    assert lora_backward(lddy=47) == STRIDE and lora_backward(lddx=63) == STRIDE
    need = q.lib().qlin_lora_backward_workspace_size(4, 64, 48, 16, 3)
    assert need > q.lib().qlin_lora_workspace_size(4, 64, 48, 16, 3) and lora_backward(n=need - 1) == WS
    # no tokens still write zeros, so the plan needs its workspace
    assert q.lib().qlin_lora_backward_workspace_size(0, 64, 48, 16, 3) > 0
    assert lora_backward(T=0, dy=None, x=None, ids=None, dx=None, ws=None, n=0) == WS


def logprobs(rt=1, bits=64, T=4, V=100, top=5, x=X, ld=None, t=I, lp=S, e=A, lse=B, tv=G, ti=Y, ws=W, n=BIG):
    return q.lib().qlin_token_logprobs(rt, bits, T, V, top, x, V if ld is None else ld, t, lp, e, lse, tv, ti, ws, n, None)


def logprobs_backward(rt=1, bits=64, T=4, V=100, g=S, h=A, x=X, ld=None, t=I, lse=B, e=G, out=Y, ldo=None):
    return q.lib().qlin_token_logprobs_backward(rt, bits, T, V, g, h, x, V if ld is None else ld, t, lse, e, out,
                                                V if ldo is None else ldo, None)


@pytest.mark.parametrize("call", [logprobs, logprobs_backward])
def test_logprobs_refusals(call):
    assert call(rt=3) == ARG and call(rt=-1) == ARG and call(bits=8) == ARG
    assert call(T=-1) == SHAPE and call(T=(1 << 23) + 1) == SHAPE and call(V=0) == SHAPE and call(V=-1) == SHAPE
    assert call(V=(1 << 28) + 1) == SHAPE
    assert call(x=None) == NULL and call(t=None) == NULL and call(lse=None) == NULL
    assert call(ld=99) == STRIDE and call(ld=(1 << 31) + 1) == STRIDE
    assert call(x=X + 1) == ALIGN and call(rt=0, x=X + 2) == ALIGN and call(t=I + 4) == ALIGN
    assert call(bits=32, t=I + 2) == ALIGN and call(lse=B + 2) == ALIGN and call(e=A + 1) == ALIGN


def test_logprobs_one_way_only():
    assert logprobs(top=-1) == SHAPE and logprobs(top=65) == SHAPE and logprobs(V=4) == SHAPE
    assert logprobs(lp=None) == NULL and logprobs(e=None) == NULL and logprobs(tv=None) == NULL
    assert logprobs(ti=None) == NULL and logprobs(ti=Y + 2) == ALIGN and logprobs(lp=S + 2) == ALIGN
    need = q.lib().qlin_token_logprobs_workspace_size(1, 1, 100000, 5)
    assert need > 0 and logprobs(T=1, V=100000, n=need - 1) == WS and logprobs(T=1, V=100000, ws=None, n=0) == WS
    assert logprobs(T=1, V=100000, ws=W + 4) == ALIGN
    assert q.lib().qlin_token_logprobs_workspace_size(1, 1 << 20, 100000, 5) == 0
    assert q.lib().qlin_token_logprobs_workspace_size(1, 1, 100000, 65) == 0
    assert logprobs(T=0, x=None, t=None, lp=None, ws=None, n=0) == OK
    assert logprobs_backward(g=None) == NULL and logprobs_backward(e=None) == NULL and logprobs_backward(out=None) == NULL
    assert logprobs_backward(ldo=99) == STRIDE and logprobs_backward(out=Y + 1) == ALIGN
    assert logprobs_backward(g=S + 2) == ALIGN and logprobs_backward(h=A + 2) == ALIGN
    assert logprobs_backward(T=0, g=None, x=None, t=None, out=None) == OK


def embedding(tt=1, ot=1, bits=64, T=4, V=100, H=256, ids=I, table=X, ldt=None, s=None, cols=0, c=1.0, out=Y, ldo=None):
    return q.lib().qlin_embedding(tt, ot, bits, T, V, H, ids, table, H if ldt is None else ldt, s, cols, c, out,
                                  H if ldo is None else ldo, None)


def test_embedding_refusals():
    assert embedding(tt=5) == ARG and embedding(tt=-1) == ARG and embedding(ot=3) == ARG and embedding(bits=16) == ARG
    assert embedding(T=-1) == SHAPE and embedding(T=1 << 30) == SHAPE and embedding(V=0) == SHAPE
    assert embedding(V=1 << 31) == SHAPE and embedding(H=0) == SHAPE and embedding(H=(1 << 20) + 1) == SHAPE
    assert embedding(s=S, cols=3) == SHAPE and embedding(s=S, cols=-1) == SHAPE
    assert embedding(H=200, s=S, cols=2) == SHAPE
    assert embedding(ids=None) == NULL and embedding(table=None) == NULL and embedding(out=None) == NULL
    assert embedding(cols=1) == NULL and embedding(cols=2) == NULL
    assert embedding(ldt=255) == STRIDE and embedding(ldo=255) == STRIDE
    assert embedding(ids=I + 4) == ALIGN and embedding(table=X + 1) == ALIGN and embedding(out=Y + 1) == ALIGN
    assert embedding(tt=0, table=X + 2) == ALIGN and embedding(s=S + 2, cols=1) == ALIGN
    assert embedding(T=0, ids=None, table=None, out=None) == OK


def embedding_backward(rt=1, ot=1, bits=64, T=4, V=100, H=256, ids=I, d=X, ldd=None, c=1.0, add=0, out=Y, ldt=None,
                       ws=W, n=BIG):
    return q.lib().qlin_embedding_backward(rt, ot, bits, T, V, H, ids, d, H if ldd is None else ldd, c, add, out,
                                           H if ldt is None else ldt, ws, n, None)


def test_embedding_backward_refusals():
    call = embedding_backward
    assert call(rt=3) == ARG and call(ot=4) == ARG and call(rt=1, ot=2) == ARG and call(rt=0, ot=1) == ARG
    assert call(bits=1) == ARG
    assert call(T=-1) == SHAPE and call(T=1 << 28) == SHAPE and call(V=0) == SHAPE and call(V=1 << 22) == SHAPE
    assert call(H=0) == SHAPE and call(H=(1 << 20) + 1) == SHAPE and call(T=1 << 27, H=4096) == SHAPE
    assert call(ids=None) == NULL and call(d=None) == NULL and call(out=None) == NULL
    assert call(T=0, out=None) == NULL
    assert call(ldd=255) == STRIDE and call(ldt=255) == STRIDE
    assert call(ids=I + 4) == ALIGN and call(d=X + 1) == ALIGN and call(out=Y + 1) == ALIGN
    assert call(ot=0, out=Y + 2) == ALIGN and call(ws=W + 8) == ALIGN
    need = q.lib().qlin_embedding_backward_workspace_size(4, 100, 256)
    assert need > 0 and call(n=need - 1) == WS and call(ws=None, n=0) == WS
    assert q.lib().qlin_embedding_backward_workspace_size(0, 100, 256) == 0
    assert q.lib().qlin_embedding_backward_workspace_size(4, 1 << 22, 256) == 0
    assert call(T=0, add=1, ids=None, d=None, ws=None, n=0) == OK


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refusals():
    """Everything on the CPU is refused before a launch."""
    ids = t(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        q.lora_mm(t(4, 64), t(3, 16, 64), t(3, 48, 16), ids)
    with pytest.raises(TypeError, match="bfloat16"):
        q.lora_mm(t(4, 64, dtype=torch.float16), t(3, 16, 64), t(3, 48, 16), ids)
    with pytest.raises(TypeError, match="bfloat16"):
        q.lora_mm_backward(t(4, 48), t(4, 64), t(3, 16, 64, dtype=torch.float32), t(3, 48, 16), ids)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        q.token_logprobs(t(4, 100, dtype=torch.float64), ids)
    with pytest.raises(ValueError, match="device tensor"):
        q.token_logprobs(t(4, 100), ids)
    with pytest.raises(ValueError, match="device tensor"):
        q.token_logprobs_backward(t(4, dtype=torch.float32), t(4, 100), ids, t(4, dtype=torch.float32))
    with pytest.raises(TypeError, match="table must be"):
        q.embedding(ids, t(100, 64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="device tensor"):
        q.embedding(ids, t(100, 64))
    with pytest.raises(ValueError, match="device tensor"):
        q.embedding_backward(t(4, 64), ids, 100)


# ---------------------------------------------------------------------------
# the references
# ---------------------------------------------------------------------------
def differences(f, x, step=1e-5):
    """Central differences of the scalar f at x."""
    out = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        y = x.copy()
        y[i] += step
        hi = f(y)
        y[i] -= 2 * step
        out[i] = (hi - f(y)) / (2 * step)
    return out


def test_lora_reference():
    x = np.array([[1.0, 2.0], [3.0, -1.0], [5.0, 7.0]])
    a = np.array([[[1.0, 1.0]], [[2.0, 0.0]]])
    b = np.array([[[1.0], [10.0]], [[-1.0], [0.5]]])
    y, _ = ref.lora(x, a, b, [1, 0, -1], [2.0, 3.0], np.ones((3, 2)))
    # token 0: v = 2, times 3; token 1: v = 2, times 2; token 2 has none
    assert np.array_equal(y, [[1 - 6, 1 + 3], [1 + 4, 1 + 40], [1, 1]])
    rng = np.random.default_rng(5)
    x, dy = rng.standard_normal((6, 5)), rng.standard_normal((6, 4))
    a, b, s = rng.standard_normal((3, 2, 5)), rng.standard_normal((3, 4, 2)), np.array([0.5, 2.0, 1.5])
    ids, base, zero = np.array([0, 2, -1, 0, 5, 2]), rng.standard_normal((6, 5)), np.zeros((6, 4))
    (dx, da, db), _ = ref.lora_backward(dy, x, a, b, ids, s, base)
    loss = lambda x, a, b: (dy * ref.lora(x, a, b, ids, s, zero)[0]).sum()
    assert np.allclose(dx - base, differences(lambda v: loss(v, a, b), x), atol=1e-7)
    assert np.allclose(da, differences(lambda v: loss(x, v, b), a), atol=1e-7)
    assert np.allclose(db, differences(lambda v: loss(x, a, v), b), atol=1e-7)
    assert not da[1].any() and np.array_equal(dx[2], base[2])


def test_logprobs_reference():
    inf = np.inf
    x = np.array([[0.0, 0.0, 0.0, 0.0], [np.log(3.0), 0.0, -inf, -inf], [-inf] * 4, [1.0, np.nan, 2.0, 0.0],
                  [5.0, inf, 0.0, 1.0]])
    lp, e, lse, tv, ti = ref.logprobs(x, [2, 1, 0, 3, 9], 3)
    assert np.allclose([lp[0], e[0], lse[0]], [-np.log(4), np.log(4), np.log(4)])
    assert np.allclose([lp[1], e[1], lse[1]], [np.log(0.25), -0.75 * np.log(0.75) - 0.25 * np.log(0.25), np.log(4)])
    assert lp[2] == -inf and e[2] == 0 and lse[2] == -inf
    assert np.isnan([lp[3], e[3], lse[3], e[4], lse[4]]).all() and lp[4] == 0
    assert ti.tolist() == [[0, 1, 2], [0, 1, 2], [0, 1, 2], [2, 0, 3], [1, 0, 3]]
    rng = np.random.default_rng(6)
    x, g, h = 2 * rng.standard_normal((3, 7)), rng.standard_normal(3), rng.standard_normal(3)
    target = [4, -1, 6]
    _, e, lse, _, _ = ref.logprobs(x, target, 0)
    dx, _ = ref.logprobs_backward(g, x, target, lse, e, h)

    def loss(v):
        lp, e, *_ = ref.logprobs(v, target, 0)
        return (g * lp + h * e).sum()

    assert np.allclose(dx, differences(loss, x), atol=1e-7)
    # a banned token stays at 0, a row of nothing else too
    x[0, 1], x[2] = -inf, -inf
    _, e, lse, _, _ = ref.logprobs(x, target, 0)
    dx, _ = ref.logprobs_backward(g, x, target, lse, e, h)
    assert dx[0, 1] == 0 and not dx[2].any() and np.isfinite(dx).all()


def test_embedding_reference():
    table = np.arange(8.0).reshape(4, 2)
    assert np.array_equal(ref.embedding([3, -1, 0, 4], table, [1, 1, 1, 0.5], 2.0), [[6, 7], [0, 0], [0, 2], [0, 0]])
    rng = np.random.default_rng(7)
    d, ids, table = rng.standard_normal((5, 3)), np.array([1, 3, 1, -1, 4]), rng.standard_normal((4, 3))
    got, _ = ref.embedding_backward(d, ids, 4, 1.5)
    assert np.allclose(got, differences(lambda v: (d * ref.embedding(ids, v, None, 1.5)).sum(), table), atol=1e-7)
    assert np.allclose(ref.embedding_backward(d, ids, 4, 1.5, table)[0], got + table)
