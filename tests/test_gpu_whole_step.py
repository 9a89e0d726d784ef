"""A training step of adapters on a frozen 4-bit product whose gradients are whole: the frozen product's own share of
x's gradient, dy times its weights, goes in as `base` (torch computes it; the library's products have no gradients)."""
import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests import reference64 as ref4
from tests import reference_ops as ref
from tests.reference64 import close, f64
from tests.test_gpu_adapter_step import DEV, GROUP, V, model

pytestmark = pytest.mark.gpu


def step(m, weights):
    x = q.embedding(m["ids"], m["table"], scale=2.0)
    y = q.w4_mm(x, m["q4"], m["s4"])
    logits = q.lora_mm(x, m["a"], m["b"], m["adapter"], m["scale"], base=y, out=y)
    logprob, entropy, lse, _, _ = q.token_logprobs(logits, m["target"])
    dlogits = q.token_logprobs_backward(m["weight"], logits, m["target"], lse, entropy, m["bonus"])
    base = torch.mm(dlogits.float(), weights).to(torch.bfloat16)
    dx, da, db = q.lora_mm_backward(dlogits, x, m["a"], m["b"], m["adapter"], m["scale"], base=base)
    dtable = q.embedding_backward(dx, m["ids"], V, scale=2.0, dtype=torch.float32)
    return dict(x=x, logits=logits, dlogits=dlogits, base=base, dx=dx, da=da, db=db, dtable=dtable)


def weights_of(codes, m):
    """The 4-bit product's weights, fp32 on the GPU and in 64 bits."""
    w = ref4.w4_weights(codes, f64(m["s4"]), None, GROUP)
    return torch.from_numpy(w).float().to(DEV), w


def test_step():
    codes, m = model(3)
    weights, w = weights_of(codes, m)
    o = step(m, weights)
    ids, adapter = m["ids"].cpu().numpy(), m["adapter"].cpu().numpy()
    a, b, s = f64(m["a"]), f64(m["b"]), f64(m["scale"])
    dl, x = f64(o["dlogits"]), f64(o["x"])
    # the frozen share: the weights are off by 2^-24, a sum of V products in fp32 by V steps at most, rounded to bf16
    want, mag = dl @ w, np.abs(dl) @ np.abs(w)
    close(f64(o["base"]), want, ref.rounded(want, ref.ADD * (V + 4) * mag))
    (dx, da, db), tol = ref.lora_backward(dl, x, a, b, adapter, s, f64(o["base"]))
    close(f64(o["dx"]), dx, ref.rounded(dx, tol[0]))
    close(f64(o["da"]), da, tol[1] + ref.F32_MIN)
    close(f64(o["db"]), db, tol[2] + ref.F32_MIN)
    want, tol = ref.embedding_backward(f64(o["dx"]), ids, V, 2.0)
    close(f64(o["dtable"]), want, ref.rounded(want, tol, ref4.F32_HALF))


def test_captured_step():
    codes, m = model(4)
    weights, _ = weights_of(codes, m)
    step(m, weights)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(m, weights)
    for turn in range(3):
        for k in ("ids", "adapter", "target"):
            m[k].copy_(m[k].roll(turn + 1))
        g.replay()
        torch.cuda.synchronize()
        now = step(m, weights)
        for k in ("x", "logits", "dlogits"):
            assert torch.equal(now[k], out[k]), (turn, k)
        # (torch's product need not give the same bits; what follows it does, from the base that it gave)
        got = q.lora_mm_backward(out["dlogits"], out["x"], m["a"], m["b"], m["adapter"], m["scale"], base=out["base"])
        for k, v in zip(("dx", "da", "db"), got):
            assert torch.equal(v, out[k]), (turn, k)
        assert torch.equal(q.embedding_backward(got[0], m["ids"], V, scale=2.0, dtype=torch.float32), out["dtable"]), turn
