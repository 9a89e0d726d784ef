"""The adapters, the log probabilities and the embedding as they are used together:
a training step of a small model on frozen 4-bit weights, tokens to adapters'
gradients.  Every stage is checked against the 64-bit reference on the values that
the stage before it gave, and the whole step captured and replayed."""
import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests import reference64 as ref4
from tests import reference_ops as ref
from tests.reference64 import close, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
V, H, T, R, L, GROUP = 1003, 256, 150, 16, 3, 64


def model(seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 16, (V, H), generator=g)
    m = dict(table=torch.randn((V, H), generator=g).to(torch.bfloat16),
             q4=torch.from_numpy(ref4.pack4(codes.numpy())), s4=(torch.rand((V, H // GROUP), generator=g) * 0.02),
             a=(torch.randn((L, R, H), generator=g) / 16).to(torch.bfloat16),
             b=(torch.randn((L, V, R), generator=g) / 8).to(torch.bfloat16),
             scale=torch.tensor([0.5, 1.0, 2.0]), ids=torch.randint(-1, V, (T,), generator=g),
             adapter=torch.randint(-1, L, (T,), generator=g), target=torch.randint(-1, V, (T,), generator=g),
             weight=-torch.rand(T, generator=g) / T, bonus=-torch.rand(T, generator=g) / T)
    return codes.numpy(), {k: v.to(DEV) for k, v in m.items()}


def step(m):
    x = q.embedding(m["ids"], m["table"], scale=2.0)
    y = q.w4_mm(x, m["q4"], m["s4"])
    logits = q.lora_mm(x, m["a"], m["b"], m["adapter"], m["scale"], base=y)
    logprob, entropy, lse, top, top_id = q.token_logprobs(logits, m["target"], top=4)
    dlogits = q.token_logprobs_backward(m["weight"], logits, m["target"], lse, entropy, m["bonus"])
    dx, da, db = q.lora_mm_backward(dlogits, x, m["a"], m["b"], m["adapter"], m["scale"])
    dtable = q.embedding_backward(dx, m["ids"], V, scale=2.0, dtype=torch.float32)
    return dict(x=x, y=y, logits=logits, logprob=logprob, entropy=entropy, lse=lse, top=top, top_id=top_id,
                dlogits=dlogits, dx=dx, da=da, db=db, dtable=dtable)


def test_step():
    codes, m = model(1)
    o = step(m)
    ids, adapter, target = (m[k].cpu().numpy() for k in ("ids", "adapter", "target"))
    x = ref.embedding(ids, f64(m["table"]), None, 2.0)
    close(f64(o["x"]), x, ref.rounded(x, 0 * x))
    ref4.w4_check(o["y"], f64(o["x"]), codes, f64(m["s4"]), None, GROUP)
    a, b, s = f64(m["a"]), f64(m["b"]), f64(m["scale"])
    want, tol = ref.lora(f64(o["x"]), a, b, adapter, s, f64(o["y"]))
    close(f64(o["logits"]), want, ref.rounded(want, tol))
    logits = f64(o["logits"])
    want = ref.logprobs(logits, target, 4)
    tol = ref.logprobs_bounds(logits, target, want[4])
    for name, w, t in zip(("logprob", "entropy", "lse", "top"), want, tol):
        close(f64(o[name]), w, t, name)
    assert np.array_equal(o["top_id"].cpu().numpy(), want[4])
    want, tol = ref.logprobs_backward(f64(m["weight"]), logits, target, f64(o["lse"]), f64(o["entropy"]), f64(m["bonus"]))
    close(f64(o["dlogits"]), want, ref.rounded(want, tol))
    want, tol = ref.lora_backward(f64(o["dlogits"]), f64(o["x"]), a, b, adapter, s, np.zeros((T, H)))
    close(f64(o["dx"]), want[0], ref.rounded(want[0], tol[0]))
    close(f64(o["da"]), want[1], tol[1] + ref.F32_MIN)
    close(f64(o["db"]), want[2], tol[2] + ref.F32_MIN)
    want, tol = ref.embedding_backward(f64(o["dx"]), ids, V, 2.0)
    close(f64(o["dtable"]), want, ref.rounded(want, tol, ref4.F32_HALF))


def test_captured_step():
    _, m = model(2)
    step(m)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(m)
    for turn in range(3):
        for k in ("ids", "adapter", "target"):
            m[k].copy_(m[k].roll(turn + 1))
        m["a"].mul_(-1)
        g.replay()
        torch.cuda.synchronize()
        for k, v in step(m).items():
            assert torch.equal(v, out[k]), (turn, k)
