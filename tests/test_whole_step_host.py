"""What a training step of adapters on frozen products is made of, in 64 bits: the gradient that reaches x is the
adapters' share and the frozen product's, dy times its weights, which the caller adds as `base`."""
import numpy as np

from tests import reference_ops as ref
from tests.test_ops_host import differences


def test_gradients_of_a_step():
    rng = np.random.default_rng(11)
    V, H, T, R, L = 7, 5, 6, 2, 3
    table, W = rng.standard_normal((V, H)), rng.standard_normal((V, H))
    a, b, s = rng.standard_normal((L, R, H)), rng.standard_normal((L, V, R)), np.array([0.5, 2.0, 1.5])
    ids, adapter, target = np.array([1, 3, 1, -1, 6, 0]), np.array([0, 2, -1, 1, 0, 2]), np.array([4, -1, 6, 0, 2, 2])
    g, h = rng.standard_normal(T), rng.standard_normal(T)

    def forward(table, a, b):
        x = ref.embedding(ids, table, None, 1.5)
        logits = ref.lora(x, a, b, adapter, s, x @ W.T)[0]
        return x, logits, ref.logprobs(logits, target, 0)

    def loss(table, a, b):
        lp, entropy, *_ = forward(table, a, b)[2]
        return (g * lp + h * entropy).sum()

    x, logits, (_, entropy, lse, _, _) = forward(table, a, b)
    dlogits = ref.logprobs_backward(g, logits, target, lse, entropy, h)[0]
    (dx, da, db), _ = ref.lora_backward(dlogits, x, a, b, adapter, s, dlogits @ W)
    dtable = ref.embedding_backward(dx, ids, V, 1.5)[0]
    assert np.allclose(dtable, differences(lambda t: loss(t, a, b), table), atol=1e-6)
    assert np.allclose(da, differences(lambda t: loss(table, t, b), a), atol=1e-6)
    assert np.allclose(db, differences(lambda t: loss(table, a, t), b), atol=1e-6)
    # the adapters' share alone is not the gradient
    part = ref.embedding_backward(dx - dlogits @ W, ids, V, 1.5)[0]
    assert not np.allclose(part, dtable, atol=1e-2)
