"""Expert routing on the GPU (moe_sort, moe_permute, moe_dispatch,
moe_combine and the gradients) against plain 64-bit references, and the whole
layer with the grouped products between."""
import sys

import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests import reference64 as ref

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-moe]", *a, flush=True)
    sys.stdout.flush()


def make_ids(T, topk, E, kind, seed=0):
    g = np.random.default_rng([seed, T, topk, E])
    if kind == "one":                       # every slot wants one expert
        return np.full((T, topk), E - 1, np.int64)
    if kind == "none":                      # every slot is absent
        return np.full((T, topk), -1, np.int64)
    ids = g.integers(0, E, (T, topk))
    if kind == "absent":                    # padding, other ranks' experts
        ids = np.where(g.random(ids.shape) < 0.3, g.choice([-1, E, E + 7, -(1 << 31), (1 << 31) - 1], ids.shape), ids)
        ids[: T // 4] = -1
    return ids.astype(np.int64)


SORTS = [(0, 2, 4), (1, 1, 1), (1, 8, 128), (3, 5, 7), (16, 8, 128), (64, 1, 2048), (333, 2, 16), (512, 8, 60),
         (513, 8, 64), (2000, 6, 257), (8191, 8, 128), (70001, 8, 5)]


@pytest.mark.parametrize("T,topk,E", SORTS)
@pytest.mark.parametrize("kind", ["even", "absent", "one", "none"])
def test_sort_matches_definition(T, topk, E, kind):
    ids = make_ids(T, topk, E, kind)
    off, row = ref.sort_reference(ids, E)
    for dt in (torch.int32, torch.int64):
        say("sort", T, topk, E, kind, dt)
        d = torch.from_numpy(ids).to(dt).cuda()
        o, r = q.moe_sort(d, E)
        torch.cuda.synchronize()
        assert np.array_equal(o.cpu().numpy(), off) and np.array_equal(r.cpu().numpy(), row)


def test_sort_of_64_bit_ids_does_not_wrap():
    ids = torch.tensor([[1, (1 << 32) + 1], [0, -(1 << 32)]], dtype=torch.int64, device="cuda")
    o, r = q.moe_sort(ids, 2)
    assert o.tolist() == [0, 1, 2] and r.tolist() == [[1, -1], [0, -1]]


def rows_of(shape, dt, seed):
    g = torch.Generator().manual_seed(seed)
    if dt in (torch.int8, torch.uint8, torch.float8_e4m3fn):
        return torch.randint(0, 127, shape, generator=g, dtype=torch.uint8).view(dt)
    return torch.randn(shape, generator=g).to(dt)


def raw(t):
    t = t.detach().cpu().contiguous()
    return t.view(torch.uint8).numpy().reshape(t.shape[0], -1) if t.numel() else np.zeros((t.shape[0], 0), np.uint8)


DISPATCHES = [
    (1, 1, 1, 1, torch.int8, None), (1, 8, 128, 2048, torch.bfloat16, None), (5, 3, 4, 100, torch.bfloat16, None),
    (16, 8, 128, 2048, torch.int8, 1), (17, 8, 60, 130, torch.float32, 1), (64, 2, 8, 768, torch.float8_e4m3fn, 6),
    (300, 4, 2048, 1027, torch.bfloat16, None), (1025, 8, 128, 384, torch.float8_e4m3fn, 3),
    (2000, 6, 16, 333, torch.float16, 2), (4, 2, 4, 40000, torch.int8, 300),
    (256, 8, 128, 200, torch.int8, 1), (257, 8, 128, 200, torch.int8, 1), (2048, 1, 2000, 16, torch.bfloat16, None),
    (2, 1024, 300, 64, torch.float32, None),
]


@pytest.mark.parametrize("T,topk,E,K,dt,cols", DISPATCHES)
@pytest.mark.parametrize("kind", ["even", "absent"])
def test_dispatch_moves_every_row(T, topk, E, K, dt, cols, kind):
    say("dispatch", T, topk, E, K, dt, cols, kind)
    ids = make_ids(T, topk, E, kind, 1)
    off, row = ref.sort_reference(ids, E)
    x = rows_of((T, K), dt, 2)
    sc = None if cols is None else torch.rand((T,) if cols == 1 else (T, cols))
    rows = T * topk + 2
    out = rows_of((rows, K), dt, 3).cuda()                # what is there stays in the rows of no slot
    so = None if sc is None else torch.full((rows, *sc.shape[1:]), -3.0).cuda()
    before = raw(out)
    want = ref.permute_reference(raw(x), row, before)
    d = torch.from_numpy(ids).cuda()
    y, ys, o, r = q.moe_dispatch(x.cuda(), d, E, None if sc is None else sc.cuda(), out=out, out_scale=so)
    torch.cuda.synchronize()
    assert np.array_equal(o.cpu().numpy(), off) and np.array_equal(r.cpu().numpy(), row)
    assert np.array_equal(raw(y), want)
    if sc is not None:
        ws = ref.permute_reference(sc.numpy(), row, np.full(tuple(so.shape), -3.0, np.float32))
        assert np.array_equal(ys.cpu().numpy(), ws)
    else:
        assert ys is None
    # moe_permute alone, rows inside a wider buffer, fewer rows than slots
    few = max(1, T * topk // 2)
    wide = rows_of((few, K + 5), dt, 4).cuda()
    want = ref.permute_reference(raw(x), row, raw(wide[:, :K]))
    beside = raw(wide[:, K:])
    xw = rows_of((T, K + 3), dt, 5).cuda()
    xw[:, 1:K + 1].view(torch.uint8).copy_(x.cuda().view(torch.uint8)) if dt.itemsize == 1 else \
        xw[:, 1:K + 1].copy_(x.cuda())
    q.moe_permute(xw[:, 1:K + 1], r, out=wide[:, :K])
    torch.cuda.synchronize()
    assert np.array_equal(raw(wide[:, :K]), want) and np.array_equal(raw(wide[:, K:]), beside)


COMBINES = [(1, 1, 1, 1), (1, 8, 128, 2048), (5, 3, 4, 100), (16, 8, 128, 2048), (17, 8, 60, 131), (333, 2, 16, 1027),
            (1025, 8, 128, 384), (3, 40, 8, 515), (2, 2, 4, 9000)]


@pytest.mark.parametrize("T,topk,E,K", COMBINES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32, torch.float16])
@pytest.mark.parametrize("kind", ["even", "absent"])
def test_combine_and_gradients(T, topk, E, K, dt, kind):
    say("combine", T, topk, E, K, dt, kind)
    ids = make_ids(T, topk, E, kind, 2)
    _, row = ref.sort_reference(ids, E)
    used = np.zeros(T * topk + 2, bool)
    used[row[row >= 0]] = True
    y = rows_of((T * topk + 2, K), dt, 6)
    y[torch.from_numpy(~used)] = float("nan")             # rows of no slot are not read
    w = torch.rand((T, topk))
    w[torch.from_numpy(row < 0)] = float("nan")           # nor are absent slots' weights
    r = torch.from_numpy(row).cuda()
    out = q.moe_combine(y.cuda(), r, w.cuda())
    half = ref.HALF[dt]
    tiny = 2.0 ** -24 if dt == torch.float16 else ref.F32_MIN          # half a step of the least fp16 value, or less
    y64, w64 = np.where(used[:, None], ref.f64(y), 0.0), np.where(row < 0, 0.0, ref.f64(w))
    want, mag = ref.combine_reference(y64, row, w64)
    # topk products and sums in fp32 (fused or not: at most 2 topk roundings), one rounding to the type
    ref.close(ref.f64(out), want, half * np.abs(want) + 1.01 * (2 * topk + 1) * 2.0 ** -24 * mag + tiny, "combine")

    dout = rows_of((T, K), dt, 7)
    dy0 = rows_of((T * topk + 2, K), dt, 8)
    dy, dw = q.moe_combine_backward(dout.cuda(), y.cuda(), r, w.cuda(), dy=dy0.cuda())
    wdy, wdw, dmag = ref.combine_backward_reference(ref.f64(dout), y64, row, w64, ref.f64(dy0))
    # one fp32 product, one rounding to the type (fp32: the product alone)
    ref.close(ref.f64(dy), wdy, (half + 1.01 * 2.0 ** -24) * np.abs(wdy) + tiny, "dy")
    # a term passes at most K / 64 + 24 additions of its lane's and the lanes' sums, and its own product
    ref.close(ref.f64(dw), wdw, 1.01 * (K / 64 + 25) * 2.0 ** -24 * dmag + ref.F32_MIN, "dweights")

    dx = q.moe_permute_backward(y.cuda(), r)
    want, mag = ref.combine_reference(y64, row, None)
    ref.close(ref.f64(dx), want, half * np.abs(want) + 1.01 * (topk + 1) * 2.0 ** -24 * mag + tiny, "dx")


def test_gradients_against_differences():
    # combine is linear in y and in w: a difference along a direction is the
    # derivative exactly, up to the fp32 roundings of the two losses
    T, topk, E, K = 20, 3, 6, 70
    _, row = ref.sort_reference(make_ids(T, topk, E, "absent", 3), E)
    r = torch.from_numpy(row).cuda()
    g = torch.Generator().manual_seed(9)
    y, vy = (torch.randn((T * topk, K), generator=g).cuda() for _ in range(2))
    w, vw = (torch.rand((T, topk), generator=g).cuda() for _ in range(2))
    d = torch.randn((T, K), generator=g).cuda()
    dy, dw = q.moe_combine_backward(d, y, r, w, dy=torch.zeros_like(y))
    loss = lambda a, b: float((d.double() * q.moe_combine(a, r, b).double()).sum())
    size = float((d.double().abs() * q.moe_combine(y.abs() + vy.abs(), r, w + vw).double()).sum())
    tol = 8 * (topk + 2) * 2.0 ** -24 * size              # roundings of y +- v, products and sums, both losses
    assert abs((loss(y + vy, w) - loss(y - vy, w)) / 2 - float((dy.double() * vy.double()).sum())) <= tol
    assert abs((loss(y, w + vw) - loss(y, w - vw)) / 2 - float((dw.double() * vw.double()).sum())) <= tol
    # permute: the loss <rows, P x> along a direction of x
    x, vx = (torch.randn((T, K), generator=g).cuda() for _ in range(2))
    dr = torch.randn((T * topk, K), generator=g).cuda()
    dx = q.moe_permute_backward(dr, r)
    loss = lambda a: float((dr.double() * q.moe_permute(a, r, out=torch.zeros_like(dr))[0].double()).sum())
    size = float((dr.double().abs() * q.moe_permute(x.abs() + vx.abs(), r, out=torch.zeros_like(dr))[0].double()).sum())
    assert abs((loss(x + vx) - loss(x - vx)) / 2 - float((dx.double() * vx.double()).sum())) \
        <= 8 * (topk + 2) * 2.0 ** -24 * size


def test_slot_rows_outside_the_buffers_count_as_absent():
    T, topk, K = 6, 2, 48
    row = np.array([[0, 99], [-7, 1], [2, 1 << 30], [-(1 << 31), 3], [4, 12], [5, (1 << 31) - 1]], np.int32)
    r = torch.from_numpy(row).cuda()
    whole = torch.zeros((12 + 4, K), dtype=torch.bfloat16, device="cuda")
    x = rows_of((T, K), torch.bfloat16, 10)
    q.moe_permute(x.cuda(), r, out=whole[:12])
    want = ref.permute_reference(raw(x), np.where((row >= 0) & (row < 12), row, -1), raw(torch.zeros((12, K), dtype=torch.bfloat16)))
    assert np.array_equal(raw(whole[:12]), want) and bool((whole[12:] == 0).all())
    w = torch.ones((T, topk), device="cuda")
    out = q.moe_combine(whole[:12], r, w)
    assert torch.equal(out.cpu(), x)
    dy, dw = q.moe_combine_backward(x.cuda(), whole[:12], r, w, dy=torch.zeros((12, K), dtype=torch.bfloat16, device="cuda"))
    assert bool((dw.cpu()[torch.from_numpy((row < 0) | (row >= 12))] == 0).all())
    assert np.array_equal(raw(dy), want)


def test_infinities_and_nan_stay_in_their_token():
    T, topk, E, K = 9, 2, 4, 64
    _, row = ref.sort_reference(make_ids(T, topk, E, "even", 4), E)
    r = torch.from_numpy(row).cuda()
    y = rows_of((T * topk, K), torch.bfloat16, 11)
    y[row[3, 1], 5] = float("inf")
    y[row[6, 0], 7] = float("nan")
    out = q.moe_combine(y.cuda(), r, torch.ones((T, topk), device="cuda")).cpu()
    assert torch.isinf(out[3, 5]) and torch.isnan(out[6, 7])
    out[3, 5] = out[6, 7] = 0
    assert bool(torch.isfinite(out).all())


def test_empty_calls():
    e = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    rows, sc, off, row = q.moe_dispatch(x, e, 3)
    assert rows.shape == (0, 64) and sc is None and off.tolist() == [0, 0, 0, 0] and row.shape == (0, 2)
    w = torch.empty((0, 2), device="cuda")
    assert q.moe_combine(x, e, w).shape == (0, 64) and q.moe_permute_backward(x, e).shape == (0, 64)
    dy, dw = q.moe_combine_backward(x, x, e, w)
    assert dy.shape == (0, 64) and dw.shape == (0, 2)
    # tokens without any sorted row
    r = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    out = q.moe_combine(x, r, torch.ones((4, 2), device="cuda"))
    assert out.shape == (4, 64) and bool((out == 0).all())
    assert bool((q.moe_combine_backward(out, x, r, torch.ones((4, 2), device="cuda"))[1] == 0).all())


def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(q.QlinError):
        q.moe_sort(ids, 0)
    with pytest.raises(q.QlinError):
        q.moe_sort(ids, 1 << 40)
    with pytest.raises(ValueError):
        q.moe_sort(ids.t(), 4)
    with pytest.raises(ValueError):
        q.moe_dispatch(x[:3], ids, 4)
    with pytest.raises(q.QlinError) as e:
        q.moe_dispatch(x, ids, 4, out=x.new_empty((7, 64)))             # fewer rows than slots
    assert e.value.status == 2
    with pytest.raises(ValueError):
        q.moe_dispatch(x, ids, 4, scale=torch.ones((3,), device="cuda"))
    with pytest.raises(ValueError):
        q.moe_dispatch(x, ids, 4, out_scale=torch.ones((8,), device="cuda"))
    with pytest.raises(TypeError):
        q.moe_combine(x, ids, torch.ones((4, 2), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        q.moe_combine(x.double(), ids, torch.ones((4, 2), device="cuda"))
    with pytest.raises(ValueError):
        q.moe_combine(x.t(), ids, torch.ones((4, 2), device="cuda"))
    with pytest.raises(ValueError):
        q.moe_combine_backward(x[:3], x, ids, torch.ones((4, 2), device="cuda"))


def layer(x, ids, w, E, gate_up, down, T):
    """A decode MoE layer with 4-bit gate_up and int8 down weights."""
    rows, _, off, row = q.moe_dispatch(x, ids, E)
    h = q.grouped_w4_mm(rows, *gate_up[:2], off, T, gate_up[2])
    a, sa = q.silu_and_mul_dynamic_per_token_quant(h, torch.int8)
    y = q.grouped_scaled_mm(a, sa, *down, off, T)
    return q.moe_combine(y, row, w)


@pytest.mark.parametrize("T", [1, 16, 200])
def test_moe_layer_runs_together_and_in_graphs(T):
    topk, E, K, H = 4, 16, 512, 256
    g = torch.Generator().manual_seed(21)
    codes = torch.randint(0, 16, (E, 2 * H, K), generator=g, dtype=torch.uint8).numpy()
    s = (0.002 + 0.002 * torch.rand((E, 2 * H, K // 128), generator=g)).to(torch.bfloat16)
    z = torch.randint(6, 10, (E, 2 * H, K // 128), generator=g, dtype=torch.uint8)
    gate_up = (torch.from_numpy(ref.pack4(codes)).cuda(), s.cuda(), z.cuda())
    dq = torch.randint(-127, 128, (E, K, H), generator=g, dtype=torch.int8)
    ds = 0.0005 + 0.0005 * torch.rand((E, K), generator=g)
    down = (dq.cuda(), ds.cuda())

    def inputs(seed):
        g = torch.Generator().manual_seed(seed)
        x = torch.randn((T, K), generator=g).to(torch.bfloat16)
        p = torch.softmax(torch.randn((T, E), generator=g), dim=1)
        w, ids = torch.topk(p, topk, dim=1)
        ids[-1, 1:] = -1                                  # a padded token's slots
        return x, ids, w.contiguous()

    def reference(x, ids, w):
        out = np.zeros((T, K))
        for t in range(T):
            for j in range(topk):
                e = int(ids[t, j])
                if e < 0:
                    continue
                h = ref.w4_weights(codes[e], ref.f64(s[e]), z[e].numpy(), 128) @ ref.f64(x[t])
                a = h[:H] / (1 + np.exp(-h[:H])) * h[H:]
                out[t] += float(w[t, j]) * (ref.f64(dq[e]) * ref.f64(ds[e])[:, None] @ a)
        return out

    def check(got, x, ids, w, what):
        want = reference(x, ids, w)
        err = np.linalg.norm(ref.f64(got) - want) / np.linalg.norm(want)
        # int8 activations: an error of at most half a step, amax / 254, on each value, spread evenly:
        # amax / 254 / sqrt(3) beside a root mean square of the SiLU products of at least amax / 16 gives
        # 0.037; the four bf16 roundings add less than 2^-7
        assert err < 0.037 + 2.0 ** -7, (what, err)

    a = inputs(30)
    say("layer", T)
    check(layer(*(t.cuda() for t in a), E, gate_up, down, T), *a, "eager")
    # two graphs over the same weights, each replayed between eager runs of the other's inputs
    graphs = []
    for k in range(2):
        st = [t.cuda() for t in inputs(31 + k)]
        layer(*st, E, gate_up, down, T)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = layer(*st, E, gate_up, down, T)
        graphs.append((gr, st, out))
    for rep in range(3):
        for k, (gr, st, out) in enumerate(graphs):
            new = inputs(40 + 2 * rep + k)
            for dst, src in zip(st, new):
                dst.copy_(src)
            gr.replay()
            torch.cuda.synchronize()
            got = out.clone()
            eager = layer(*(t.cuda() for t in new), E, gate_up, down, T)
            assert torch.equal(got, eager), (rep, k)
            check(got, *new, f"replay {rep} {k}")


def test_training_step_in_two_streams_and_a_graph():
    # permute, combine and all gradients: eager on two streams at once, then captured
    T, topk, E, K = 3000, 4, 32, 256
    ids = torch.from_numpy(make_ids(T, topk, E, "absent", 5)).cuda()
    g = torch.Generator().manual_seed(50)
    x, d = (torch.randn((T, K), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w = torch.rand((T, topk), generator=g).cuda()

    def step():
        zeros = torch.zeros((T * topk, K), dtype=torch.bfloat16, device="cuda")
        rows, _, off, row = q.moe_dispatch(x, ids, E, out=zeros)
        out = q.moe_combine(rows, row, w)
        dy, dw = q.moe_combine_backward(d, rows, row, w, dy=torch.zeros_like(rows))
        return off, row, out, dw, q.moe_permute_backward(dy, row)

    want = step()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got += [step() for _ in range(3)]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = step()
    for rep in range(3):
        gr.replay()
        torch.cuda.synchronize()
        say("training replay", rep)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        step()


def test_rows_past_4_gib():
    # sorted rows 64 Mi elements apart: permute, combine and both gradients on 8 to 10 GiB of rows
    T, topk, E, K = 40, 2, 7, 130
    ids = make_ids(T, topk, E, "absent", 8)
    _, row = ref.sort_reference(ids, E)
    g = torch.Generator().manual_seed(70)
    x = torch.randn((T, K), generator=g).to(torch.bfloat16)
    w = torch.rand((T, topk), generator=g)
    ld = (1 << 26) + 2
    say("far rows")
    far = torch.empty(T * topk * ld, dtype=torch.bfloat16, device="cuda").as_strided((T * topk, K), (ld, 1))
    far.zero_()
    r = torch.from_numpy(row).cuda()
    q.moe_permute(x.cuda(), r, out=far)
    near, _ = q.moe_permute(x.cuda(), r, out=torch.zeros((T * topk, K), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(far, near)
    assert torch.equal(q.moe_combine(far, r, w.cuda()), q.moe_combine(near, r, w.cuda()))
    assert torch.equal(q.moe_permute_backward(far, r), q.moe_permute_backward(near, r))
    dy, dw = q.moe_combine_backward(x.cuda(), near, r, w.cuda(), dy=torch.zeros_like(near))
    _, fw = q.moe_combine_backward(x.cuda(), near, r, w.cuda(), dy=far)
    assert torch.equal(far, dy) and torch.equal(fw, dw)


def test_quantized_codes_through_the_router_match_the_unsorted_product():
    # int8 codes and their scales dispatched, the grouped product, and back: each
    # row is the single product's, bit for bit up to the combine's one rounding
    T, topk, E, K, N = 40, 2, 5, 256, 64
    g = torch.Generator().manual_seed(60)
    x = torch.randn((T, K), generator=g).to(torch.bfloat16).cuda()
    b = torch.randint(-127, 128, (E, N, K), generator=g, dtype=torch.int8).cuda()
    sb = (0.01 * torch.rand((E, N), generator=g)).cuda()
    ids = torch.from_numpy(make_ids(T, topk, E, "even", 6)).cuda()
    a, sa = q.quant_per_token(x, torch.int8)
    rows, rs, off, row = q.moe_dispatch(a, ids, E, scale=sa)
    y = q.grouped_scaled_mm(rows, rs, b, sb, off, T * topk)
    for e in range(E):
        one = q.scaled_mm(a, sa, b[e], sb[e])
        t, j = torch.nonzero(ids == e, as_tuple=True)
        assert torch.equal(y[row[t, j].long()], one[t])
