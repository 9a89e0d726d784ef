"""The 4-bit products (w4_mm, grouped_w4_mm) on the GPU against fp64, within
the bound their arithmetic allows (tests/reference64.py)."""
import sys

import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests import reference64 as ref

pytestmark = pytest.mark.gpu

SCALES = (torch.float32, torch.bfloat16, torch.float16)


def say(*a):
    print("[gpu-w4]", *a, flush=True)
    sys.stdout.flush()


def weights(lead, K, group, st, zero, seed):
    """(codes, scale tensor, zero points) on the host; every code occurs."""
    g = np.random.default_rng([seed, K, group, *lead])
    codes = g.integers(0, 16, (*lead, K), dtype=np.uint8)
    s = torch.from_numpy((0.002 + 0.01 * g.random((*lead, K // group))).astype(np.float32)).to(st)
    z = g.integers(0, 16, (*lead, K // group), dtype=np.uint8) if zero else None
    return codes, s, z


def tokens(M, K, seed):
    g = np.random.default_rng([seed, M, K])
    return torch.from_numpy(g.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16)


def dev(a):
    return None if a is None else (a if isinstance(a, torch.Tensor) else torch.from_numpy(a)).cuda()


# one token to hundreds; one column to thousands; K of one group upwards, and
# Ks whose last 128 (or 256) are not full; every group, scale and zero point
SHAPES = [
    (1, 1, 32, 32), (1, 16, 128, 128), (1, 17, 96, 32), (1, 2048, 2048, 128), (1, 300, 5120, 64),
    (2, 33, 320, 64), (3, 40, 640, 128), (4, 64, 256, 128), (5, 100, 1152, 128), (7, 1, 2048, 32),
    (8, 48, 1024, 32), (15, 31, 192, 64), (16, 33, 2048, 64), (17, 130, 384, 128), (31, 64, 4096, 32),
    (32, 512, 5120, 64), (33, 65, 768, 64), (48, 80, 224, 32), (64, 96, 512, 32), (65, 200, 1024, 128),
    (100, 257, 1152, 128), (130, 129, 96, 32), (257, 70, 160, 32), (300, 384, 1024, 128), (515, 272, 704, 64),
]


@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_w4_matches_fp64(M, N, K, group):
    i = SHAPES.index((M, N, K, group))
    for st, zero in ((SCALES[i % 3], False), (SCALES[(i + 1) % 3], True)):
        say(M, N, K, group, st, zero)
        codes, s, z = weights((N,), K, group, st, zero, 1)
        x = tokens(M, K, 2)
        y = q.w4_mm(dev(x), dev(ref.pack4(codes)), dev(s), dev(z))
        torch.cuda.synchronize()
        ref.w4_check(y, ref.f64(x), codes, ref.f64(s), z, group, f"{(M, N, K, group, st, zero)}")


# the streaming kernel's larger workgroups; the tiles of 16 to 64 tokens and 64
# to 256 weight rows, K whole and split,
# stages of K that end inside a stage and that do not
TILES = [
    (5, 4500, 8192), (8, 4200, 8288), (3, 33000, 640), (50, 200, 32), (9, 300, 64), (9, 700, 640), (9, 700, 768), (40, 16400, 640), (40, 16400, 512), (20, 8200, 96), (20, 8200, 256),
    (20, 3001, 1152), (20, 3001, 1280), (77, 16400, 640), (77, 16400, 512), (20, 16400, 96), (40, 16400, 256),
    (700, 100, 256), (1200, 1100, 384), (96, 3001, 2528), (64, 8200, 2048), (301, 20000, 96), (301, 20000, 160), (301, 20000, 256), (30, 700, 8352),
]


@pytest.mark.parametrize("M,N,K", TILES)
def test_w4_every_tile(M, N, K):
    for i, group in enumerate(g for g in (32, 64, 128) if K % g == 0):
        st = SCALES[(i + K // 32) % 3]
        for zero in (False, True):
            say("tile", M, N, K, group, st, zero)
            codes, s, z = weights((N,), K, group, st, zero, 31)
            x = tokens(M, K, 32)
            a = [dev(t) for t in (x, ref.pack4(codes), s, z)]
            y = q.w4_mm(*a)
            assert torch.equal(y, q.w4_mm(*a))
            # every row of x, a spread of the weights' rows with the first and last ones
            pick = np.unique(np.concatenate([np.arange(0, N, 97), np.arange(70), np.arange(max(0, N - 140), N)]))
            ref.w4_check(y[:, torch.from_numpy(pick).cuda()], ref.f64(x), codes[pick], ref.f64(s)[pick],
                         None if z is None else z[pick], group, f"{(M, N, K, group, st, zero)}")


@pytest.mark.parametrize("M", [1, 8, 9, 40, 200])
def test_w4_values_whose_products_pass_fp32(M):
    # finite tokens so large that x (128 + q) is not finite in fp32; the formula's value is
    N, K, group = 96, 512, 128
    codes, s, z = weights((N,), K, group, torch.float32, True, 41)
    x = tokens(M, K, 42)
    x[::2, 5], x[::2, 9] = 2.0 ** 126, -1.5 * 2.0 ** 126
    say("large", M)
    y = q.w4_mm(dev(x), dev(ref.pack4(codes)), dev(s), dev(z))
    ref.w4_check(y, ref.f64(x), codes, ref.f64(s), z, group, f"large {M}")


@pytest.mark.parametrize("M", [2, 40])
def test_w4_rows_and_experts_past_4_gib(M):
    # rows of y 128 Mi elements apart (of few, 1 Gi: 10 and 12 GiB), experts' weights 2 GiB apart
    N, K, group = 100, 256, 64
    codes, s, z = weights((3, N), K, group, torch.bfloat16, True, 48)
    x = tokens(3 * M, K, 49)
    packed = ref.pack4(codes)
    say("far", M)
    ldy = ((1 << 30) if M < 10 else (1 << 27)) + 8
    rows = max(M, 6)
    x = torch.cat([x, x])
    y = torch.empty(rows * ldy, dtype=torch.bfloat16, device="cuda")
    out = y.as_strided((rows, N), (ldy, 1))
    q.w4_mm(dev(x[:rows]), dev(packed[0]), dev(s[0]), dev(z[0]), out=out)
    ref.w4_check(out, ref.f64(x[:rows]), codes[0], ref.f64(s[0]), z[0], group, "far rows")
    del y, out
    apart = (1 << 31) + 64
    b = torch.empty(3 * apart, dtype=torch.uint8, device="cuda").as_strided((3, N, K // 2), (apart, K // 2, 1))
    b.copy_(dev(packed))
    off = torch.tensor([0, M, 2 * M, 3 * M], dtype=torch.int32, device="cuda")
    got = q.grouped_w4_mm(dev(x[:3 * M]), b, dev(s), off, M, dev(z))
    for e in range(3):
        ref.w4_check(got[e * M:(e + 1) * M], ref.f64(x[e * M:(e + 1) * M]), codes[e], ref.f64(s[e]), z[e], group,
                     f"far expert {e}")


@pytest.mark.parametrize("M,N,K", [(1, 5120, 8192), (300, 4096, 4096)])
def test_w4_nothing_but_nan(M, N, K):
    x = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    b, s = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda"), torch.ones((N, K // 128), device="cuda")
    say("nan", M, N, K)
    assert bool(torch.isnan(q.w4_mm(x, b, s)).all())


@pytest.mark.parametrize("M", [1, 30, 300])
def test_w4_upper_bits_of_zero_points_are_not_read(M):
    N, K, group = 200, 768, 64
    codes, s, z = weights((N,), K, group, torch.bfloat16, True, 43)
    x, b, sd = dev(tokens(M, K, 44)), dev(ref.pack4(codes)), dev(s)
    more = np.random.default_rng(45).integers(0, 16, z.shape, dtype=np.uint8) << 4
    say("zero points", M)
    assert torch.equal(q.w4_mm(x, b, sd, dev(z)), q.w4_mm(x, b, sd, dev(z | more)))


def test_w4_two_streams_and_two_graphs_with_parts_of_k():
    # 30 tokens on a long K: every call sums parts in a workspace of its own
    M, N, K, group = 30, 300, 8192, 128
    codes, s, z = weights((N,), K, group, torch.bfloat16, False, 46)
    b, sd = dev(ref.pack4(codes)), dev(s)
    xs = [dev(tokens(M, K, 47 + i)) for i in range(2)]
    want = [q.w4_mm(x, b, sd) for x in xs]
    ref.w4_check(want[0], ref.f64(xs[0]), codes, ref.f64(s), None, group, "parts")
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for rep in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(q.w4_mm(xs[i], b, sd))
    torch.cuda.synchronize()
    say("streams")
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    graphs = []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = q.w4_mm(x, b, sd)
        graphs.append((g, y))
    for rep in range(3):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        say("graphs", rep)
        assert all(torch.equal(y, w) for (_, y), w in zip(graphs, want))
        assert torch.equal(q.w4_mm(xs[0], b, sd), want[0])


@pytest.mark.parametrize("M,N,K,group", [(3, 50, 512, 64), (40, 50, 512, 32), (200, 140, 512, 128)])
def test_w4_strides_and_neighbours(M, N, K, group):
    # rows inside wider buffers, the columns beside them untouched
    codes, s, z = weights((N,), K, group, torch.bfloat16, True, 3)
    x = tokens(M, K, 4)
    xb = torch.full((M, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    xb[:, :K] = dev(x)
    bb = torch.full((N, K // 2 + 32), 0xFF, dtype=torch.uint8, device="cuda")
    bb[:, :K // 2] = dev(ref.pack4(codes))
    yb = torch.full((M, N + 13), 7.0, dtype=torch.bfloat16, device="cuda")
    say("strides", M, N, K, group)
    out = q.w4_mm(xb[:, :K], bb[:, :K // 2], dev(s), dev(z), out=yb[:, :N])
    torch.cuda.synchronize()
    assert out.data_ptr() == yb.data_ptr()
    ref.w4_check(yb[:, :N], ref.f64(x), codes, ref.f64(s), z, group, "strided")
    assert bool((yb[:, N:] == 7.0).all())
    assert torch.equal(out, q.w4_mm(dev(x), dev(ref.pack4(codes)), dev(s), dev(z)))


@pytest.mark.parametrize("M,N,K,group", [(2, 40, 384, 128), (20, 40, 384, 64), (150, 70, 384, 32)])
def test_w4_nonfinite_rows(M, N, K, group):
    # an infinity gives what the formula gives (infinite, or NaN where its
    # weight is 0); a NaN gives a NaN row; the other rows are as ever
    codes, s, z = weights((N,), K, group, torch.float32, True, 5)
    x = tokens(M, K, 6)
    x[0, 5] = float("inf")
    x[1, 100] = float("nan")
    if M > 2:
        x[M - 1, K - 1] = float("-inf")
        x[M - 2, 0], x[M - 2, 1] = float("inf"), float("-inf")
    say("nonfinite", M, N, K, group)
    y = ref.f64(q.w4_mm(dev(x), dev(ref.pack4(codes)), dev(s), dev(z)))
    with np.errstate(invalid="ignore"):
        want = (ref.f64(x)[:, None, :] * ref.w4_weights(codes, ref.f64(s), z, group)[None]).sum(axis=2)
    odd = ~np.isfinite(ref.f64(x)).all(axis=1)
    assert np.array_equal(np.isnan(y[odd]), np.isnan(want[odd]))
    fine = ~np.isnan(want[odd])
    assert np.array_equal(y[odd][fine], want[odd][fine])
    keep = torch.from_numpy(np.flatnonzero(~odd))
    if keep.numel():
        ref.w4_check(torch.from_numpy(y)[keep], ref.f64(x)[~odd], codes, ref.f64(s), z, group, "finite rows")


def test_w4_empty_and_refused():
    b, s = torch.zeros((64, 128), dtype=torch.uint8, device="cuda"), torch.ones((64, 2), device="cuda")
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    assert q.w4_mm(x[:0], b, s).shape == (0, 64)
    assert q.w4_mm(x, b[:0], s[:0]).shape == (4, 0)
    with pytest.raises(ValueError):
        q.w4_mm(x, b, torch.ones((64, 16), device="cuda"))              # a group of 16
    with pytest.raises(ValueError):
        q.w4_mm(x, b[:, :64], s)
    with pytest.raises(ValueError):
        q.w4_mm(x, b, s.t().contiguous().t())
    with pytest.raises(TypeError):
        q.w4_mm(x, b, s.double())
    with pytest.raises(TypeError):
        q.w4_mm(x, b, s, s)
    with pytest.raises(q.QlinError) as e:
        q.w4_mm(x.view(-1)[4:4 + 256].view(1, 256), b, s)               # 8 bytes off
    assert e.value.status == 4
    with pytest.raises(ValueError):
        q.w4_mm(x, b, s, out=torch.empty((4, 63), dtype=torch.bfloat16, device="cuda"))


def grouped_case(sizes, N, K, group, st, zero, seed, behind=0):
    E = len(sizes)
    codes, s, z = weights((E, N), K, group, st, zero, seed)
    x = tokens(int(sum(sizes)) + behind, K, seed + 1)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    return x, codes, s, z, off


def grouped_check(y, case, group, max_rows, fill, what):
    x, codes, s, z, off = case
    yh = y.cpu()
    written = torch.zeros(yh.shape[0], dtype=torch.bool)
    for e in range(len(off) - 1):
        lo, hi = int(off[e]), min(int(off[e + 1]), int(off[e]) + max_rows)
        if hi > lo:
            written[lo:hi] = True
            ref.w4_check(yh[lo:hi], ref.f64(x[lo:hi]), codes[e], ref.f64(s[e]), None if z is None else z[e], group,
                         f"{what} expert {e}")
    assert bool((yh[~written] == fill).all()), f"{what}: rows of no expert"


GROUPED = [
    ([2, 0, 1, 5, 0, 0, 3, 6, 1, 0, 2, 4], 96, 512, 128),
    ([0, 0, 1], 17, 96, 32),
    ([16, 17, 0, 31, 1], 64, 320, 64),
    ([130, 0, 257, 64, 1], 80, 256, 128),
    ([40, 33, 90], 144, 768, 64),
    ([1] * 40, 33, 256, 32),
    ([3] * 20 + [60, 0, 200], 1300, 384, 128),
    ([20, 9, 31, 12] * 12, 700, 512, 64),
    ([100, 70, 0, 129] * 6, 1030, 160, 32),
    ([70, 33, 0, 90] * 16, 1300, 320, 64),
    ([25, 10, 31, 40] * 16, 1300, 256, 128),
    ([1, 9, 0, 14, 20, 3] * 20, 1100, 192, 32),
    ([90, 300, 1, 65] * 10, 100, 160, 32),
]


@pytest.mark.parametrize("sizes,N,K,group", GROUPED, ids=[str(i) for i in range(len(GROUPED))])
def test_grouped_w4_matches_fp64(sizes, N, K, group):
    i = GROUPED.index((sizes, N, K, group))
    for st, zero in ((SCALES[i % 3], True), (SCALES[(i + 1) % 3], False)):
        # rows behind the last expert stay; bounds exact, loose and too small
        case = grouped_case(sizes, N, K, group, st, zero, 7, behind=3)
        x, codes, s, z, off = case
        for max_rows in (max(sizes), 4096, max(1, max(sizes) // 2)):
            say("grouped", sizes[:6], N, K, group, st, zero, max_rows)
            y = torch.full((x.shape[0], N), 3.0, dtype=torch.bfloat16, device="cuda")
            q.grouped_w4_mm(dev(x), dev(ref.pack4(codes)), dev(s), dev(off), max_rows, dev(z), out=y)
            torch.cuda.synchronize()
            grouped_check(y, case, group, max_rows, 3.0, f"{i} {max_rows}")


def test_grouped_w4_offsets_stay_inside_the_buffers():
    # offsets past the rows, negative and falling: held to 0..rows, rows of
    # experts that end up empty are not computed, nothing else is touched
    sizes, N, K, group = [3, 4, 5], 32, 256, 64
    case = grouped_case(sizes, N, K, group, torch.float32, False, 9)
    x, codes, s, z, _ = case
    off = np.array([-5, 4, 2, 100000], np.int32)     # rows 2 and 3 are two experts': either's
    whole = torch.full((x.shape[0] + 64, N), 3.0, dtype=torch.bfloat16, device="cuda")
    say("bad offsets")
    q.grouped_w4_mm(dev(x), dev(ref.pack4(codes)), dev(s), dev(off), 64, out=whole[:x.shape[0]])
    torch.cuda.synchronize()
    assert bool((whole[x.shape[0]:] == 3.0).all())
    y = whole[:x.shape[0]].cpu()
    ref.w4_check(y[0:2], ref.f64(x[0:2]), codes[0], ref.f64(s[0]), None, group, "expert 0")
    ref.w4_check(y[4:], ref.f64(x[4:]), codes[2], ref.f64(s[2]), None, group, "expert 2")


def test_grouped_w4_equals_single_product():
    # one expert with every row, and the expert stride of a wider buffer
    M, N, K, group = 50, 72, 384, 128
    codes, s, z = weights((2, N), K, group, torch.bfloat16, True, 11)
    x = dev(tokens(M, K, 12))
    wide = torch.zeros((2, N + 5, K // 2), dtype=torch.uint8, device="cuda")
    wide[:, :N] = dev(ref.pack4(codes))
    off = torch.tensor([0, 0, M], dtype=torch.int32, device="cuda")
    y = q.grouped_w4_mm(x, wide[:, :N], dev(s), off, M, dev(z))
    assert torch.equal(y, q.w4_mm(x, wide[1, :N], dev(s)[1], dev(z)[1]))


@pytest.mark.parametrize("M", [1, 24, 200])
def test_w4_graph_replay(M):
    # captured on a side stream, replayed with eager work between
    N, K, group = 160, 1024, 128
    codes, s, z = weights((N,), K, group, torch.bfloat16, False, 13)
    b, sd = dev(ref.pack4(codes)), dev(s)
    x = dev(tokens(M, K, 14))
    out = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    q.w4_mm(x, b, sd, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.w4_mm(x, b, sd, out=out)
    for rep in range(3):
        x.copy_(dev(tokens(M, K, 20 + rep)))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        say("replay", M, rep)
        assert torch.equal(out, q.w4_mm(x, b, sd))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y = q.w4_mm(x, b, sd)
    st.synchronize()
    assert torch.equal(out, y)
