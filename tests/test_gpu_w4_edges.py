"""4-bit products on the GPU at the edges of what the header allows."""
import sys

import numpy as np
import pytest
import torch

import int8_gemm_linear_amd as q
from tests import reference64 as ref

pytestmark = pytest.mark.gpu

LOW, HIGH = -(1 << 31), (1 << 31) - 1


def say(*a):
    print("[gpu-w4-edges]", *a, flush=True)
    sys.stdout.flush()


def weights(lead, K, group, seed):
    """(packed codes, codes, fp32 scales, zero points) on the GPU and the host."""
    g = np.random.default_rng([seed, K, group, *lead])
    codes = g.integers(0, 16, (*lead, K), dtype=np.uint8)
    s = (0.002 + 0.01 * g.random((*lead, K // group))).astype(np.float32)
    z = g.integers(0, 16, (*lead, K // group), dtype=np.uint8)
    return codes, s, z


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def tokens(M, K, seed):
    return torch.randn((M, K), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("rows", [12, 120])
def test_offsets_whose_differences_pass_32_bits_stay_inside_the_buffers(rows):
    # few rows and many: both kernels.  The second expert's offsets fall by 2^31 and
    # more, the third's rise by as much; x and y have rows behind those of the call
    N, K, group, mid = 40, 256, 64, rows // 12
    codes, s, z = weights((3, N), K, group, 1)
    x = tokens(rows + 40, K, 2)
    xd, b, sd, zd = x.cuda(), gpu(ref.pack4(codes)), gpu(s), gpu(z)
    for off in ([0, mid, LOW, rows], [0, mid, LOW, HIGH], [mid, HIGH, LOW, HIGH]):
        say("offsets", rows, off)
        whole = torch.full((rows + 40, N), 3.0, dtype=torch.bfloat16, device="cuda")
        q.grouped_w4_mm(xd[:rows], b, sd, torch.tensor(off, dtype=torch.int32, device="cuda"), 4 * rows, zd,
                        out=whole[:rows])
        torch.cuda.synchronize()
        assert bool((whole[rows:] == 3.0).all())
        # the third expert has all rows; those before `mid` (or behind) are the first's too
        lo, hi = (mid, rows) if off[0] == 0 else (0, mid)
        ref.w4_check(whole[lo:hi], ref.f64(x[lo:hi]), codes[2], s[2], z[2], group, str(off))


@pytest.mark.parametrize("M,N,K,group", [(1, 700, 8192, 128), (8, 5120, 2528, 32), (30, 300, 25600, 64),
                                         (200, 1030, 4160, 64), (700, 600, 1152, 128)])
def test_infinities_and_nan_at_the_size_of_a_layer(M, N, K, group):
    # every kernel and the sum of the parts: an infinity in each row (in half of them
    # one of either sign as well), a NaN row and a row of values whose products pass
    # fp32, against the formula in fp64 on the GPU
    codes, s, z = weights((N,), K, group, 3)
    x = tokens(M, K, 4)
    r = torch.arange(M)
    x[r, (r * 37) % K] = float("inf")
    x[r[::2], (r[::2] * 37 + 5) % K] = float("-inf")
    if M > 2:
        x[1] = tokens(1, K, 5)[0] * 2.0 ** 124
        x[2, K - 1] = float("nan")
    say("infinities", M, N, K, group)
    b, sd, zd = gpu(ref.pack4(codes)), gpu(s), gpu(z)
    y = q.w4_mm(x.cuda(), b, sd, zd).double().cpu()
    w = torch.from_numpy(ref.w4_weights(codes, s, z, group)).cuda()
    want = torch.empty((M, N), dtype=torch.float64, device="cuda")
    for m in range(M):                                  # elementwise: no product's own way with NaN
        want[m] = (w * x[m].cuda().double()).sum(dim=1)
    want = want.cpu()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(y[inf], want[inf]) and bool(inf.any())
    if M > 2:
        # bf16 ends at (2 - 2^-7) 2^127; from half a step above, (2 - 2^-8) 2^127, a value
        # rounds to an infinity (none of these lies within 2^-20 of that border)
        past = (want[1].abs() >= (2 - 2.0 ** -8) * 2.0 ** 127).numpy()
        assert np.array_equal(ref.f64(y[1])[past], np.sign(ref.f64(want[1])[past]) * np.inf)
        ref.w4_check(y[1:2, torch.from_numpy(~past)], ref.f64(x[1:2]), codes[~past], s[~past], z[~past], group,
                     "large values")


@pytest.mark.parametrize("M", [2, 40])
def test_infinite_scales_multiply_their_groups_sum(M):
    # the formula scales a group's sum, not its terms: an infinite scale gives an
    # infinity of that sum's sign, also where some of the group's codes equal its zero point
    N, K, group = 70, 512, 128
    codes, s, z = weights((N,), K, group, 6)
    codes[:, ::3] = np.repeat(z, group, axis=1)[:, ::3]
    s[::2, 1] = np.inf
    x = tokens(M, K, 7)
    say("infinite scale", M)
    y = ref.f64(q.w4_mm(x.cuda(), gpu(ref.pack4(codes)), gpu(s), gpu(z)))
    sums = ((codes - np.repeat(z, group, axis=1).astype(np.float64))[None] * ref.f64(x)[:, None, :])
    sums = sums.reshape(M, N, K // group, group).sum(axis=3)
    assert np.array_equal(y[:, ::2], np.sign(sums[:, ::2, 1]) * np.inf)
    ref.w4_check(torch.from_numpy(y[:, 1::2]), ref.f64(x), codes[1::2], s[1::2], z[1::2], group, "finite scales")


def test_strides_of_a_single_expert_or_row_are_not_read():
    M, K, group = 20, 256, 64
    x = tokens(M, K, 8).cuda()
    for G, N, strides in ((1, 24, (7, K // 2, 1)), (3, 1, (K // 2, 7, 1)), (1, 1, (5, 3, 1))):
        say("strides", G, N)
        codes, s, z = weights((G, N), K, group, 9)
        b, sd, zd = gpu(ref.pack4(codes)), gpu(s), gpu(z)
        off = torch.tensor([0, *[M - G + 1 + g for g in range(G)]], dtype=torch.int32, device="cuda")
        want = q.grouped_w4_mm(x, b, sd, off, M, zd)
        assert torch.equal(q.grouped_w4_mm(x, b.as_strided((G, N, K // 2), strides), sd, off, M, zd), want)
