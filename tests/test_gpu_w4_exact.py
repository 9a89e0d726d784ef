"""4-bit products bit for bit: whole-number tokens of at most 2 and scales that are
powers of two make every product and every fp32 sum exact, in whatever order (in
units of the least scale no sum passes 25600 * 2 * 15 * 4 < 2^22, and inside a group
128 * 2 * 158 < 2^16), so the outputs are the formula's values rounded once.  Tokens
that are mostly zero keep the sums below 256 or so, where bf16 holds every whole
number and a single product too many or too few shows."""
import sys

import pytest
import torch

import int8_gemm_linear_amd as q
from tests import w4_cases

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-w4-exact]", *a, flush=True)
    sys.stdout.flush()


def generator(*seed):
    return torch.Generator(device="cuda").manual_seed(hash(seed) & 0x7fffffff)


def weights(lead, K, group, st, zero, g):
    """(packed codes, scales, zero points or None, the weights in fp64)."""
    codes = torch.randint(0, 16, (*lead, K), generator=g, device="cuda", dtype=torch.uint8)
    s = 2.0 ** -torch.randint(0, 3, (*lead, K // group), generator=g, device="cuda").double()
    z = torch.randint(0, 16, s.shape, generator=g, device="cuda", dtype=torch.uint8) if zero else None
    w = codes.view(*s.shape, group).double()
    w = (w - (8.0 if z is None else z.double().unsqueeze(-1))) * s.unsqueeze(-1)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), s.to(st), z, w.view(*lead, K)


def tokens(M, K, g, few):
    x = torch.randint(-2, 3, (M, K), generator=g, device="cuda")
    if few:
        x = torch.where(torch.rand((M, K), generator=g, device="cuda") < 256 / K, x, 0)
    return x.to(torch.bfloat16)


def formula(x, w):
    return torch.matmul(x.double(), w.t()).to(torch.bfloat16)


def forms(i):
    """Scale types and zero points of case i: both sizes of a scale, with and without."""
    for st in (torch.float32, (torch.bfloat16, torch.float16)[i % 2]):
        for zero in (False, True):
            yield st, zero


@pytest.mark.parametrize("i", range(len(w4_cases.DENSE)), ids=lambda i: "-".join(map(str, w4_cases.DENSE[i])))
def test_w4_is_exact(i):
    M, N, K, group = w4_cases.DENSE[i]
    for st, zero in forms(i):
        say(M, N, K, group, st, zero)
        g = generator(M, N, K, group, zero)
        b, s, z, w = weights((N,), K, group, st, zero, g)
        for few in (False, True):
            x = tokens(M, K, g, few)
            assert torch.equal(q.w4_mm(x, b, s, z), formula(x, w)), (st, zero, few)


@pytest.mark.parametrize("i", range(len(w4_cases.EXPERTS)), ids=lambda i: "-".join(map(str, w4_cases.EXPERTS[i])))
def test_grouped_w4_is_exact(i):
    E, rows, N, K, group = w4_cases.EXPERTS[i]
    for st, zero in forms(i):
        say(E, rows, N, K, group, st, zero)
        g = generator(E, rows, N, K, group, zero)
        b, s, z, w = weights((E, N), K, group, st, zero, g)
        # ragged experts, some without rows, and a few rows behind the last
        cuts = torch.randint(0, max(1, rows - 3) + 1, (E + 1,), generator=g, device="cuda").sort().values
        cuts[0], off = 0, None
        off = cuts.to(torch.int32)
        most = int((off[1:] - off[:-1]).max())
        for few in (False, True):
            x = tokens(rows, K, g, few)
            want = torch.full((rows, N), -3.0, dtype=torch.bfloat16, device="cuda")
            y = want.clone()
            for e in range(E):
                lo, hi = int(off[e]), int(off[e + 1])
                if hi > lo:
                    want[lo:hi] = formula(x[lo:hi], w[e])
            q.grouped_w4_mm(x, b, s, off, most, z, out=y)
            assert torch.equal(y, want), (st, zero, few)


@pytest.mark.parametrize("M,N,K", [(3, 90, 1024), (3, 90, 96), (40, 90, 1024), (40, 90, 96)])
def test_values_below_the_normal_range_are_kept(M, N, K):
    # tokens of a few steps of bf16's least value, 2^-133: their products are whole
    # numbers of it and fp32 holds them; scales of 2^120 bring the sums back
    say("subnormal", M, N, K)
    g = generator(M, N, K)
    b, s, z, w = weights((N,), K, 32, torch.float32, True, g)
    x = tokens(M, K, g, False)
    small = (x.double() * 2.0 ** -133).to(torch.bfloat16)
    assert torch.equal(small.double() * 2.0 ** 133, x.double())
    assert torch.equal(q.w4_mm(small, b, s * 2.0 ** 120, z).double(), (formula(x, w).double() * 2.0 ** -13))
