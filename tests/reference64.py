"""Plain 64-bit references of the 4-bit products and the expert routing, and
the error bounds the kernels' arithmetic allows.  numpy on the CPU; nothing
here is shared with the library."""
import numpy as np
import torch

BF16_HALF = 2.0 ** -8         # half a step of bf16, relative
F16_HALF = 2.0 ** -11
F32_HALF = 2.0 ** -24
HALF = {torch.bfloat16: BF16_HALF, torch.float16: F16_HALF, torch.float32: F32_HALF}
F32_MIN = 2.0 ** -126


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def pack4(codes):
    """Codes 0..15 [..., K] -> bytes [..., K/2], k even in the low nibble."""
    codes = np.asarray(codes, np.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def w4_weights(codes, scale, zero, group):
    """s (q - z) in fp64, [N, K]."""
    z = 8.0 if zero is None else np.repeat(np.asarray(zero, np.float64), group, axis=-1)
    return np.repeat(np.asarray(scale, np.float64), group, axis=-1) * (np.asarray(codes, np.float64) - z)


def w4_check(y, x, codes, scale, zero, group, what=""):
    """y (bf16 tensor) against x W^T in fp64.

    Bound: each value is rounded to bf16 once (half a step of the result);
    before that the sums are fp32.  Inside a group the kernels add products
    of x with 128 + q and take (128 + z) times the group's sum of x away, or
    with 143 + q - z and 143 times it: at most group + 4 additions, each off
    by at most 2^-23 (the matrix cores need not round to nearest) of
    sum |x| (286 + q), which is at least sum |x| (256 + q + z) and
    sum |x| (286 + q - z); then K / group + 40 additions (groups, then waves)
    of the groups' true values times s (groups of 128 may be taken in two)."""
    x, codes = np.asarray(x, np.float64), np.asarray(codes)
    s = np.repeat(np.asarray(scale, np.float64), group, axis=-1)
    z = np.full(codes.shape, 8.0) if zero is None else np.repeat(np.asarray(zero, np.float64), group, axis=-1)
    ref = x @ (s * (codes - z)).T
    ax, K = np.abs(x), x.shape[1]
    inner = ax @ (np.abs(s) * (286.0 + codes)).T
    outer = ax @ (np.abs(s) * np.abs(codes - z)).T
    tol = BF16_HALF * np.abs(ref) + 1.01 * 2.0 ** -23 * ((group + 4) * inner + (2 * (K // group) + 40) * outer) + F32_MIN
    got = f64(y)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} values off; first at " \
        f"{tuple(np.argwhere(bad)[0])}: {got[tuple(np.argwhere(bad)[0])]} for {ref[tuple(np.argwhere(bad)[0])]}"
    return ref


def sort_reference(ids, experts):
    """(offsets, slot_row) by the definition, slots in order."""
    flat = np.asarray(ids).reshape(-1)
    offsets = np.array([np.sum((flat >= 0) & (flat < e)) for e in range(experts + 1)], np.int32)
    row = np.full(flat.shape, -1, np.int32)
    for e in range(experts):
        at = np.flatnonzero(flat == e)
        row[at] = offsets[e] + np.arange(at.size)
    return offsets, row.reshape(np.asarray(ids).shape)


def permute_reference(x, slot_row, out):
    """`out` with out[slot_row[t, j]] = x[t] (any numpy type)."""
    out = np.array(out)
    for j in range(slot_row.shape[1]):
        at = (slot_row[:, j] >= 0) & (slot_row[:, j] < out.shape[0])
        out[slot_row[at, j]] = x[at]
    return out


def combine_reference(y, slot_row, weights):
    """(sum_j w y, sum_j |w y|) in fp64; weights None: 1."""
    y = np.asarray(y, np.float64)
    out = np.zeros((slot_row.shape[0], y.shape[1]))
    mag = np.zeros_like(out)
    for j in range(slot_row.shape[1]):
        at = (slot_row[:, j] >= 0) & (slot_row[:, j] < y.shape[0])
        v = y[slot_row[at, j]]
        if weights is not None:
            v = v * np.asarray(weights, np.float64)[at, j][:, None]
        out[at] += v
        mag[at] += np.abs(v)
    return out, mag


def combine_backward_reference(dout, y, slot_row, weights, dy):
    """(dy, dweights, sum_k |dout y|) in fp64; rows of no slot as in dy."""
    dout, y, dy = np.asarray(dout, np.float64), np.asarray(y, np.float64), np.array(dy, np.float64)
    dw = np.zeros(slot_row.shape)
    mag = np.zeros(slot_row.shape)
    for j in range(slot_row.shape[1]):
        at = (slot_row[:, j] >= 0) & (slot_row[:, j] < y.shape[0])
        r = slot_row[at, j]
        dy[r] = np.asarray(weights, np.float64)[at, j][:, None] * dout[at]
        dw[at, j] = (dout[at] * y[r]).sum(axis=1)
        mag[at, j] = np.abs(dout[at] * y[r]).sum(axis=1)
    return dy, dw, mag


def close(got, ref, tol, what=""):
    got, ref = np.asarray(got), np.asarray(ref)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; first at {at}: {got[at]} for {ref[at]}")
