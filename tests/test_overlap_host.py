"""Outputs over inputs are refused: the library's own arithmetic (csrc/qlin_overlap.h) against sets of bytes, and the
calls that take it, on addresses that no call reads."""
import os
import random
import subprocess

import int8_gemm_linear_amd as q
from tests import test_ops_host as ops
from tests.test_ops_host import ARG, A, B, G, S, X, Y, Z

CSRC = os.path.join(os.path.dirname(q.LIB_PATH), "csrc")
PROGRAM = r"""
#include <stdio.h>
#include "qlin_overlap.h"
int main()
{
    long v[8];
    while (scanf("%ld %ld %ld %ld %ld %ld %ld %ld", v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6, v + 7) == 8) {
        const qlin::Region a{(void *)v[0], v[1], v[2], v[3]}, b{(void *)v[4], v[5], v[6], v[7]};
        printf("%d %d\n", (int)qlin::overlap(a, b), (int)qlin::overlap(b, a));
    }
}
"""


def held(at, rows, width, stride):
    return {at + r * stride + c for r in range(rows) for c in range(width)}


def test_overlap_of_rows(tmp_path):
    (tmp_path / "o.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "o")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(tmp_path / "o.cpp"), "-o", exe], check=True)
    rng = random.Random(3)
    cases = []
    for _ in range(20000):
        two = []
        stride = rng.randint(1, 12)
        for _ in range(2):
            width = rng.randint(1, stride)
            kind = rng.random()
            rows = 1 if kind < 0.2 else rng.randint(1, 5)
            two += [rng.randint(100, 160), rows, width, width if kind < 0.5 else stride]
        cases.append(two)
    out = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in cases), text=True, capture_output=True,
                         check=True).stdout.split("\n")
    seen = set()
    for c, line in zip(cases, out):
        want = bool(held(*c[:4]) & held(*c[4:]))
        assert line == f"{int(want)} {int(want)}", c
        seen.add(want)
    assert seen == {True, False}
    # rows of two strides are let through, nothing overlaps nothing
    line = subprocess.run([exe], input="100 3 4 8 100 3 4 9\n0 3 4 4 1 3 4 4\n100 0 4 4 100 1 4 4\n", text=True,
                          capture_output=True, check=True).stdout
    assert line == "0 0\n0 0\n0 0\n"


def test_lora():
    # T = 4, K = 64, N = 48, R = 16, L = 3: x takes 512 bytes, y 384, a 6144, b 4608, ids 16, scale 12
    call = ops.lora
    assert call(y=X + 2) == ARG and call(y=X + 510) == ARG and call(y=X - 382) == ARG
    assert call(y=A + 6142) == ARG and call(y=B - 2) == ARG and call(y=ops.I + 12) == ARG and call(y=S - 380) == ARG
    assert call(y=Z + 2) == ARG and call(y=Z, ldy=50) == ARG and call(y=Z - 96) == ARG
    assert call(y=ops.W + 16) == ARG and call(ws=X + 16, y=Y) == ARG and call(ws=B, y=Y) == ARG
    # columns of x's own rows
    assert call(ldx=200, ldy=200, y=X + 2 * 60) == ARG and call(ldx=200, ldy=200, y=X + 2 * 160) == ARG


def test_lora_backward():
    # dy takes 384 bytes, x and dx 512, da 12288, db 9216
    call = dict(da=0xA0000, db=0xB0000)
    f = lambda **kw: ops.lora_backward(**{**call, **kw})
    assert f(dx=X + 2) == ARG and f(dx=G - 510) == ARG and f(dx=A + 2) == ARG and f(dx=B) == ARG
    assert f(dx=Z + 128) == ARG and f(dx=Z, lddx=70) == ARG
    assert f(da=A) == ARG and f(db=B + 4604) == ARG and f(da=X) == ARG and f(db=G + 4) == ARG and f(da=0xB0000) == ARG
    assert f(db=0xA0000 + 12284) == ARG and f(da=Y + 4) == ARG and f(db=S + 8) == ARG and f(da=Z) == ARG
    assert f(da=ops.W) == ARG and f(ws=X) == ARG


def test_log_probabilities():
    # 4 rows of 100 in bf16, 5 alternatives: 800, 32, 16, 16, 16, 80 and 80 bytes
    call = dict(lp=0xA0000, lse=0xB0000)
    f = lambda **kw: ops.logprobs(**{**call, **kw})
    assert f(lp=X + 796) == ARG and f(e=ops.I + 28) == ARG and f(lse=0xA0000 + 12) == ARG and f(tv=Y - 76) == ARG
    assert f(ti=X) == ARG and f(ti=0xA0000) == ARG
    f = lambda **kw: ops.logprobs_backward(**{**dict(lse=0xA0000, e=0xB0000), **kw})
    assert f(out=X + 2) == ARG and f(out=X, ldo=101) == ARG and f(out=X - 798) == ARG and f(out=S) == ARG
    assert f(out=A + 12) == ARG and f(out=0xA0000) == ARG and f(out=0xB0000) == ARG and f(out=ops.I) == ARG


def test_embedding():
    # a table of 100 rows of 256 in bf16, 51200 bytes, 4 rows of it
    f = ops.embedding
    assert f(out=X + 2) == ARG and f(out=X + 51198) == ARG and f(out=X) == ARG and f(out=ops.I + 30) == ARG
    assert f(s=S, cols=1, out=S + 398) == ARG
    f = ops.embedding_backward
    assert f(out=X) == ARG and f(out=X + 2046) == ARG and f(out=X - 51198) == ARG and f(out=ops.I) == ARG
    assert f(out=ops.W) == ARG and f(ws=X) == ARG
