"""How the 4-bit products divide their work, without a GPU: the library's own
arithmetic (csrc/qlin_w4_plan.h) compiled for the host."""
import os
import subprocess

import pytest

import int8_gemm_linear_amd as q

CSRC = os.path.join(os.path.dirname(q.LIB_PATH), "csrc")
LOW, HIGH = -(1 << 31), (1 << 31) - 1

PROGRAM = r"""
#include <stdio.h>
#include "qlin_w4_plan.h"
int main()
{
    int from, to, rows, most, beg;
    while (scanf("%d %d %d %d", &from, &to, &rows, &most) == 4) {
        const int n = qlin::w4::expert_rows(from, to, rows, most, beg);
        printf("%d %d\n", beg, n);
    }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    exe = str(d / "plan")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow",
                           "-fno-sanitize-recover", "-D__host__=", "-D__device__=", "-I", CSRC,
                           str(d / "plan.cpp"), "-o", exe])
    return exe


def test_rows_of_any_offset_table_lie_inside_the_buffers(plan):
    values = [LOW, LOW + 1, -5, -1, 0, 1, 4, 5, 6, 1 << 24, HIGH - 4, HIGH]
    cases = [(f, t, rows, most) for f in values for t in values for rows in (0, 1, 6, 1 << 24)
             for most in (1, 3, 6, 1 << 24)]
    out = subprocess.run([plan], input="\n".join(" ".join(map(str, c)) for c in cases), text=True,
                         capture_output=True, check=True).stdout.split()
    got = list(zip(map(int, out[::2]), map(int, out[1::2])))
    assert len(got) == len(cases)
    for (f, t, rows, most), (beg, n) in zip(cases, got):
        lo, hi = (min(max(v, 0), rows) for v in (f, t))
        assert beg == lo and n == min(max(hi - lo, 0), most), (f, t, rows, most, beg, n)
        assert 0 <= beg and beg + n <= rows


def test_products_of_more_threads_than_a_launch_takes_are_refused():
    # a grid of 2^32 threads would be taken modulo that: nothing is launched here
    shape, p = 2, 0x10000
    lib = q.lib()
    big = 1 << 24
    assert lib.qlin_w4_mm(big, big, 32, 32, p, 32, p, 16, 0, p, None, p, big, None, 0, None) == shape
    # experts of few rows (streamed) and of many (tiles)
    for rows in (16, big):
        assert lib.qlin_grouped_w4_mm(65535, p, rows, rows, big, 32, 32, p, 32, p, 16, 1 << 28, 0, p, None, p, big,
                                      None) == shape, rows
    # a K so long that parts would pay: not where their sum is more than one launch
    assert lib.qlin_w4_workspace_size(1 << 17, 1 << 15, 1 << 20) == 0
    assert lib.qlin_w4_workspace_size(32, 5120, 25600) > 0
