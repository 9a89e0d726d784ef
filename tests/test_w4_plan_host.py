"""How the 4-bit products divide their work, without a GPU: the library's own
arithmetic (csrc/qlin_w4_plan.h) compiled for the host."""
import math
import os
import random
import subprocess

import pytest

import int8_gemm_linear_amd as q
from tests import w4_cases

CSRC = os.path.join(os.path.dirname(q.LIB_PATH), "csrc")
LOW, HIGH = -(1 << 31), (1 << 31) - 1

PROGRAM = r"""
#include <stdio.h>
#include "qlin_w4_plan.h"
using namespace qlin::w4;
// rows FROM TO ROWS MOST -> first row, rows
// pick M N K GROUP EXPERTS ROWS -> 0 u waves end, or 1 tb rb ks parts end
int main()
{
    char what[8];
    while (scanf("%7s", what) == 1) {
        if (what[0] == 'r') {
            int from, to, rows, most, beg;
            if (scanf("%d %d %d %d", &from, &to, &rows, &most) != 4)
                return 1;
            const int n = expert_rows(from, to, rows, most, beg);
            printf("%d %d\n", beg, n);
            continue;
        }
        long M, N, K, group, experts, rows;
        if (scanf("%ld %ld %ld %ld %ld %ld", &M, &N, &K, &group, &experts, &rows) != 6)
            return 1;
        if (streams(M, N, experts, rows)) {
            const StreamPick p = pick_stream(N, K, experts, rows);
            printf("0 %d %d %d\n", p.u, p.waves, (int)stream_end(K, K / group));
        } else {
            const TilePick p = pick_tile(M, N, K, experts, rows);
            printf("1 %d %d %d %d %d\n", p.tb, p.rb, p.ks, p.splits, (int)tile_end(K, p.ks));
        }
    }
}
"""


def ask(exe, lines):
    """The program's answer to each line, as tuples of numbers."""
    out = subprocess.run([exe], input="\n".join(lines), text=True, capture_output=True, check=True).stdout
    answers = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert len(answers) == len(lines)
    return answers


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
    got = ask(plan, ["rows %d %d %d %d" % c for c in cases])
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


def combination(case, answer):
    """What of a kernel a call comes to: see tests/w4_cases.py."""
    M, N, K, group, experts, rows = case
    if answer[0] == 0:
        return "stream", experts > 0, answer[1], answer[3], group
    return "tile", experts > 0, answer[1], answer[2], answer[4] > 1, answer[5], group


def combinations(plan, cases):
    return [combination(c, a) for c, a in zip(cases, ask(plan, ["pick %d %d %d %d %d %d" % c for c in cases]))]


def test_the_exact_cases_cover_every_kernel_and_tile(plan):
    listed = [(M, N, K, group, 0, 0) for M, N, K, group in w4_cases.DENSE] + \
        [(rows, N, K, group, E, rows) for E, rows, N, K, group in w4_cases.EXPERTS]
    covered = set(combinations(plan, listed))
    rng = random.Random(7)

    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    drawn = []
    while len(drawn) < 60000:
        group = rng.choice([32, 64, 128])
        if rng.random() < 0.6:
            drawn.append((size(1, 1200), size(1, 52000), group * size(1, 25600 // group), group, 0, 0))
        else:
            rows = size(1, 16000)
            drawn.append((rows, size(1, 2500), group * size(1, 4096 // group), group, rng.choice([1, 3, 8, 16, 60, 128]),
                          rows))
    for case, c in zip(drawn, combinations(plan, drawn)):
        assert c in covered, f"no exact test of {c}, as in {case}"
