// How a 4-bit product is divided: arithmetic on sizes, without GPU code, so that it
// is checked on the host too.
#pragma once

#include <stdint.h>

namespace qlin {
namespace w4 {

// Rows of an expert whose offsets are `from` and `to`, whatever they hold: both are
// held to 0..rows before the difference is taken, which then passes no 32 bits
// (0 and -2^31 are 2^31 apart).  `beg`: its first row; at most `most` rows.
__host__ __device__ inline int expert_rows(int from, int to, int rows, int most, int &beg)
{
    beg = from < 0 ? 0 : from > rows ? rows : from;
    const int end = to < 0 ? 0 : to > rows ? rows : to;
    return end <= beg ? 0 : end - beg < most ? end - beg : most;
}

}  // namespace w4
}  // namespace qlin
