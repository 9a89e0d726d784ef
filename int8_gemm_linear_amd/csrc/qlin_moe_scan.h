// Running sums over a wave, for counts of experts' slots and tiles.
#pragma once

#include <hip/hip_runtime.h>

namespace qlin {

// v of this lane and all lower ones; every lane of the wave must be active.
// Within each row of 16 lanes four shifts on the data path; the rows' sums are
// read out of their last lanes.  (Six shuffles through the LDS crossbar, one after
// another, and the offsets not loaded ahead: 32 tokens through 128 experts of
// 2048 x 768 25.0 us, so 24.5; one token on 1536 x 2048 10.7 and 10.3.)
__device__ inline int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);     // row_shr:1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    const int r0 = __builtin_amdgcn_readlane(v, 15), r1 = r0 + __builtin_amdgcn_readlane(v, 31),
              r2 = r1 + __builtin_amdgcn_readlane(v, 47);
    const int row = (threadIdx.x & 63) >> 4;
    return v + (row == 0 ? 0 : row == 1 ? r0 : row == 2 ? r1 : r2);
}

}  // namespace qlin
