// 4-bit products of more than 8 tokens, groups of 128.
#include "qlin_w4_tile.h"

namespace qlin {
namespace w4 {

hipError_t launch_tile_128(const Args &a, hipStream_t s) { return tile_any<128>(a, s); }

}  // namespace w4
}  // namespace qlin
