// 4-bit products of few tokens, groups of 64.
#include "qlin_w4_stream.h"

namespace qlin {
namespace w4 {

hipError_t launch_stream_64(const Args &a, hipStream_t s) { return stream_any<64>(a, s); }

}  // namespace w4
}  // namespace qlin
