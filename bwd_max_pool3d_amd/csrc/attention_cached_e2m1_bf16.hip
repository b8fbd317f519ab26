// attention_cached_e2m1_bf16.hip -- attention over caches: the kernels of one
// format and type.
#include "attention_cached.hpp"

namespace mp3d {

template <>
hipError_t launch_cached<BF16, kE2M1>(const CachedArgs &c, hipStream_t s)
{
    return run_cached_width<BF16, kE2M1>(c, s);
}

}  // namespace mp3d
