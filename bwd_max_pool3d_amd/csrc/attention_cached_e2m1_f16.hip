// attention_cached_e2m1_f16.hip -- attention over caches: the kernels of one
// format and type.
#include "attention_cached.hpp"

namespace mp3d {

template <>
hipError_t launch_cached<F16, kE2M1>(const CachedArgs &c, hipStream_t s)
{
    return run_cached_width<F16, kE2M1>(c, s);
}

}  // namespace mp3d
