// attention_cached_e4m3_f32.hip -- attention over caches: the kernels of one
// format and type.
#include "attention_cached.hpp"

namespace mp3d {

template <>
hipError_t launch_cached<F32, kE4M3>(const CachedArgs &c, hipStream_t s)
{
    return run_cached_width<F32, kE4M3>(c, s);
}

}  // namespace mp3d
